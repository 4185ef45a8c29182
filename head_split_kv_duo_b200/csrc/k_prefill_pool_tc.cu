// k_prefill_pool_tc.cu -- ragged pre-fill attention over the paged pool on the tcgen05
// tensor cores (bf16 in, fp32 accumulate, head_dim 128, up to 16 query heads per KV head).
//
// The n_s new tokens of each listed sequence s, at positions len_s .. len_s+n_s-1, attend
// ("Chunked Pre-filling", masks of "The Full and Streaming Attention Masks"), scale c:
//   out_i = sum_j p_ij v_j / l_i,  p_ij = exp(c q_i.k_j - m_i),  l_i = sum_j p_ij
//   over  j <= i (retrieval heads),  j <= i and (j < S or i - j < W) (streaming heads)
// with the sums taken in one pass over tiles of 128 keys: a running reference m, and O and
// l rescaled when a row's maximum passes it by 2^8.  Keys come straight from where they
// are: the sequence's pages (one page = one tile), its sinks and ring slots in slot order
// (the softmax does not ask for an order; masks say which slot holds a visible position),
// and the call's own k and v.  The cache is only read; the append is a later launch.
//
// An item is two 128-row query tiles of one (sequence, KV head) -- a row is one of G query
// heads at one of 128 / G consecutive positions (rows past G * (128 / G) idle) -- sharing
// every K/V tile.  The grid is one CTA per SM; a CTA works through whole items and then
// through its share of the last ones, which are cut by key tiles so that every CTA has as
// much to do (few queries over a long history are nothing but that share).
// A cut item's CTAs leave unnormalised rows, max and sum in the scratch; the append launch
// that follows joins them.  12 warps:
//   warp 0      TMA: the K ring (2 stages)
//   warp 1      owns TMEM; one elected lane issues every tcgen05.mma
//   warp 2      TMA: both Q tiles, the V ring (2 stages), but the last tile of a chunk row by row:
//               rows behind it belong to the next sequence, and 0 * NaN would carry a
//               broken neighbour's values over, so they are written as zeros
//   warp 3      lists the CTA's pieces for the others, up to four ahead
//   warps 4-7 and 8-11  softmax of query tile 0 and 1, one thread per row
// TMEM: S_t at 128 t (P_t, bf16 pairs, over its first 64 columns), O_t at 256 + 128 t.
// The MMA thread issues PV_0(j), S_0(j+1), PV_1(j), S_1(j+1): one tile's products run
// while the other tile's softmax works.  MMAs of one thread complete in order, so S_t(j+1)
// overwrites P_t(j) after PV_t(j) has read it, and once S_t(j) has landed O_t may be
// rescaled in place.  The next piece's first products overwrite S_t after the last
// PV_t has read P_t, and O_t after its softmax warps, which have read it out, have
// published their next P_t.
//
// Every mbarrier wait is bounded; one that runs out latches kDevTimeout, and every role
// drains and exits.
//
// Bound: a pair of tiles (256 rows x 128 keys) costs 2048 cycles of the tensor core and as
// many of MUFU (exponentials of two warps per scheduler); it takes 3120 with every SM at
// work (one query tile of 128 rows: 2740), a piece 7400 more, and long calls run at the
// power limit.  8 KV heads (4 of them retrieval heads) of 4 query heads, fork and append included:
//   8192 tokens on 24576: alone 1.51 ms (1.67 GHz), 1.30 PFLOP/s; back to back 1.74 ms, 1.13
//   64 tokens on 131000, back to back: 73 us (0.27 GB and 69 GFLOP: 41 us at either rate)
// Steps from a first version of 1.89 ms and 96 us (one CTA per item, the maximum before the
// exponentials, P handed over whole, lane 0 alone issuing), in that order, each pass alone:
//   products of a tile's first 96 keys start before the other 32 are done, the maximum is
//   checked beside the exponentials, K and V are waited for before P, the issuing warp runs
//   on uniform values (issue 3700 -> 2000 cycles a pair of tiles): 1.61 ms
//   rows out through shared memory, partial rows transposed, masks as two runs: 1.55 ms
//   one site each for listing and storing (84 -> 75 KB of code: the loops then stay in the
//   instruction cache): 1.51 ms
//   even shares by cost: 630 -> 340 us for eight sequences of very different lengths
// Without gain: part of the exponentials as polynomials on the FMA pipe (1.55 to 1.76 ms for
// an eighth to a third of them), P in halves (1.65) or whole (1.54), tiles fetched into L2
// ahead of their loads (73 -> 85 us), listing pieces with a function call.
#include "pool_internal.h"
#include "tcgen05.cuh"

namespace duo {

namespace {

constexpr int kBM = 128, kBN = 128, kD = 128, kQT = 2;
constexpr int kSoftWarp0 = 4;
constexpr int kThreads = 32 * (kSoftWarp0 + 4 * kQT);
constexpr int kKStages = 2, kVStages = 2;
constexpr int kTile = 32768;  // bytes of a 128-row operand tile: two 128B-swizzled [128][64] halves
constexpr int kHalf = 16384;

constexpr int kSmQ = 0, kSmK = kSmQ + kQT * kTile, kSmV = kSmK + kKStages * kTile, kSmBar = kSmV + kVStages * kTile;
constexpr int kSmMisc = kSmBar + 256;
constexpr int kPieces = 4;  // pieces listed ahead
constexpr int kSmOut = kSmMisc + 768;  // per softmax warp: 32 rows' 32 dims on their way out
constexpr int kSmLists = kSmOut + 4 * kQT * 2048;
constexpr int kSmemAlloc = kSmLists + static_cast<int>(sizeof(PrefillLists)) + 1024;  // slack: the base at 1 KiB
constexpr int kTmS = 0, kTmO = 256;
constexpr int kPFirst = 96;  // keys of a tile whose P is handed over first

constexpr int kBarQ = 0, kBarQEmpty = 1, kBarKFull = 2, kBarKEmpty = kBarKFull + kKStages,
              kBarVFull = kBarKEmpty + kKStages, kBarVEmpty = kBarVFull + kVStages, kBarSFull = kBarVEmpty + kVStages,
              kBarPFull = kBarSFull + kQT, kBarPRest = kBarPFull + kQT, kBarOFull = kBarPRest + kQT,
              kBarPiece = kBarOFull + kQT, kBarPieceFree = kBarPiece + kPieces, kBarDrain = kBarPieceFree + kPieces, kBarStall = kBarDrain + 1, kNumBars = kBarStall + 1;
static_assert(kNumBars * 8 <= 256 && kSmemAlloc <= 227 * 1024, "shared memory");

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// A piece of a CTA's work: key tiles [j0, j0 + nt) of an item.
struct Piece {
  int g, idx, retr;     // KV head, its index among heads of its kind
  int len, n, slot, tok0;
  int r0, nq;           // first position in the chunk, query tiles
  int j0, nt;           // nt = 0: the CTA's work is done
  int part;             // partial rows' place in the scratch, -1: the whole item
  PrefillRun runs[kPrefillMaxRuns];
};
static_assert(sizeof(Piece) * kPieces + 16 <= 768, "shared memory");
struct Tile {
  int src, y;  // source, first row
};

// Item `u` of the call; its tiles go into `runs`.  Returns how many there are.
__device__ __forceinline__ int item_of(const PoolPrefillCall &c, const PrefillLists &lists, int u, Piece &w) {
  w.retr = u < c.retr_items;
  const int *first = w.retr ? lists.rfirst : lists.sfirst;
  const int v = w.retr ? u : u - c.retr_items;
  int lo = 0, hi = c.nseq - 1;  // the last sequence with first <= v
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= v) lo = mid;
    else hi = mid - 1;
  }
  w.len = lists.len[lo];
  w.n = lists.n[lo];
  w.slot = lists.slot[lo];
  w.tok0 = lists.tok0[lo];
  // heads fastest (neighbours in the grid read different heads' keys at the same places),
  // query blocks from the last -- the longest -- to the first
  const int npos = c.npos, heads = w.retr ? c.Hr : c.Hs, rem = v - first[lo], back = rem / heads;
  w.idx = rem - back * heads;
  w.g = w.retr ? lists.retr_head[w.idx] : lists.strm_head[w.idx];
  w.r0 = (lists.blocks[lo] - 1 - back) * kQT * npos;
  w.nq = w.n - w.r0 > npos ? kQT : 1;
  const int k = prefill_runs(w.retr, w.len, w.n, w.r0, npos, c.S, c.W, w.runs);
  int tiles = 0;
  for (int i = 0; i < k; ++i) tiles += w.runs[i].count;
  return tiles;
}
__device__ __forceinline__ Tile tile_at(const PrefillRun *runs, int j) {
  while (j >= runs->count) {
    j -= runs->count;
    ++runs;
  }
  return {runs->src, (runs->first + j) * kBN};
}

// bits below x (x <= 0: none, x >= 32: all)
__device__ __forceinline__ uint32_t bits_below(int x) {
  uint32_t r;
  asm("shl.b32 %0, 0xffffffff, %1;" : "=r"(r) : "r"(max(x, 0)));  // a shift by 32 or more gives 0
  return ~r;
}

// 128 consecutive fp32 columns of this thread's lane; one wait that names every register,
// so that no use is scheduled before it
#define DUO_R4(x) "+r"(r[(x)]), "+r"(r[(x) + 1]), "+r"(r[(x) + 2]), "+r"(r[(x) + 3])
#define DUO_R16(x) DUO_R4(x), DUO_R4((x) + 4), DUO_R4((x) + 8), DUO_R4((x) + 12)
__device__ __forceinline__ void load_row(uint32_t taddr, float (&v)[128]) {
  uint32_t r[128];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t *q = r + 32 * c;
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]), "=r"(q[8]),
          "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15]), "=r"(q[16]),
          "=r"(q[17]), "=r"(q[18]), "=r"(q[19]), "=r"(q[20]), "=r"(q[21]), "=r"(q[22]), "=r"(q[23]), "=r"(q[24]),
          "=r"(q[25]), "=r"(q[26]), "=r"(q[27]), "=r"(q[28]), "=r"(q[29]), "=r"(q[30]), "=r"(q[31])
        : "r"(taddr + 32 * c));
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : DUO_R16(0), DUO_R16(16), DUO_R16(32), DUO_R16(48), DUO_R16(64), DUO_R16(80), DUO_R16(96), DUO_R16(112)
               :
               : "memory");
#pragma unroll
  for (int i = 0; i < 128; ++i) v[i] = __uint_as_float(r[i]);
}
#undef DUO_R4
#undef DUO_R16

__device__ __forceinline__ float largest(const float (&v)[128]) {
  float m[8];  // independent chains of three-input maxima
#pragma unroll
  for (int u = 0; u < 8; ++u) m[u] = fmaxf(v[2 * u], v[2 * u + 1]);
#pragma unroll
  for (int e = 16; e < 128; e += 2) {
    float &x = m[(e >> 1) & 7];
    asm("max.f32 %0, %1, %2, %3;" : "=f"(x) : "f"(x), "f"(v[e]), "f"(v[e + 1]));
  }
#pragma unroll
  for (int u = 4; u > 0; u >>= 1)
#pragma unroll
    for (int i = 0; i < u; ++i) m[i] = fmaxf(m[i], m[i + u]);
  return m[0];
}

// P = exp2(c v - mc) of logits v[32 B .. 32 B + 32) as bf16 pairs into columns 16 B .. of
// `cols` (not waited for); returns their fp32 sum.  P is rounded to bf16 for the tensor core,
// which takes both operands in one type, V's: half a step, 2^-8 relative at most, of random
// sign over a row.  With the output's own rounding that is 2.2e-3 of the result's norm
// against 64 bits, where a P of 32 bits leaves 1.7e-3; P as two bf16 parts would cost a
// second product.  The sum takes the unrounded values, and lse is that of 32 bits.
template <int B>
__device__ __forceinline__ float probabilities(const float (&v)[128], float c, float mc, uint32_t cols) {
  const uint64_t cc = pack2(c, c), mm = pack2(-mc, -mc);
  uint64_t sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
  uint32_t pk[16];
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float x0, x1;
    unpack2(ffma2(pack2(v[32 * B + e], v[32 * B + e + 1]), cc, mm), x0, x1);
    x0 = ex2(x0);
    x1 = ex2(x1);
    sum[(e >> 1) & 1] = fadd2(sum[(e >> 1) & 1], pack2(x0, x1));
    const __nv_bfloat162 b = __floats2bfloat162_rn(x0, x1);
    pk[e >> 1] = *reinterpret_cast<const uint32_t *>(&b);
  }
  tc::st16(cols + 16 * B, pk);
  float a0, a1, b0, b1;
  unpack2(sum[0], a0, a1);
  unpack2(sum[1], b0, b1);
  return (a0 + a1) + (b0 + b1);
}

// A V tile whose rows from `valid` on are not the sequence's: a warp copies its rows and
// writes zeros behind them, in the layout a swizzled TMA load leaves.
__device__ __forceinline__ void copy_ragged_tile(const char *src, int64_t row_bytes, int valid, uint32_t dst,
                                                 int lane) {
  for (int i = lane; i < kBN * 16; i += 32) {
    const int row = i >> 4, chunk = i & 15;
    const uint32_t to = dst + (chunk >> 3) * kHalf + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
    const char *from = src + (row < valid ? row : 0) * row_bytes + chunk * 16;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(row < valid ? 16 : 0)
                 : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  tc::fence_async_smem();
}

__global__ void __launch_bounds__(kThreads, 1) prefill_pool_kernel(const __grid_constant__ PoolPrefillCall c) {
  extern __shared__ char smem_raw[];
  char *smem = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + kSmBar + 8u * i; };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kSmMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kSmMisc + 4);
  Piece *pieces = reinterpret_cast<Piece *>(smem + kSmMisc + 16);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int npos = c.npos;
  PrefillLists &lists = *reinterpret_cast<PrefillLists *>(smem + kSmLists);

  // What is done before griddepcontrol.wait overlaps the end of the kernel before: barriers,
  // the first pieces' listing and fetching the tensor maps touch no memory of its.  The
  // lists are copied side by side: read one by one as parameters, each first touch would
  // wait for the constant cache.
  static_assert(sizeof(PrefillLists) / 16 <= 2 * kThreads, "two vectors a thread");
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = tid + k * kThreads;
    if (i < static_cast<int>(sizeof(PrefillLists) / 16))
      reinterpret_cast<uint4 *>(&lists)[i] = reinterpret_cast<const uint4 *>(&c.lists)[i];
  }
  if (tid < kNumBars) {
    const bool softmax = tid >= kBarPFull && tid < kBarPFull + 2 * kQT;
    const bool listed = tid >= kBarPieceFree && tid < kBarPieceFree + kPieces;
    mbar_init(bar(tid), softmax ? kBM / 32 : listed ? 3 + 4 * kQT : 1);
    fence_mbar_init();
    if (tid == 0) *abort_flag = 0;
  }
  static_assert(kNumBars <= 32, "one thread a barrier");
  if (tid >= 32 && tid < 39) tc::prefetch_map(&c.tm_q + (tid - 32));
  __syncthreads();
  uint32_t tmem = 0;
  if (warp != 3) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 1 || warp >= kSoftWarp0) {  // (tensor memory: a kernel before may still have wanted some)
      if (warp == 1) tc::tmem_alloc(smem_u32(tmem_slot), 512);
      tc::fence_before();
      tc::named_sync(1, 32 * (1 + 4 * kQT));
      tc::fence_after();
      tmem = *tmem_slot;
    }
  }

  // The roles take the pieces in order: piece p is at p % kPieces while they hold it.
  auto take = [&](int p, bool &ok) -> const Piece * {
    if (ok) ok = tc::wait_bar(bar(kBarPiece + p % kPieces), (p / kPieces) & 1, c.status, abort_flag);
    return ok ? pieces + p % kPieces : nullptr;
  };
  auto leave = [&](int p) { mbar_arrive(bar(kBarPieceFree + p % kPieces)); };

  // Shares of the launch's 384 * 168 registers: the softmax warps hold a row of logits.
  if (warp < kSoftWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 3) {
      // ================= lists the pieces =================
      if (lane == 0) {
        int p = 0;
        bool ok = true;
        auto slot = [&]() -> Piece * {
          if (p >= kPieces)
            ok = tc::wait_bar(bar(kBarPieceFree + p % kPieces), (p / kPieces - 1) & 1, c.status, abort_flag);
          return ok ? pieces + p % kPieces : nullptr;
        };
        auto publish = [&] {
          mbar_arrive(bar(kBarPiece + p % kPieces));
          ++p;
        };
        const PrefillShare sh = lists.share[blockIdx.x];
        int u = blockIdx.x, j0 = 0, left = sh.tiles;
        while (ok) {
          const bool whole = u < c.whole_items;
          if (!whole && left == sh.tiles) {  // on to the share
            u = sh.item;
            j0 = sh.tile;
          }
          if (!whole && left == 0) break;
          Piece *w = slot();
          if (!ok) break;
          const int tiles = item_of(c, lists, u, *w), nt = whole ? tiles : min(tiles - j0, left);
          w->j0 = j0;
          w->nt = nt;
          w->part = nt == tiles ? -1 : (u == sh.item ? sh.part : sh.part + 1);
          publish();
          u += whole ? gridDim.x : 1;
          if (!whole) {
            left -= nt;
            j0 = 0;
          }
        }
        if (ok) {
          Piece *w = slot();
          if (ok) {
            w->nt = 0;
            publish();
          }
        }
      }
    } else if (warp == 0 || warp == 2) {
      // ================= producers: warp 0 K, warp 2 Q and V =================
      const bool is_k = warp == 0;
      const uint32_t stage0 = sbase + (is_k ? kSmK : kSmV);
      const int full0 = is_k ? kBarKFull : kBarVFull, empty0 = is_k ? kBarKEmpty : kBarVEmpty;
      constexpr int kStages = kKStages;
      static_assert(kKStages == kVStages, "one producer loop for both rings");
      int issued = 0, queries = 0;
      bool ok = true;
      for (int p = 0;; ++p) {
        const Piece *w = take(p, ok);
        if (!__all_sync(0xffffffffu, ok) || w->nt == 0) break;
        if (!is_k) {
          if (lane == 0 && p > 0) ok = tc::wait_bar(bar(kBarQEmpty), (p - 1) & 1, c.status, abort_flag);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0);
          if (!ok) break;
          if (lane == 0) {
            mbar_expect_tx(bar(kBarQ), 256 * c.G * npos * w->nq);
            for (int q = 0; q < w->nq; ++q)
              for (int h = 0; h < 2; ++h)  // box: 64 dims x G heads x npos positions
                tc::tma_3d(sbase + kSmQ + q * kTile + h * kHalf, &c.tm_q, 64 * h, w->g * c.G,
                           w->tok0 + w->r0 + q * npos, bar(kBarQ));
          }
          ++queries;
        }
        const CUtensorMap *pages = is_k ? &c.tm_kr : &c.tm_vr, *slots = is_k ? &c.tm_ks : &c.tm_vs;
        const CUtensorMap *chunk = is_k ? &c.tm_k : &c.tm_v;
        const int *row = c.table + static_cast<int64_t>(w->slot) * c.pages_per_seq;
        Tile t = tile_at(w->runs, w->j0);
        int page = t.src == kPages ? row[t.y / kBN] : 0;
        for (int j = 0; j < w->nt; ++j) {
          const int s = issued % kStages;
          // the next tile's page number is on its way while this one waits for its stage
          Tile next = t;
          int next_page = 0;
          if (j + 1 < w->nt) {
            next = tile_at(w->runs, w->j0 + j + 1);
            if (next.src == kPages) next_page = row[next.y / kBN];
          }
          if (lane == 0 && issued >= kStages)
            ok = tc::wait_bar(bar(empty0 + s), ((issued / kStages) - 1) & 1, c.status, abort_flag);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0);
          if (!ok) break;
          const uint32_t dst = stage0 + s * kTile, fb = bar(full0 + s);
          const int valid = t.src == kChunk ? w->n - t.y : kBN;
          if (!is_k && valid < kBN) {
            copy_ragged_tile(c.v + (static_cast<int64_t>(w->tok0 + t.y) * c.Hkv + w->g) * 256,
                             static_cast<int64_t>(c.Hkv) * 256, valid, dst, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(fb);
          } else if (lane == 0) {
            mbar_expect_tx(fb, kTile);
            for (int h = 0; h < 2; ++h) {
              const uint32_t to = dst + h * kHalf;
              if (t.src == kPages) tc::tma_3d(to, pages, 64 * h, 0, page * c.Hr + w->idx, fb);
              else if (t.src == kSlots) tc::tma_3d(to, slots, 64 * h, t.y, w->slot * c.Hs + w->idx, fb);
              else tc::tma_3d(to, chunk, 64 * h, w->g, w->tok0 + t.y, fb);
            }
          }
          ++issued;
          t = next;
          page = next_page;
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) leave(p);
      }
      if (lane == 0) {  // nothing may still be landing in shared memory when the CTA ends
        if (queries > 0) mbar_wait(bar(kBarQ), (queries - 1) & 1, c.status);
        tc::drain_loads(bar(full0), kStages, issued, c.status);
      }
    } else {
      // ================= MMA issuer =================
      // The warp runs the loop as one, on values that are the same in all its lanes, and one
      // elected lane issues: descriptors then stay in uniform registers.
      constexpr uint32_t kIdS = tc::idesc_bf16(kBM, kBN, false, false);
      constexpr uint32_t kIdPV = tc::idesc_bf16(kBM, kD, false, true);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      // operands lie below 256 KiB, so one at byte offset o is the base's descriptor + (o >> 4)
      const uint64_t qd0 = tc::sdesc(sbase + kSmQ, 16, 1024), kd0 = tc::sdesc(sbase + kSmK, 16, 1024);
      const uint64_t vd0 = tc::sdesc(sbase + kSmV, kHalf, 1024);
      auto wait = [&](int b, int phase) {
        return __all_sync(0xffffffffu, tc::wait_bar(bar(b), phase & 1, c.status, abort_flag)) != 0;
      };
      // S_t = Q_t K^T with the K tile of stage s, d 128 in 8 steps of 16
      auto issue_s = [&](int t, int s) {
        const uint64_t qd = qd0 + t * (kTile >> 4), kd = kd0 + s * (kTile >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t o = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
          tc::mma_ss(tm + kTmS + t * 128, qd + o, kd + o, kIdS, kk > 0 ? 1u : 0u);
        }
        tc::commit(bar(kBarSFull + t));
      };
      // O_t (+)= P_t V with the V tile of stage s, 128 keys in 8 steps of 16
      auto issue_pv = [&](int t, int s, bool first, int from, int to) {
        const uint64_t vd = vd0 + s * (kTile >> 4);
#pragma unroll
        for (int kk = from; kk < to; ++kk)
          tc::mma_ts(tm + kTmO + t * 128, tm + kTmS + t * 128 + kk * 8, vd + kk * (2048 >> 4), kIdPV,
                     kk > 0 || !first ? 1u : 0u);
      };
      bool ok = true;
      int k_tile = 0, v_tile = 0, p_tile[kQT] = {0, 0};
      for (int p = 0;; ++p) {
        const Piece *w = take(p, ok);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int nt = __shfl_sync(0xffffffffu, w->nt, 0), nq = __shfl_sync(0xffffffffu, w->nq, 0);
        if (lane == 0) leave(p);
        if (nt == 0) break;
        ok = wait(kBarQ, p) && wait(kBarKFull + k_tile % kKStages, k_tile / kKStages);
        if (!ok) break;
        tc::fence_after();
        if (elect()) {
          issue_s(0, k_tile % kKStages);
          if (nq > 1) issue_s(1, k_tile % kKStages);
          tc::commit(bar(kBarKEmpty + k_tile % kKStages));
          if (nt == 1) tc::commit(bar(kBarQEmpty));
        }
        __syncwarp();
        ++k_tile;
        for (int j = 0; j < nt && ok; ++j) {
#pragma unroll
          for (int t = 0; t < kQT; ++t) {
            if (t >= nq || !ok) break;
            // K and V first: they are there long before P, and only P should be waited for
            if (t == 0) ok = wait(kBarVFull + v_tile % kVStages, v_tile / kVStages);
            if (ok && t == 0 && j + 1 < nt) ok = wait(kBarKFull + k_tile % kKStages, k_tile / kKStages);
            if (ok) ok = wait(kBarPFull + t, p_tile[t]);
            if (!ok) break;
            tc::fence_after();
            if (elect()) issue_pv(t, v_tile % kVStages, j == 0, 0, kPFirst / 16);
            __syncwarp();
            ok = wait(kBarPRest + t, p_tile[t]);
            ++p_tile[t];
            if (!ok) break;
            tc::fence_after();
            if (elect()) {
              issue_pv(t, v_tile % kVStages, false, kPFirst / 16, 8);
              if (t == nq - 1) tc::commit(bar(kBarVEmpty + v_tile % kVStages));
              if (j + 1 == nt) {
                tc::commit(bar(kBarOFull + t));
              } else {
                issue_s(t, k_tile % kKStages);
                if (t == nq - 1) {
                  tc::commit(bar(kBarKEmpty + k_tile % kKStages));
                  if (j + 2 == nt) tc::commit(bar(kBarQEmpty));
                }
              }
            }
            __syncwarp();
            if (t == nq - 1) {
              ++v_tile;
              if (j + 1 < nt) ++k_tile;
            }
          }
        }
      }
      // every MMA issued has completed before TMEM is freed
      if (elect()) {
        tc::commit(bar(kBarDrain));
        mbar_wait(bar(kBarDrain), 0, c.status);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ================= softmax of query tile qt: one thread per query row =================
    constexpr float kSlack = 8.0f;
    const int qt = (warp - kSoftWarp0) >> 2, row = ((warp & 3) << 5) | lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) << 5) << 16);
    const uint32_t s_cols = lane_base + kTmS + qt * 128, o_cols = lane_base + kTmO + qt * 128;
    const float scale = c.scale_log2;
    bool ok = true;
    int s_tile = 0, done = 0;  // tiles and pieces of this query tile so far
    for (int p = 0;; ++p) {
      const Piece *w = take(p, ok);
      if (!__all_sync(0xffffffffu, ok) || w->nt == 0) break;
      if (qt >= w->nq) {
        __syncwarp();
        if (lane == 0) leave(p);
        continue;
      }
      const int len = w->len, n = w->n, nt = w->nt, retr = w->retr;
      const int rpos = w->r0 + qt * npos + row / c.G;  // position of the row in the chunk
      const int i = len + rpos;                        // and in the sequence
      float m = -INFINITY, l = 0.f;
      const PrefillRun *run = w->runs;
      int skip = w->j0;
      for (; skip >= run->count; ++run) skip -= run->count;
      Tile next = {run->src, (run->first + skip) * kBN};
      int left = run->count - skip;
      // Slots that row i sees: [0, front) and [ring.lo2, ring.hi2).  Either run of the ring
      // starts at its first slot, and continues the sinks, or the other run is empty.
      PrefillRing ring = prefill_ring(i, len, c.S, c.W);
      int front = min(c.S, len);
      if (ring.lo1 == c.S) {
        front = max(front, ring.hi1);
      } else {
        ring.lo2 = ring.lo1;
        ring.hi2 = ring.hi1;
      }

      for (int j = 0; j < nt; ++j) {
        // columns of the tile that this row sees; most tiles are seen whole
        const Tile t = next;
        // columns [0, front_t) and [from, to) of it
        int front_t, from = 0, to = 0;
        if (t.src == kPages) {
          front_t = len - t.y;
        } else if (t.src == kSlots) {
          front_t = front - t.y;
          from = ring.lo2 - t.y;
          to = ring.hi2 - t.y;
        } else {
          const int base = len + t.y;
          front_t = to = min(i - base + 1, n - t.y);
          if (!retr) {
            front_t = min(to, c.S - base);
            from = i - c.W + 1 - base;
          }
        }
        const bool whole = front_t >= kBN || (from <= max(front_t, 0) && to >= kBN);

        if (--left > 0) {
          next.y += kBN;
        } else if (j + 1 < nt) {
          ++run;
          left = run->count;
          next = {run->src, run->first * kBN};
        }

        if (c.debug_stall && p == 0 && j == 0 && ok) ok = tc::wait_bar(bar(kBarStall), 0, c.status, abort_flag);
        if (ok) ok = tc::wait_bar(bar(kBarSFull + qt), s_tile & 1, c.status, abort_flag);
        ++s_tile;
        tc::fence_after();
        float v[128];
        load_row(s_cols, v);
        if (!whole) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t vis = bits_below(front_t - 32 * k) | (bits_below(to - 32 * k) & ~bits_below(from - 32 * k));
            if (vis != ~0u) {  // a warp's rows are few positions: most groups of 32 are seen whole
#pragma unroll
              for (int e = 0; e < 32; ++e) v[32 * k + e] = (vis >> e) & 1u ? v[32 * k + e] : -INFINITY;
            }
          }
        }
        // Weights relative to the reference m so far, their largest logit beside them; when
        // it passes m by 2^8 (rare after the first tiles) m moves, O_t and l are rescaled and
        // the weights are done again.  S_t(j) has landed, so P_t(j-1) V_{j-1} has too and O_t
        // may be rescaled in place.
        float alpha = 1.f, sum;
        if (j == 0) m = largest(v) * scale;  // -inf when the row sees nothing of the tile
        while (true) {
          const float mc = m == -INFINITY ? 0.f : m;  // masked logits are -inf and give 0
          sum = probabilities<0>(v, scale, mc, s_cols) + probabilities<1>(v, scale, mc, s_cols);
          sum += probabilities<2>(v, scale, mc, s_cols);
          const float tmax = largest(v) * scale;
          const bool need = tmax > m + kSlack;
          if (!__any_sync(0xffffffffu, need)) break;
          // stores land in no order: these weights before the ones that go over them.  (Here: the
          // same wait behind the loop below made long calls 3 to 6 % slower, 2.59 for 2.51 M
          // cycles, 8192 tokens on 24576, by how the compiler laid it out.)
          tc::st_wait();
          const float a = need ? ex2(m - tmax) : 1.f;  // 0 while m is -inf
          if (need) m = tmax;
          alpha *= a;
#pragma unroll 1
          for (int q = 0; q < 8; ++q) {
            float x[16];
            tc::ld<16>(o_cols + 16 * q, x);
            uint32_t u[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(x[e] * a);
            tc::st16(o_cols + 16 * q, u);
          }
        }
        tc::st_wait();
        tc::fence_before();
        mbar_arrive_warp(bar(kBarPFull + qt));
        sum += probabilities<3>(v, scale, m == -INFINITY ? 0.f : m, s_cols);
        tc::st_wait();
        tc::fence_before();
        mbar_arrive_warp(bar(kBarPRest + qt));
        l = fmaf(l, alpha, sum);
      }
      const int part = w->part, tok = w->tok0 + rpos, head = w->g * c.G + row % c.G;
      const bool live = row < c.G * npos && rpos < n;
      __syncwarp();
      if (lane == 0) leave(p);
      if (ok) ok = tc::wait_bar(bar(kBarOFull + qt), done & 1, c.status, abort_flag);
      ++done;
      tc::fence_after();
      if (part >= 0) {
        // a piece's rows as they are, 16 bytes of 128 rows side by side; a row may have seen
        // nothing (m = -inf, l = 0)
        float4 *to = reinterpret_cast<float4 *>(c.partials) + (part * kQT + qt) * (kPrefillRow / 4) * kBM + row;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          float x[32];
          tc::ld<32>(o_cols + 32 * q, x);
          if (live) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              to[(8 * q + e) * kBM] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
          }
        }
        if (live) to[(kD / 4) * kBM] = make_float4(m, l, 0.f, 0.f);
      } else {
        const int64_t at = live ? static_cast<int64_t>(tok) * c.Hq + head : -1;
        const float inv = 1.f / l;
        // through shared memory: a warp's store then covers eight rows' 64 bytes
        uint4 *out = reinterpret_cast<uint4 *>(smem + kSmOut + (warp - kSoftWarp0) * 2048);
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          float x[32];
          tc::ld<32>(o_cols + 32 * q, x);
          __syncwarp();
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t b16[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(x[8 * u + 2 * e] * inv, x[8 * u + 2 * e + 1] * inv);
              b16[e] = *reinterpret_cast<const uint32_t *>(&b);
            }
            out[lane * 4 + (u ^ ((lane >> 1) & 3))] = make_uint4(b16[0], b16[1], b16[2], b16[3]);
          }
          __syncwarp();
          uint4 y[4];
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const int r = 8 * it + (lane >> 2);
            y[it] = out[r * 4 + ((lane & 3) ^ ((r >> 1) & 3))];
          }
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const int64_t to = __shfl_sync(0xffffffffu, at, 8 * it + (lane >> 2));
            if (to >= 0) *reinterpret_cast<uint4 *>(c.out + to * (kD * 2) + q * 64 + (lane & 3) * 16) = y[it];
          }
        }
        if (live && c.lse) c.lse[at] = (m + lg2(l)) * kLn2;
      }
      // O_t has been read: ordered before the next piece's first P_t, which frees it
      tc::fence_before();
    }
  }

  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 1) tc::tmem_free(tmem, 512);
}

}  // namespace

// Every host step that can fail: tensor maps, the shared-memory limit.
cudaError_t prepare_prefill_pool_tc(PoolPrefillCall *c, const void *q, const void *k, const void *v, int tokens) {
  const uint64_t row = kD * 2, T = static_cast<uint64_t>(tokens);
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const uint64_t dq[3] = {kD, static_cast<uint64_t>(c->Hq), T}, sq[2] = {row, row * c->Hq};
  const uint32_t bq[3] = {64, static_cast<uint32_t>(c->G), static_cast<uint32_t>(kBM / c->G)};
  const uint64_t dk[3] = {kD, static_cast<uint64_t>(c->Hkv), T}, sk[2] = {row, row * c->Hkv};
  const uint32_t bk[3] = {64, 1, kBN};
  if (!tc::make_map(&c->tm_q, bf, q, 3, dq, sq, bq, sw) || !tc::make_map(&c->tm_k, bf, k, 3, dk, sk, bk, sw) ||
      !tc::make_map(&c->tm_v, bf, v, 3, dk, sk, bk, sw))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> attr{0};
  return opt_in_smem(prefill_pool_kernel, kSmemAlloc, attr);
}

cudaError_t launch_prefill_pool_tc(const PoolPrefillCall &c, cudaStream_t st) {
  return launch_overlapped(prefill_pool_kernel, c.ctas, kThreads, kSmemAlloc, st, c);
}

}  // namespace duo
