// pool_prefill.cu -- duo_pool_prefill: ragged pre-fill attention over the paged pool.  The
// attention is k_prefill_pool_tc.cu; here are the plan of a call, and its last launch,
// which joins split rows and appends the tokens.
//
// A row whose keys were cut into pieces with partial sums O_s, maxima m_s (base 2) and
// weights l_s is O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, M = max m_s, lse = (M +
// log2 of the denominator) ln 2; pieces in order, so a result does not depend on timing.
//
// The last launch is bound by latency when it is short (4 to 5 us: parameters, partial
// rows, stores, one after the other) and by the partial rows otherwise: 8192 tokens on
// 24576, 28 MB of them and 33 MB of k and v in, 17 MB of rows out, 18 us.
#include <cmath>
#include <exception>

#include "device_common.cuh"
#include "nvtx_range.h"
#include "pool_internal.h"

namespace duo {

namespace {

// An item whose key tiles several CTAs share: its query rows and the places of its pieces
// in the scratch, part0, part1, part1 + 2, ...
struct PrefillCut {
  int n, tok0;  // of its sequence
  int block, head, pieces, part0, part1;
  int join0;  // blocks of the last launch that join cuts before it
};
struct FinishSeq {
  int slot, len, n, tok0;
  int page0;  // its entries in `pages`, from logical page len / 128 on
  int unused[3];
};

// The call's last launch, sequences in the caller's order (and one that starts where the
// last ends).  What belongs together lies together: a short launch waits for the first
// touch of every line of its parameters.
struct PoolFinishCall {
  const HeadMap *hm;  // device
  char *rk, *rv, *sk, *sv;
  int *table;
  int pages_per_seq;
  const char *k, *v;
  char *out;
  float *lse;
  const float *partials;
  int nseq, tokens, Hq, Hkv, Hr, Hs, G, S, W, npos, npages, ncuts, join_blocks;
  FinishSeq seq[kPoolMaxSeqs + 1];
  uint8_t cut_of[4 * kPrefillCtas];  // of each kJoinGroups blocks that join
  PrefillCut cuts[kPrefillCtas];
  int pages[kPrefillMaxPages];
};

// the last sequence with first <= x, of those where `first` is its tok0 or page0
template <int FinishSeq::*kFirst>
__device__ __forceinline__ int find(const PoolFinishCall &c, int x) {
  int lo = 0, hi = c.nseq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (c.seq[mid].*kFirst <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A block joins sixteen dimensions of a cut item's 256 rows, one thread per row, two pieces'
// loads in flight (three blocks an SM; with four in flight, two); or, of more than four
// pieces, of 64 of its rows, four threads per row, each joining every fourth piece, and the
// first of them the four.
constexpr int kJoinVecs = 4;   // float4 vectors of a thread
constexpr int kJoinAhead = 2;  // pieces whose loads are in flight
constexpr int kJoinGroups = 32 / kJoinVecs;
static_assert(kPrefillCtas <= 256, "cut_of");
__host__ __device__ inline int join_threads(int pieces) { return pieces > 4 ? 4 : 1; }
__device__ __forceinline__ void join_rows(const PoolFinishCall &c, int block) {
  __shared__ float others[3][2 + 4 * kJoinVecs][64];
  const PrefillCut &cut = c.cuts[c.cut_of[block / kJoinGroups]];
  const int pieces = cut.pieces, threads = join_threads(pieces), rows = kPrefillRows / threads;
  const int local = block - cut.join0, group = local % kJoinGroups * kJoinVecs, thread = threadIdx.x / rows;
  const int r = local / kJoinGroups * rows + threadIdx.x % rows, tile = r / 128, row = r % 128;
  const int pos = (cut.block * 2 + tile) * c.npos + row / c.G;
  const bool live = row < c.G * c.npos && pos < cut.n;
  if (threads == 1 && !live) return;
  auto part = [&](int i) {
    const int place = i == 0 ? cut.part0 : cut.part1 + 2 * (i - 1);
    return reinterpret_cast<const float4 *>(c.partials) + (place * 2 + tile) * (kPrefillRow / 4) * 128 + row;
  };
  float m = -INFINITY, l = 0.f, o[4 * kJoinVecs] = {};
  for (int i0 = thread; i0 < pieces && live; i0 += kJoinAhead * threads) {
    float4 ml[kJoinAhead], x[kJoinAhead][kJoinVecs];
#pragma unroll
    for (int e = 0; e < kJoinAhead; ++e) {
      ml[e] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
      const bool there = i0 + e * threads < pieces;
      const float4 *p = part(there ? i0 + e * threads : i0);
      if (there) ml[e] = p[32 * 128];
#pragma unroll
      for (int k = 0; k < kJoinVecs; ++k) {
        x[e][k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (there) x[e][k] = p[(group + k) * 128];
      }
    }
    float top = m;
#pragma unroll
    for (int e = 0; e < kJoinAhead; ++e) top = fmaxf(top, ml[e].x);
    if (top == -INFINITY) continue;  // the row saw nothing so far
    const float old = ex2(m - top);  // 0 while m is -inf
    m = top;
    l *= old;
#pragma unroll
    for (int k = 0; k < 4 * kJoinVecs; ++k) o[k] *= old;
#pragma unroll
    for (int e = 0; e < kJoinAhead; ++e) {
      const float w = ex2(ml[e].x - m);
      l = fmaf(ml[e].y, w, l);
#pragma unroll
      for (int k = 0; k < kJoinVecs; ++k) {
        o[4 * k] = fmaf(w, x[e][k].x, o[4 * k]);
        o[4 * k + 1] = fmaf(w, x[e][k].y, o[4 * k + 1]);
        o[4 * k + 2] = fmaf(w, x[e][k].z, o[4 * k + 2]);
        o[4 * k + 3] = fmaf(w, x[e][k].w, o[4 * k + 3]);
      }
    }
  }
  if (threads > 1) {
    const int i = threadIdx.x % 64;
    if (thread > 0) {
      float *to = &others[thread - 1][0][i];
      to[0] = m;
      to[64] = l;
#pragma unroll
      for (int k = 0; k < 4 * kJoinVecs; ++k) to[64 * (2 + k)] = o[k];
    }
    __syncthreads();
    if (thread > 0 || !live) return;
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      const float *from = &others[t][0][i];
      const float top = fmaxf(m, from[0]);
      if (top == -INFINITY) continue;
      const float a = ex2(m - top), b = ex2(from[0] - top);
      m = top;
      l = l * a + from[64] * b;
#pragma unroll
      for (int k = 0; k < 4 * kJoinVecs; ++k) o[k] = o[k] * a + from[64 * (2 + k)] * b;
    }
  }
  const float inv = 1.f / l;
  const int64_t out = static_cast<int64_t>(cut.tok0 + pos) * c.Hq + cut.head * c.G + row % c.G;
#pragma unroll
  for (int k = 0; k < kJoinVecs / 2; ++k) {
    uint32_t b16[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(o[8 * k + 2 * e] * inv, o[8 * k + 2 * e + 1] * inv);
      b16[e] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(c.out + out * 256 + group * 8 + k * 16) = make_uint4(b16[0], b16[1], b16[2], b16[3]);
  }
  if (group == 0 && c.lse) c.lse[out] = (m + lg2(l)) * kLn2;
}

// Blocks: those that join cut items; then warps, one per (eight tokens, KV head), K on the
// lower lanes, V on the upper; then one per (sequence, retrieval head) for the rest of a
// page that the call opened, and the block-table entries.
constexpr int kAppendTokens = 8;
__global__ void __launch_bounds__(256, 3) pool_prefill_finish_kernel(const __grid_constant__ PoolFinishCall c) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (static_cast<int>(blockIdx.x) < c.join_blocks) return join_rows(c, blockIdx.x);
  int64_t w = (static_cast<int64_t>(blockIdx.x - c.join_blocks) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t append = static_cast<int64_t>((c.tokens + kAppendTokens - 1) / kAppendTokens) * c.Hkv;
  if (w < append) {
    const int t0 = static_cast<int>(w / c.Hkv) * kAppendTokens, g = static_cast<int>(w % c.Hkv);
    const int idx = c.hm->kind_idx[g];
    const bool is_k = lane < 16, retr = c.hm->is_retr[g];
    const char *src = (is_k ? c.k : c.v) + (static_cast<int64_t>(t0) * c.Hkv + g) * 256 + (lane & 15) * 16;
    char *base = retr ? (is_k ? c.rk : c.rv) : (is_k ? c.sk : c.sv);
    uint4 x[kAppendTokens];
#pragma unroll
    for (int i = 0; i < kAppendTokens; ++i)
      if (t0 + i < c.tokens) x[i] = __ldg(reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(i) * c.Hkv * 256));
    int s = find<&FinishSeq::tok0>(c, t0);
#pragma unroll
    for (int i = 0; i < kAppendTokens; ++i) {
      const int t = t0 + i;
      if (t >= c.tokens) break;
      while (t >= c.seq[s + 1].tok0) ++s;
      const FinishSeq &q = c.seq[s];
      const int pos = q.len + t - q.tok0, end = q.len + q.n;
      int64_t row;
      if (retr) {
        const int page = c.pages[q.page0 + pos / kPoolTile - q.len / kPoolTile];
        row = (static_cast<int64_t>(page) * c.Hr + idx) * kPoolTile + pos % kPoolTile;
      } else {
        if (pos >= c.S && pos < end - c.W) continue;  // evicted within the call
        row = (static_cast<int64_t>(q.slot) * c.Hs + idx) * (c.S + c.W) + (pos < c.S ? pos : c.S + pos % c.W);
      }
      *reinterpret_cast<uint4 *>(base + row * 256 + (lane & 15) * 16) = x[i];
    }
    return;
  }
  w -= append;
  if (w < static_cast<int64_t>(c.nseq) * c.Hr) {
    const int s = static_cast<int>(w / c.Hr), h = static_cast<int>(w % c.Hr);
    const FinishSeq &q = c.seq[s];
    const int end = q.len + q.n, last = end / kPoolTile * kPoolTile;  // first row of the page that holds `end`
    if (end != last && last >= q.len) {  // this layer opened it with this call
      const int page = c.pages[c.seq[s + 1].page0 - 1];
      const int64_t at = ((static_cast<int64_t>(page) * c.Hr + h) * kPoolTile + end - last) * 256;
      for (int i = lane; i < (last + kPoolTile - end) * 16; i += 32) {
        reinterpret_cast<uint4 *>(c.rk + at)[i] = make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint4 *>(c.rv + at)[i] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  const int64_t i = w * 32 + lane;
  if (i < c.npages) {
    const FinishSeq &q = c.seq[find<&FinishSeq::page0>(c, static_cast<int>(i))];
    c.table[static_cast<int64_t>(q.slot) * c.pages_per_seq + q.len / kPoolTile + i - q.page0] = c.pages[i];
  }
}

// Deals the items out: whole ones in rounds, item r * ctas + c to CTA c, as long as no CTA
// gets more than its even share of the cost, so that neighbours read the same keys at about
// the same time; then the rest, cut where a CTA's share is full.  Costs are in quarters of a
// retrieval head's key tile (3120 cycles with every SM at work): a streaming head's tile,
// masked for the most part, is five (3250 to 3780 cycles by the window), and a piece sixteen
// more than its tiles.  A whole piece between others measures 7400 cycles beside its tiles
// (queries, the first product, masks at its ends, the rows' way out), which would be ten; a
// cut one also leaves partial rows, which the last launch reads again.  A short call is
// launched on as many CTAs as it has tiles (calls of 20 to 100 us with their forks: 6 %
// shorter than with two tiles or more for each); shares grow in steps until everything is
// dealt, so some of them may stay without work (4 x 5 tokens: 128 of 148 have some).
struct Item {
  int tiles, tile_cost;
};
struct Deal {
  int whole = 0, ctas = 1;
  std::vector<PrefillShare> share;
  struct Cut {
    int item, pieces, part0, part1;
  };
  std::vector<Cut> cuts;
};
constexpr int kTileCost = 4, kStreamingTileCost = 5, kPieceCost = 16;
void deal_items(const std::vector<Item> &items, int sms, Deal *d) {
  const int n = static_cast<int>(items.size());
  auto cost = [&](int u) { return static_cast<int64_t>(items[u].tiles) * items[u].tile_cost + kPieceCost; };
  int64_t tiles = 0, total = 0;
  for (int u = 0; u < n; ++u) {
    tiles += items[u].tiles;
    total += cost(u);
  }
  d->ctas = static_cast<int>(std::min<int64_t>(std::min(sms, kPrefillCtas), tiles));
  const int ctas = d->ctas;
  std::vector<int64_t> load(ctas);
  for (int64_t even = (total + ctas - 1) / ctas;;) {
    std::fill(load.begin(), load.end(), 0);
    int u = 0;
    for (bool fits = true; fits && u + ctas <= n;) {
      for (int c = 0; c < ctas; ++c) fits &= load[c] + cost(u + c) <= even;
      if (!fits) break;
      for (int c = 0; c < ctas; ++c) load[c] += cost(u + c);
      u += ctas;
    }
    d->whole = u;
    d->share.assign(ctas, PrefillShare{0, 0, 0, 0});
    d->cuts.clear();
    int rank = 0;
    int t0 = 0;  // tiles of item u already dealt
    for (int c = 0; c < ctas && u < n; ++c) {
      int64_t room = even - load[c];
      PrefillShare &sh = d->share[c];
      sh = {u, t0, 0, 2 * rank};
      while (u < n) {
        const int rest = items[u].tiles - t0;
        const int64_t can = (room - kPieceCost) / items[u].tile_cost;
        if (can < 1) break;
        const int take = static_cast<int>(std::min<int64_t>(rest, can));
        if (t0 > 0) ++d->cuts.back().pieces;
        else if (take < rest) d->cuts.push_back({u, 1, sh.item == u ? sh.part : sh.part + 1, 2 * (rank + 1)});
        sh.tiles += take;
        room -= take * items[u].tile_cost + kPieceCost;
        t0 += take;
        if (t0 < items[u].tiles) break;
        ++u;
        t0 = 0;
      }
      if (sh.tiles > 0) ++rank;
    }
    if (u == n) return;
    int64_t rest = -static_cast<int64_t>(t0) * items[u].tile_cost;
    for (int i = u; i < n; ++i) rest += cost(i);
    even += std::max<int64_t>({1, rest / ctas, even / 128});
  }
}

// Does every CTA's every piece end before waits do?
bool pieces_fit(const std::vector<Item> &items, const Deal &d) {
  auto fits = [](const Item &i) { return i.tiles <= kPrefillMaxPiece; };
  if (std::all_of(items.begin(), items.end(), fits)) return true;
  if (!std::all_of(items.begin(), items.begin() + d.whole, fits)) return false;
  for (const PrefillShare &s : d.share) {
    int u = s.item, tile = s.tile;
    for (int left = s.tiles; left > 0; tile = 0, ++u) {
      const int nt = std::min(items[u].tiles - tile, left);
      if (nt > kPrefillMaxPiece) return false;
      left -= nt;
    }
  }
  return true;
}

duo_status prefill(duo_pool *P, int layer, int nseq, const int *seqs, const int *n, const void *q, const void *k,
                   const void *v, void *out, float *lse, cudaStream_t st) {
  std::vector<uint8_t> seen(P->max_seqs, 0);
  int64_t tokens = 0, fresh = 0, entries = 0;
  for (int i = 0; i < nseq; ++i) {
    const int s = seqs[i];
    if (!P->is_open(s) || seen[s] || n[i] < 1) return DUO_ERR_INVALID;
    seen[s] = 1;
    tokens += n[i];
  }
  if (tokens > kPrefillMaxTokens) return DUO_ERR_INVALID;
  {  // the results overlap neither the inputs, nor one another, nor the pool
    auto span = [](const void *p, int64_t bytes) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      return Span{at, at + static_cast<uintptr_t>(p ? bytes : 0)};
    };
    const int64_t qb = tokens * P->Hq * 256, kb = tokens * P->Hkv * 256;
    const Span o = span(out, qb), l = span(lse, tokens * P->Hq * 4);
    if (o.meets(l)) return DUO_ERR_INVALID;
    for (const Span &x : {span(q, qb), span(k, kb), span(v, kb), span(P->buf, static_cast<int64_t>(P->bytes))})
      if (x.meets(o) || x.meets(l)) return DUO_ERR_INVALID;
  }
  std::vector<int64_t> need(nseq), tiles(nseq);
  const int Hr = P->hr[layer], Hs = P->hs[layer];
  for (int i = 0; i < nseq; ++i) {
    const int64_t len = P->len[seqs[i]][layer], end = len + n[i];
    if (end > P->max_len) return DUO_ERR_CAPACITY;
    need[i] = (end + kPoolTile - 1) / kPoolTile;
    fresh += std::max<int64_t>(0, need[i] - static_cast<int64_t>(P->pages[seqs[i]].size()));
    entries += need[i] - len / kPoolTile;
    tiles[i] = (len + kPoolTile - 1) / kPoolTile + (n[i] + kPoolTile - 1) / kPoolTile;
  }
  if (fresh > static_cast<int64_t>(P->free_pages.size())) return DUO_ERR_CAPACITY;
  const duo_status r = pool_init(P, st);
  if (r != DUO_OK) return r;

  std::vector<int> order(nseq);
  for (int i = 0; i < nseq; ++i) order[i] = i;
  std::stable_sort(order.begin(), order.end(), [&](int a, int b) { return tiles[a] > tiles[b]; });

  PoolPrefillCall a{};
  PoolFinishCall f{};
  f.hm = &P->d_layers[layer].hm;
  const PoolLayerDesc &desc = P->h_layers[layer];
  f.rk = desc.rk;
  f.rv = desc.rv;
  f.sk = desc.sk;
  f.sv = desc.sv;
  a.tm_kr = desc.tm_kr;
  a.tm_vr = desc.tm_vr;
  a.tm_ks = desc.tm_ks;
  a.tm_vs = desc.tm_vs;
  a.table = f.table = P->d_table;
  a.pages_per_seq = f.pages_per_seq = P->pages_per_seq;
  a.v = f.v = static_cast<const char *>(v);
  f.k = static_cast<const char *>(k);
  a.out = f.out = static_cast<char *>(out);
  a.lse = f.lse = lse;
  a.partials = P->partials;
  f.partials = P->partials;
  a.status = P->status;
  a.nseq = f.nseq = nseq;
  a.Hq = f.Hq = P->Hq;
  a.Hkv = f.Hkv = P->Hkv;
  a.G = f.G = P->G;
  a.S = f.S = P->S;
  a.W = f.W = P->W;
  a.Hr = f.Hr = Hr;
  a.Hs = f.Hs = Hs;
  a.scale_log2 = P->scale * kLog2e;
  a.debug_stall = device_stall();
  f.tokens = static_cast<int>(tokens);
  a.npos = f.npos = prefill_tile_positions(P->G);
  f.npages = static_cast<int>(entries);
  int tok = 0, page = 0;
  for (int i = 0; i < nseq; ++i) {
    const int len = static_cast<int>(P->len[seqs[i]][layer]);
    f.seq[i] = {seqs[i], len, n[i], tok, page, {}};
    tok += n[i];
    page += static_cast<int>(need[i] - len / kPoolTile);
  }
  f.seq[nseq] = {0, 0, 0, tok, page, {}};
  std::vector<Item> items;
  for (int kind = 0; kind < 2; ++kind) {  // retrieval heads' items, then streaming heads'
    const int heads = kind == 0 ? Hr : Hs;
    int *first = kind == 0 ? a.lists.rfirst : a.lists.sfirst;
    for (int i = 0; i < nseq; ++i) {
      const int s = order[i], blocks = prefill_blocks(n[s], P->G);
      first[i + 1] = first[i] + blocks * heads;
      for (int b = blocks - 1; b >= 0 && heads > 0; --b) {
        PrefillRun runs[kPrefillMaxRuns];
        const int k = prefill_runs(kind == 0, f.seq[s].len, n[s], b * 2 * f.npos, f.npos, P->S, P->W, runs);
        int t = 0;
        for (int r = 0; r < k; ++r) t += runs[r].count;
        items.insert(items.end(), heads, Item{t, kind == 0 ? kTileCost : kStreamingTileCost});
      }
    }
  }
  for (int i = 0; i < nseq; ++i) {
    const int s = order[i];
    a.lists.slot[i] = f.seq[s].slot;
    a.lists.len[i] = f.seq[s].len;
    a.lists.n[i] = f.seq[s].n;
    a.lists.tok0[i] = f.seq[s].tok0;
    a.lists.blocks[i] = prefill_blocks(n[s], P->G);
  }
  const HeadMap &hm = desc.hm;
  std::copy(hm.retr_head, hm.retr_head + Hr, a.lists.retr_head);
  std::copy(hm.strm_head, hm.strm_head + Hs, a.lists.strm_head);
  a.retr_items = a.lists.rfirst[nseq];
  Deal deal;
  deal_items(items, P->num_sms, &deal);
  if (!pieces_fit(items, deal)) return DUO_ERR_UNSUPPORTED;
  a.whole_items = deal.whole;
  a.ctas = deal.ctas;
  std::copy(deal.share.begin(), deal.share.end(), a.lists.share);
  f.ncuts = static_cast<int>(deal.cuts.size());
  for (int i = 0; i < f.ncuts; ++i) {
    const Deal::Cut &cut = deal.cuts[i];
    const bool retr = cut.item < a.retr_items;
    const int u = retr ? cut.item : cut.item - a.retr_items, heads = retr ? Hr : Hs;
    const int *first = retr ? a.lists.rfirst : a.lists.sfirst;
    const int at = static_cast<int>(std::upper_bound(first, first + nseq, u) - first) - 1;
    const int rem = u - first[at];
    const FinishSeq &q = f.seq[order[at]];
    f.cuts[i] = {q.n, q.tok0, prefill_blocks(q.n, P->G) - 1 - rem / heads,
                 retr ? hm.retr_head[rem % heads] : hm.strm_head[rem % heads], cut.pieces, cut.part0, cut.part1,
                 f.join_blocks};
    for (int j = 0; j < join_threads(cut.pieces); ++j, f.join_blocks += kJoinGroups)
      f.cut_of[f.join_blocks / kJoinGroups] = static_cast<uint8_t>(i);
  }
  if (!dry_run() && prepare_prefill_pool_tc(&a, q, k, v, f.tokens) != cudaSuccess) return DUO_ERR_CUDA;
  for (int i = 0; i < nseq; ++i) duo_pool::make_room(P->pages[seqs[i]], static_cast<size_t>(need[i]));

  // from here on nothing throws; pages that the call opens go back if a launch fails
  std::vector<size_t> have(nseq);
  for (int i = 0; i < nseq; ++i) {
    std::vector<int> &pg = P->pages[seqs[i]];
    have[i] = pg.size();
    while (static_cast<int64_t>(pg.size()) < need[i]) pg.push_back(P->take_page());
    for (int e = f.seq[i].page0; e < f.seq[i + 1].page0; ++e)
      f.pages[e] = pg[f.seq[i].len / kPoolTile + e - f.seq[i].page0];
  }
  cudaError_t e = launch_via_hook([&] { return launch_prefill_pool_tc(a, st); });
  if (e == cudaSuccess)
    e = launch_via_hook([&] {
      const int64_t tail = std::max<int64_t>(static_cast<int64_t>(nseq) * Hr, (f.npages + 31) / 32);
      const int64_t warps = (tokens + kAppendTokens - 1) / kAppendTokens * P->Hkv + tail;
      return launch_overlapped(pool_prefill_finish_kernel, f.join_blocks + (warps + 7) / 8, 256, 0, st, f);
    });
  if (e != cudaSuccess) {  // the cache is written by the last launch alone
    for (int i = nseq - 1; i >= 0; --i) {
      std::vector<int> &pg = P->pages[seqs[i]];
      for (; pg.size() > have[i]; pg.pop_back()) P->drop_page(pg.back());
    }
    return DUO_ERR_CUDA;
  }
  for (int i = 0; i < nseq; ++i) P->len[seqs[i]][layer] += n[i];
  return DUO_OK;
}

}  // namespace

}  // namespace duo

using namespace duo;

extern "C" duo_status duo_pool_prefill(duo_pool *P, int layer, int nseq, const int *seqs, const int *n, const void *q,
                                       const void *k, const void *v, void *out, float *lse, void *stream) {
  DUO_NVTX_RANGE("duo_pool_prefill");
  if (!P || layer < 0 || layer >= P->layers || nseq < 1 || nseq > kPoolMaxSeqs || !seqs || !n || !q || !k || !v || !out)
    return DUO_ERR_INVALID;
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
        reinterpret_cast<uintptr_t>(out)) & 15u) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return DUO_ERR_INVALID;
  try {
    return prefill(P, layer, nseq, seqs, n, q, k, v, out, lse, static_cast<cudaStream_t>(stream));
  } catch (const std::exception &) {  // out of host memory, before anything was taken
    return DUO_ERR_INVALID;
  }
}

extern "C" duo_status duo_debug_prefill_runs(int retrieval, int len, int n, int r0, int npos, int S, int W,
                                             int (*runs)[3], int *nruns, int ring[4]) {
  if ((retrieval != 0 && retrieval != 1) || len < 0 || n < 1 || r0 < 0 || r0 >= n || npos < 1 || npos > 128 ||
      S < 0 || S > (1 << 24) || W < 1 || W > (1 << 24) || n > (1 << 30) || len > (1 << 30) || !runs || !nruns || !ring)
    return DUO_ERR_INVALID;
  PrefillRun r[kPrefillMaxRuns];
  *nruns = prefill_runs(retrieval == 1, len, n, r0, npos, S, W, r);
  for (int i = 0; i < *nruns; ++i) {
    runs[i][0] = r[i].src;
    runs[i][1] = r[i].first;
    runs[i][2] = r[i].count;
  }
  const PrefillRing v = prefill_ring(len + r0, len, S, W);
  ring[0] = v.lo1;
  ring[1] = v.hi1;
  ring[2] = v.lo2;
  ring[3] = v.hi2;
  return DUO_OK;
}

extern "C" duo_status duo_debug_prefill_deal(int nitems, const int *tiles, const int *tile_cost, int sms, int *whole,
                                             int *ctas, int (*shares)[4], int (*cuts)[4], int *ncuts) {
  if (nitems < 1 || !tiles || !tile_cost || sms < 1 || !whole || !ctas || !shares || !cuts || !ncuts)
    return DUO_ERR_INVALID;
  for (int i = 0; i < nitems; ++i)
    if (tiles[i] < 1 || tile_cost[i] < 1 || tiles[i] > (1 << 24) || tile_cost[i] > 64) return DUO_ERR_INVALID;
  try {
    std::vector<Item> items(nitems);
    for (int i = 0; i < nitems; ++i) items[i] = {tiles[i], tile_cost[i]};
    Deal deal;
    deal_items(items, sms, &deal);
    *whole = deal.whole;
    *ctas = deal.ctas;
    *ncuts = static_cast<int>(deal.cuts.size());
    for (int c = 0; c < deal.ctas; ++c) {
      const PrefillShare &s = deal.share[c];
      shares[c][0] = s.item;
      shares[c][1] = s.tile;
      shares[c][2] = s.tiles;
      shares[c][3] = s.part;
    }
    for (int i = 0; i < *ncuts; ++i) {
      const Deal::Cut &x = deal.cuts[i];
      cuts[i][0] = x.item;
      cuts[i][1] = x.pieces;
      cuts[i][2] = x.part0;
      cuts[i][3] = x.part1;
    }
  } catch (const std::exception &) {  // out of host memory
    return DUO_ERR_INVALID;
  }
  return DUO_OK;
}
