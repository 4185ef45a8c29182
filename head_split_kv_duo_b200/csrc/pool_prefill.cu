// pool_prefill.cu -- duo_pool_prefill: ragged pre-fill attention over the paged pool.  The
// attention is k_prefill_pool_tc.cu; here are the plan of a call, and its last launch,
// which joins split rows and appends the tokens.
//
// A row whose keys were split into segments with partial sums O_s, maxima m_s (base 2) and
// weights l_s is O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, M = max m_s, lse = (M +
// log2 of the denominator) ln 2; segments in order, so a result does not depend on timing.
#include <cmath>
#include <exception>

#include "device_common.cuh"
#include "nvtx_range.h"
#include "pool_internal.h"

namespace duo {

namespace {

// The call's last launch, sequences in the caller's order.
struct PoolFinishCall {
  const PoolLayerDesc *layer;
  int *table;
  int pages_per_seq;
  const char *k, *v;
  char *out;
  float *lse;
  const float *partials;
  int nseq, tokens, Hq, Hkv, G, S, W, Hr, npos, npages;
  int64_t join_rows;
  int slot[kPoolMaxSeqs], len[kPoolMaxSeqs], n[kPoolMaxSeqs];
  int tok0[kPoolMaxSeqs + 1];
  int page0[kPoolMaxSeqs + 1];  // a sequence's entries in `pages`, from logical page len / 128 on
  int segs[kPoolMaxSeqs], seg0[kPoolMaxSeqs];
  int join0[kPoolMaxSeqs + 1];  // rows to join before a sequence's
  int pages[kPrefillMaxPages];
};

// index of the last entry of first[0 .. n) that is <= x (first[0] <= x)
__device__ __forceinline__ int find(const int *first, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// One warp per split row: weights of its segments over the lanes, then four dimensions a
// lane, eight segments' loads in flight.
__device__ __forceinline__ void join_row(const PoolFinishCall &c, const PoolLayerDesc &L, int r, int lane) {
  const int s = find(c.join0, c.nseq, r);
  int rem = r - c.join0[s];
  const int gq = rem % c.G;
  rem /= c.G;
  const int h = rem % c.Hr, pos = rem / c.Hr;
  const int block = pos / (2 * c.npos), in = pos % (2 * c.npos), segs = c.segs[s];
  const int row = in / c.npos * 128 + in % c.npos * c.G + gq;
  const float *part = c.partials +
                      (static_cast<int64_t>(c.seg0[s] + (block * c.Hr + h) * segs) * kPrefillRows + row) * kPrefillRow;
  constexpr int64_t kSeg = static_cast<int64_t>(kPrefillRows) * kPrefillRow;
  constexpr int kPer = kPrefillSegs / 32;
  float w[kPer], m = -INFINITY, l = 0.f;
  float2 ml[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int seg = lane + 32 * i;
    ml[i] = seg < segs ? *reinterpret_cast<const float2 *>(part + seg * kSeg + 128) : make_float2(-INFINITY, 0.f);
    m = fmaxf(m, ml[i].x);
  }
  m = warp_max(m);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    // a segment that the row saw nothing of has no sum (its O was never written)
    w[i] = ml[i].x == -INFINITY ? 0.f : ex2(ml[i].x - m);
    l = fmaf(ml[i].y, w[i], l);
  }
  l = warp_sum(l);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    for (int b = 0; b < 32 && 32 * i + b < segs; b += 8) {
      float4 x[8];
      float ws[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int seg = 32 * i + b + e;
        ws[e] = __shfl_sync(0xffffffffu, w[i], b + e);
        x[e] = seg < segs && ws[e] != 0.f ? *reinterpret_cast<const float4 *>(part + seg * kSeg + 4 * lane)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o.x = fmaf(ws[e], x[e].x, o.x);
        o.y = fmaf(ws[e], x[e].y, o.y);
        o.z = fmaf(ws[e], x[e].z, o.z);
        o.w = fmaf(ws[e], x[e].w, o.w);
      }
    }
  }
  const float inv = 1.f / l;
  const int64_t at = static_cast<int64_t>(c.tok0[s] + pos) * c.Hq + L.hm.retr_head[h] * c.G + gq;
  const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), b = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  reinterpret_cast<uint2 *>(c.out + at * 256)[lane] =
      make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
  if (lane == 0 && c.lse) c.lse[at] = (m + lg2(l)) * kLn2;
}

// Warps: one per split row; then one per (token, KV head), K on the lower lanes, V on the
// upper; then one per (sequence, retrieval head) for the rest of a page that the call
// opened, and the block-table entries.
__global__ void __launch_bounds__(256) pool_prefill_finish_kernel(const __grid_constant__ PoolFinishCall c) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const PoolLayerDesc &L = *c.layer;
  if (w < c.join_rows) return join_row(c, L, static_cast<int>(w), lane);
  w -= c.join_rows;
  if (w < static_cast<int64_t>(c.tokens) * c.Hkv) {
    const int t = static_cast<int>(w / c.Hkv), g = static_cast<int>(w % c.Hkv), idx = L.hm.kind_idx[g];
    const int s = find(c.tok0, c.nseq, t), pos = c.len[s] + t - c.tok0[s], end = c.len[s] + c.n[s];
    const bool is_k = lane < 16;
    char *dst;
    if (L.hm.is_retr[g]) {
      const int page = c.pages[c.page0[s] + pos / kPoolTile - c.len[s] / kPoolTile];
      dst = (is_k ? L.rk : L.rv) + ((static_cast<int64_t>(page) * L.Hr + idx) * kPoolTile + pos % kPoolTile) * 256;
    } else {
      if (pos >= c.S && pos < end - c.W) return;  // evicted within the call
      const int slot = pos < c.S ? pos : c.S + pos % c.W;
      dst = (is_k ? L.sk : L.sv) + ((static_cast<int64_t>(c.slot[s]) * L.Hs + idx) * (c.S + c.W) + slot) * 256;
    }
    const char *src = (is_k ? c.k : c.v) + w * 256;
    reinterpret_cast<uint4 *>(dst)[lane & 15] = __ldg(reinterpret_cast<const uint4 *>(src) + (lane & 15));
    return;
  }
  w -= static_cast<int64_t>(c.tokens) * c.Hkv;
  if (w < static_cast<int64_t>(c.nseq) * L.Hr) {
    const int s = static_cast<int>(w / L.Hr), h = static_cast<int>(w % L.Hr);
    const int end = c.len[s] + c.n[s], last = end / kPoolTile * kPoolTile;  // first row of the page that holds `end`
    if (end != last && last >= c.len[s]) {  // this layer opened it with this call
      const int page = c.pages[c.page0[s + 1] - 1];
      const int64_t at = ((static_cast<int64_t>(page) * L.Hr + h) * kPoolTile + end - last) * 256;
      for (int i = lane; i < (last + kPoolTile - end) * 16; i += 32) {
        reinterpret_cast<uint4 *>(L.rk + at)[i] = make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint4 *>(L.rv + at)[i] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  const int64_t i = w * 32 + lane;
  if (i < c.npages) {
    const int s = find(c.page0, c.nseq, static_cast<int>(i));
    c.table[static_cast<int64_t>(c.slot[s]) * c.pages_per_seq + c.len[s] / kPoolTile + i - c.page0[s]] = c.pages[i];
  }
}

// Splits the keys of retrieval CTAs into segments: segs[s] per CTA of sequence s.  `tiles`
// and `ctas` are its key tiles and its CTAs, streaming CTAs run beside them.  With fewer
// CTAs than SMs, the shortest segments that still give every CTA an SM of its own; with
// more, only what is longer than an SM's even share.  A segment has at least four tiles
// (its start and its partial rows cost about two), and all segments of split rows fit
// the scratch.
void plan_segments(const std::vector<int64_t> &tiles, const std::vector<int64_t> &ctas, int64_t streaming_ctas,
                   int num_sms, std::vector<int> *segs) {
  const size_t n = tiles.size();
  int64_t retr_ctas = 0, work = 0;
  for (size_t s = 0; s < n; ++s) {
    retr_ctas += ctas[s];
    work += ctas[s] * tiles[s];
  }
  segs->assign(n, 1);
  if (retr_ctas == 0) return;
  const int64_t sms = std::max<int64_t>(num_sms - streaming_ctas, num_sms / 2);
  for (int64_t target = std::max<int64_t>(4, (work + sms - 1) / sms);; target += std::max<int64_t>(1, target / 16)) {
    int64_t all = 0, split = 0;
    for (size_t s = 0; s < n; ++s) {
      const int64_t k = (tiles[s] + target - 1) / target;
      (*segs)[s] = static_cast<int>(std::min<int64_t>(k, kPrefillSegs + 1));
      all += ctas[s] * k;
      split += k > 1 ? ctas[s] * k : 0;
    }
    if (split <= kPrefillSegs && (retr_ctas >= sms || all <= sms)) return;
  }
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
  std::vector<int64_t> need(nseq), tiles(nseq), ctas(nseq);
  const int Hr = P->hr[layer], Hs = P->hs[layer];
  int64_t streaming = 0;
  for (int i = 0; i < nseq; ++i) {
    const int64_t len = P->len[seqs[i]][layer], end = len + n[i];
    if (end > P->max_len) return DUO_ERR_CAPACITY;
    need[i] = (end + kPoolTile - 1) / kPoolTile;
    fresh += std::max<int64_t>(0, need[i] - static_cast<int64_t>(P->pages[seqs[i]].size()));
    entries += need[i] - len / kPoolTile;
    tiles[i] = (len + kPoolTile - 1) / kPoolTile + (n[i] + kPoolTile - 1) / kPoolTile;
    ctas[i] = static_cast<int64_t>(prefill_blocks(n[i], P->G)) * Hr;
    streaming += static_cast<int64_t>(prefill_blocks(n[i], P->G)) * Hs;
  }
  if (fresh > static_cast<int64_t>(P->free_pages.size())) return DUO_ERR_CAPACITY;
  const duo_status r = pool_init(P, st);
  if (r != DUO_OK) return r;

  std::vector<int> segs, order(nseq);
  plan_segments(tiles, ctas, streaming, P->num_sms, &segs);
  for (int i = 0; i < nseq; ++i) order[i] = i;
  std::stable_sort(order.begin(), order.end(), [&](int a, int b) { return tiles[a] * segs[b] > tiles[b] * segs[a]; });

  PoolPrefillCall a{};
  PoolFinishCall f{};
  a.layer = f.layer = P->d_layers + layer;
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
  a.Hs = Hs;
  a.scale_log2 = P->scale * kLog2e;
  f.tokens = static_cast<int>(tokens);
  f.npos = prefill_tile_positions(P->G);
  f.npages = static_cast<int>(entries);
  int tok = 0, page = 0, seg = 0, join = 0;
  for (int i = 0; i < nseq; ++i) {
    f.slot[i] = seqs[i];
    f.len[i] = static_cast<int>(P->len[seqs[i]][layer]);
    f.n[i] = n[i];
    f.tok0[i] = tok;
    f.page0[i] = page;
    f.segs[i] = segs[i];
    f.seg0[i] = seg;
    f.join0[i] = join;
    tok += n[i];
    page += static_cast<int>(need[i] - f.len[i] / kPoolTile);
    if (segs[i] > 1) {
      seg += static_cast<int>(ctas[i]) * segs[i];
      join += n[i] * Hr * P->G;
    }
  }
  f.tok0[nseq] = tok;
  f.page0[nseq] = page;
  f.join0[nseq] = join;
  f.join_rows = join;
  for (int i = 0; i < nseq; ++i) {
    const int s = order[i], blocks = prefill_blocks(n[s], P->G);
    a.slot[i] = f.slot[s];
    a.len[i] = f.len[s];
    a.n[i] = f.n[s];
    a.tok0[i] = f.tok0[s];
    a.segs[i] = f.segs[s];
    a.seg0[i] = f.seg0[s];
    a.rfirst[i + 1] = a.rfirst[i] + blocks * Hr * f.segs[s];
    a.sfirst[i + 1] = a.sfirst[i] + blocks * Hs;
  }
  a.retr_ctas = a.rfirst[nseq];
  a.ctas = a.retr_ctas + a.sfirst[nseq];
  if (!dry_run() && prepare_prefill_pool_tc(&a, q, k, v, f.tokens) != cudaSuccess) return DUO_ERR_CUDA;
  for (int i = 0; i < nseq; ++i) P->pages[seqs[i]].reserve(static_cast<size_t>(need[i]));

  // from here on nothing throws; pages that the call opens go back if a launch fails
  std::vector<size_t> have(nseq);
  for (int i = 0; i < nseq; ++i) {
    std::vector<int> &pg = P->pages[seqs[i]];
    have[i] = pg.size();
    while (static_cast<int64_t>(pg.size()) < need[i]) pg.push_back(P->take_page());
    for (int e = f.page0[i]; e < f.page0[i + 1]; ++e) f.pages[e] = pg[f.len[i] / kPoolTile + e - f.page0[i]];
  }
  cudaError_t e = launch_via_hook([&] { return launch_prefill_pool_tc(a, st); });
  if (e == cudaSuccess)
    e = launch_via_hook([&] {
      const int64_t tail = std::max<int64_t>(static_cast<int64_t>(nseq) * Hr, (f.npages + 31) / 32);
      const int64_t warps = f.join_rows + tokens * P->Hkv + tail;
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(static_cast<unsigned>((warps + 7) / 8));
      cfg.blockDim = dim3(256);
      cfg.stream = st;
      cudaLaunchAttribute at{};  // its start overlaps the attention's end; it waits for it
      at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at.val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = &at;
      cfg.numAttrs = 1;
      return cudaLaunchKernelEx(&cfg, pool_prefill_finish_kernel, f);
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
