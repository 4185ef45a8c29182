// pool_internal.h -- the paged pool's handle, shared by the calls on it (pool.cu,
// pool_share.cu, pool_prefill.cu).
#pragma once

#include <algorithm>
#include <exception>
#include <functional>
#include <vector>

#include "call_common.h"

struct duo_pool {
  int layers = 0, Hkv = 0, Hq = 0, G = 0, D = 0, S = 0, W = 0, max_seqs = 0, pages_per_seq = 0;
  int64_t num_pages = 0, max_len = 0;
  float scale = 0.f;
  char *buf = nullptr;
  size_t bytes = 0;
  bool initialised = false;
  int num_sms = 0;
  uint32_t *status = nullptr;
  uint32_t *counters = nullptr;  // one ticket per item of a call
  // (max CTAs + items) segments of G partial rows of a decode step, or the pieces of a
  // pre-fill (40 MB, the larger for most pools)
  float *partials = nullptr;
  int max_items = 0;
  duo::PoolLayerDesc *d_layers = nullptr;
  int *d_table = nullptr;
  std::vector<duo::PoolLayerDesc> h_layers;
  std::vector<int> hr, hs;
  std::vector<int> free_pages;                 // free physical pages, a heap with the lowest on top
  std::vector<int> refs;                       // sequences that list each physical page
  std::vector<uint8_t> open;                   // per slot
  std::vector<std::vector<int>> pages;         // per slot: physical page of each logical page
  std::vector<std::vector<int64_t>> len;       // per slot, per layer

  // Pages are handed out lowest first, so that the pages in use stay at the low end.
  int take_page() {
    std::pop_heap(free_pages.begin(), free_pages.end(), std::greater<int>());
    const int pg = free_pages.back();
    free_pages.pop_back();
    refs[pg] = 1;
    return pg;
  }
  // One sequence fewer lists the page; it is free when none does.
  void drop_page(int pg) {
    if (--refs[pg] > 0) return;
    free_pages.push_back(pg);  // within the capacity reserved at creation
    std::push_heap(free_pages.begin(), free_pages.end(), std::greater<int>());
  }
  // Room for `n` pages in a sequence's list (twice what it had at least, so that lists which
  // grow page by page are moved rarely).  May throw; take_page and push_back then do not.
  static void make_room(std::vector<int> &list, size_t n) {
    if (list.capacity() < n) list.reserve(std::max(n, 2 * list.capacity()));
  }
  bool is_open(int seq) const { return seq >= 0 && seq < max_seqs && open[seq]; }
};

namespace duo {

// First use of a pool: clears its buffer and describes its layers on the device.
duo_status pool_init(duo_pool *P, cudaStream_t st);

// ---- pre-fill attention over a pool ----
constexpr int kPrefillMaxTokens = 1 << 18;  // tokens of one call
// pages that a call's tokens can touch: theirs, and a partial one at either end of each
constexpr int kPrefillMaxPages = kPrefillMaxTokens / kPoolTile + 2 * kPoolMaxSeqs;
constexpr int kPrefillRows = 256;           // query rows of an item (two tensor-core tiles)
constexpr int kPrefillCtas = 148;           // CTAs of the attention launch, one per SM
constexpr int kPrefillParts = 2 * kPrefillCtas;  // pieces of cut items: a CTA's first and last
// floats of a partial row: 128 sums, max, sum of weights, 2 unused.  A piece is
// [2 tiles][33 groups of four][128 rows][4]: the rows' threads write and read side by side.
constexpr int kPrefillRow = 132;
constexpr int kPrefillMaxRuns = 5;
// Longest piece of a CTA, in key tiles.  A role may wait while others work through a piece (the
// lister for a free place: one piece; the second query tile's softmax, of pieces that have one
// query tile: the four listed), and waits give up after 2 s.  A tile takes 1.9 us (of one
// query tile 1.6 us): 0.25 s and 0.84 s, less than 2 s at half the clock.
constexpr int kPrefillMaxPiece = 1 << 17;

// Where an item's key tiles come from: the sequence's pages, its sinks and ring in slot
// order, the call's own rows.
enum PrefillSource { kPages, kSlots, kChunk };
// Consecutive key tiles (of 128) of one source.
struct PrefillRun {
  int src, first, count;
};

// Slot order: slot x < S holds position x; ring slot S + y holds the newest position
// p = y (mod W) below len, that is, with r = len mod W, len - r + y for y < r and
// len - r - W + y for y >= r, where it is at least S.  Query i sees it iff i - p < W.  So
// with a = i - len + r + 1 and e = S - len + r + W the visible ring slots of i are
//   y in [max(0, a - W, e - W), r)  and  y in [max(r, a, e), W).
struct PrefillRing {
  int lo1, hi1, lo2, hi2;  // slots (S + y)
};
__host__ __device__ inline int larger(int a, int b) { return a > b ? a : b; }
__host__ __device__ inline int smaller(int a, int b) { return a < b ? a : b; }
__host__ __device__ inline PrefillRing prefill_ring(int i, int len, int S, int W) {
  const int r = len % W, a = i - len + r + 1, e = S - len + r + W;
  return {S + larger(0, larger(a, e) - W), S + r, S + larger(r, larger(a, e)), S + W};
}
// Appends the tiles that meet rows [lo, hi) of a source, from tile `at` on.
__host__ __device__ inline void add_run(PrefillRun *runs, int &k, int &at, int src, int lo, int hi) {
  if (lo >= hi) return;
  const int a = larger(lo / kPoolTile, at), b = (hi + kPoolTile - 1) / kPoolTile;
  if (a < b) {
    runs[k++] = {src, a, b - a};
    at = b;
  }
}
// The key tiles of the item whose first query is position r0 of the sequence's n new
// ones, npos positions a query tile; returns how many runs.  Streaming heads skip tiles
// that hold no position visible to any of the queries; the first one reaches back
// furthest.
__host__ __device__ inline int prefill_runs(bool retr, int len, int n, int r0, int npos, int S, int W,
                                            PrefillRun *runs) {
  const int rows = smaller(r0 + 2 * npos, n);  // positions 0 .. rows-1 of the chunk are needed
  int k = 0, at = 0;
  if (retr) {
    add_run(runs, k, at, kPages, 0, len);
    at = 0;
    add_run(runs, k, at, kChunk, 0, rows);
    return k;
  }
  const PrefillRing v = prefill_ring(len + r0, len, S, W);
  add_run(runs, k, at, kSlots, 0, smaller(S, len));
  add_run(runs, k, at, kSlots, v.lo1, v.hi1);
  add_run(runs, k, at, kSlots, v.lo2, v.hi2);
  at = 0;
  add_run(runs, k, at, kChunk, 0, smaller(rows, S - len));
  add_run(runs, k, at, kChunk, larger(0, r0 - W + 1), rows);
  return k;
}

// A CTA's part of the items that are cut: `tiles` key tiles from tile `tile` of item
// `item` on.  Partial rows of its first item go to place `part`, of its last to part + 1.
struct PrefillShare {
  int item, tile, tiles, part;
};

// The attention launch.  Sequences are listed by decreasing work per item; retrieval heads'
// items come first.  CTA c works on items c, c + grid, ... below whole_items, then on its
// share of the others.
struct alignas(16) PrefillLists {
  int slot[kPoolMaxSeqs], len[kPoolMaxSeqs], n[kPoolMaxSeqs];
  int tok0[kPoolMaxSeqs];        // first of the sequence's tokens in the call's tensors
  int blocks[kPoolMaxSeqs];      // items per KV head
  int rfirst[kPoolMaxSeqs + 1], sfirst[kPoolMaxSeqs + 1];  // items before a sequence, per kind
  int unused[2];
  uint8_t retr_head[kMaxKvHeads], strm_head[kMaxKvHeads];  // KV heads of each kind
  PrefillShare share[kPrefillCtas];
};
struct PoolPrefillCall {
  CUtensorMap tm_q, tm_k, tm_v;  // q [tokens][Hq][d], k and v [tokens][Hkv][d]
  CUtensorMap tm_kr, tm_vr, tm_ks, tm_vs;  // the layer's pages, sinks and rings
  const int *table;              // device block table [max_seqs][pages_per_seq]
  int pages_per_seq;
  const char *v;
  char *out;
  float *lse, *partials;
  uint32_t *status;
  int nseq, Hq, Hkv, G, npos, S, W, Hr, Hs, retr_items, whole_items, ctas;  // npos: positions of a query tile
  float scale_log2;
  int debug_stall;  // test control: the softmax first waits for a barrier that nothing arrives at
  PrefillLists lists;
};
// Positions per query tile and items (of two tiles) that cover n positions of one KV head.
inline int prefill_tile_positions(int G) { return 128 / G; }
inline int prefill_blocks(int n, int G) {
  const int per = 2 * prefill_tile_positions(G);
  return (n + per - 1) / per;
}
cudaError_t prepare_prefill_pool_tc(PoolPrefillCall *c, const void *q, const void *k, const void *v, int tokens);
cudaError_t launch_prefill_pool_tc(const PoolPrefillCall &c, cudaStream_t st);

}  // namespace duo
