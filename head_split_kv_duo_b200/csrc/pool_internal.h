// pool_internal.h -- the paged pool's handle, shared by the calls on it (pool.cu,
// pool_share.cu, pool_prefill.cu).
#pragma once

#include <algorithm>
#include <functional>
#include <vector>

#include "duo_internal.h"

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
  float *partials = nullptr;     // (max CTAs + items) segments of G partial rows
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
  bool is_open(int seq) const { return seq >= 0 && seq < max_seqs && open[seq]; }
};

namespace duo {

// First use of a pool: clears its buffer and describes its layers on the device.
duo_status pool_init(duo_pool *P, cudaStream_t st);

// ---- pre-fill attention over a pool ----
constexpr int kPrefillMaxTokens = 1 << 18;  // tokens of one call
// pages that a call's tokens can touch: theirs, and a partial one at either end of each
constexpr int kPrefillMaxPages = kPrefillMaxTokens / kPoolTile + 2 * kPoolMaxSeqs;
constexpr int kPrefillRows = 256;           // query rows of a CTA (two tensor-core tiles)
constexpr int kPrefillSegs = 160;           // key segments whose partial rows fit the scratch
constexpr int kPrefillRow = 132;            // floats of a partial row: 128 sums, max, sum of weights, 2 unused

// The attention launch.  Sequences are listed by decreasing work per CTA; CTAs of
// retrieval heads come first.
struct PoolPrefillCall {
  CUtensorMap tm_q, tm_k, tm_v;  // q [tokens][Hq][d], k and v [tokens][Hkv][d]
  const PoolLayerDesc *layer;    // device
  const int *table;              // device block table [max_seqs][pages_per_seq]
  int pages_per_seq;
  const char *v;
  char *out;
  float *lse, *partials;
  uint32_t *status;
  int nseq, Hq, Hkv, G, S, W, Hr, Hs, retr_ctas, ctas;
  float scale_log2;
  int slot[kPoolMaxSeqs], len[kPoolMaxSeqs], n[kPoolMaxSeqs];
  int tok0[kPoolMaxSeqs];        // first of the sequence's tokens in the call's tensors
  int segs[kPoolMaxSeqs];        // key segments of each of its retrieval CTAs' rows
  int seg0[kPoolMaxSeqs];        // its first partial segment (segs > 1)
  int rfirst[kPoolMaxSeqs + 1], sfirst[kPoolMaxSeqs + 1];  // CTAs before a sequence, per kind
};
// Positions per query tile and CTAs (of two tiles) that cover n positions of one KV head.
inline int prefill_tile_positions(int G) { return 128 / G; }
inline int prefill_blocks(int n, int G) {
  const int per = 2 * prefill_tile_positions(G);
  return (n + per - 1) / per;
}
cudaError_t prepare_prefill_pool_tc(PoolPrefillCall *c, const void *q, const void *k, const void *v, int tokens);
cudaError_t launch_prefill_pool_tc(const PoolPrefillCall &c, cudaStream_t st);

}  // namespace duo
