// pool_share.cu -- sequences that branch and move: duo_pool_fork and duo_pool_copy.
//
// A fork shares what can no longer be written.  Page p of a sequence is full on every
// layer once p < floor(shortest layer / 128), and appends write only at a layer's length,
// so those pages are listed by parent and child alike (a reference count each) and only
// the pages behind them -- one, when the layers are equally long -- are copied.  The sinks
// and rings of streaming heads are overwritten in place by appends, so each child gets
// its own.  A copy into another pool shares nothing.
//
// Both are one kernel: pieces (32 or 64 rows of one head of K or V) of the source's
// pages and rings, read once and written to every destination; rows past the source's
// length are written as zeros without being read.  A piece is one block of 256 threads
// with two or four 16-byte loads each in flight, so a fork of one child is a single wave of
// loads over the GPU, and many pieces stream at the copy bandwidth of HBM.  4 retrieval
// and 4 streaming heads, S + W = 528: one child of 333 tokens on 4 layers 3.3 us (its
// launch), eight of 4200 tokens on 8 layers 15.8 us (93 MB, 14 us at the copy bandwidth),
// a copy of 32900 tokens on 8 layers 167 us (6.6 TB/s, 100 % of it).  Figures in this file:
// mean of ten calls back to back in a captured graph, without the host.
#include "device_common.cuh"
#include "nvtx_range.h"
#include "pool_internal.h"

namespace duo {

namespace {

constexpr int kShareList = 704;  // page numbers in one launch's parameter block

struct PoolShareCall {
  const PoolLayerDesc *src_layers, *dst_layers;
  const int *src_table;  // the source's block-table row
  int *dst_table;        // the destination pool's block table
  int dst_pages_per_seq;
  int src_slot, ndst, heads2, Hkv, S, W;  // heads2: 2 * Hkv (K and V)
  int shared;            // table entries the destinations take over from the source
  int page0, npages;     // logical pages copied by this launch
  int64_t len;           // tokens of the source's longest layer
  int ring_rows;         // filled rows of a sink + ring, or -1: rings are not copied here
  int pieces;            // blocks per (layer, K or V, head)
  int dst_slot[kPoolMaxSeqs];
  int list[kShareList];  // npages source pages, then [npages][ndst] destination pages
};

// rows [0, valid) of a piece of `rows` rows, read once, into the same place of every
// destination; the others as zeros
template <int kShareRows, class Dst>
__device__ __forceinline__ void copy_piece(const char *src, int rows, int valid, int ndst, Dst dst) {
  constexpr int kShareLoads = kShareRows * 16 / 256;  // 16-byte vectors of a thread
  uint4 x[kShareLoads];
#pragma unroll
  for (int j = 0; j < kShareLoads; ++j) {
    const int i = threadIdx.x + 256 * j;  // 16 vectors a row
    x[j] = i < valid * 16 ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0, 0, 0, 0);
  }
  for (int c = 0; c < ndst; ++c) {
    uint4 *d = reinterpret_cast<uint4 *>(dst(c));
#pragma unroll
    for (int j = 0; j < kShareLoads; ++j) {
      const int i = threadIdx.x + 256 * j;
      if (i < rows * 16) d[i] = x[j];
    }
  }
}

template <int kShareRows>
__global__ void __launch_bounds__(256) pool_share_kernel(const __grid_constant__ PoolShareCall c) {
  constexpr int kSharePage = kPoolTile / kShareRows;  // pieces of a page
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned piece = blockIdx.x % c.pieces, h = blockIdx.x / c.pieces;
  const int g = h % c.Hkv, kv = (h / c.Hkv) & 1, layer = h / c.heads2;
  const PoolLayerDesc &A = c.src_layers[layer], &B = c.dst_layers[layer];
  const int idx = A.hm.kind_idx[g];
  if (A.hm.is_retr[g]) {
    const int page = piece / kSharePage, row0 = piece % kSharePage * kShareRows;
    if (page < c.npages) {
      const int64_t left = c.len - static_cast<int64_t>(c.page0 + page) * kPoolTile - row0;
      const int valid = static_cast<int>(left < 0 ? 0 : left < kShareRows ? left : kShareRows);
      const char *src =
          (kv ? A.rv : A.rk) + ((static_cast<int64_t>(c.list[page]) * A.Hr + idx) * kPoolTile + row0) * 256;
      char *base = kv ? B.rv : B.rk;
      const int *to = c.list + c.npages + page * c.ndst;
      copy_piece<kShareRows>(src, kShareRows, valid, c.ndst, [&](int d) {
        return base + ((static_cast<int64_t>(to[d]) * B.Hr + idx) * kPoolTile + row0) * 256;
      });
    }
  } else if (c.ring_rows >= 0) {
    const int slots = c.S + c.W, row0 = static_cast<int>(piece) * kShareRows;
    if (row0 < slots) {
      const int rows = min(kShareRows, slots - row0), valid = max(0, min(rows, c.ring_rows - row0));
      const char *src = (kv ? A.sv : A.sk) + ((static_cast<int64_t>(c.src_slot) * A.Hs + idx) * slots + row0) * 256;
      char *base = kv ? B.sv : B.sk;
      copy_piece<kShareRows>(src, rows, valid, c.ndst, [&](int d) {
        return base + ((static_cast<int64_t>(c.dst_slot[d]) * B.Hs + idx) * slots + row0) * 256;
      });
    }
  }
  // the destinations' block tables: entries taken over, then the copied pages
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t threads = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = tid; i < static_cast<int64_t>(c.shared) * c.ndst; i += threads)
    c.dst_table[static_cast<int64_t>(c.dst_slot[i / c.shared]) * c.dst_pages_per_seq + i % c.shared] =
        c.src_table[i % c.shared];
  for (int64_t i = tid; i < static_cast<int64_t>(c.npages) * c.ndst; i += threads)
    c.dst_table[static_cast<int64_t>(c.dst_slot[i % c.ndst]) * c.dst_pages_per_seq + c.page0 + i / c.ndst] =
        c.list[c.npages + i];
}

// Gives `n` free slots of Q the contents of sequence `seq` of P: the first `shared` pages
// by reference (P == Q), the others and the rings as copies.  Pages are taken before the first
// launch, as it lists them, and go back if one fails; slots are taken when all were accepted.
duo_status share_sequence(const duo_pool *P, int seq, duo_pool *Q, int shared, int n, cudaStream_t st, int *out) {
  const std::vector<int> &src = P->pages[seq];
  const std::vector<int64_t> &lens = P->len[seq];
  const int64_t longest = *std::max_element(lens.begin(), lens.end());
  const int copied = static_cast<int>(src.size()) - shared;
  std::vector<int> slots;
  for (int i = 0; i < Q->max_seqs && static_cast<int>(slots.size()) < n; ++i)
    if (!Q->open[i]) slots.push_back(i);
  if (static_cast<int>(slots.size()) < n || longest > Q->max_len ||
      static_cast<int64_t>(copied) * n > static_cast<int64_t>(Q->free_pages.size()))
    return DUO_ERR_CAPACITY;
  std::vector<std::vector<int>> lists(n);
  std::vector<std::vector<int64_t>> new_lens(n, lens);
  for (auto &l : lists) {
    l.reserve(src.size());
    l.assign(src.begin(), src.begin() + shared);
  }
  const duo_status r = pool_init(Q, st);  // the last step that can fail before the first launch
  if (r != DUO_OK) return r;
  for (auto &l : lists)
    for (int i = 0; i < copied; ++i) l.push_back(Q->take_page());

  PoolShareCall c{};
  c.src_layers = P->d_layers;
  c.dst_layers = Q->d_layers;
  c.src_table = P->d_table + static_cast<int64_t>(seq) * P->pages_per_seq;
  c.dst_table = Q->d_table;
  c.dst_pages_per_seq = Q->pages_per_seq;
  c.src_slot = seq;
  c.ndst = n;
  c.Hkv = P->Hkv;
  c.heads2 = 2 * P->Hkv;
  c.S = P->S;
  c.W = P->W;
  c.len = longest;
  for (int i = 0; i < n; ++i) c.dst_slot[i] = slots[i];
  const bool rings = std::any_of(P->hs.begin(), P->hs.end(), [](int h) { return h > 0; });
  const int per_launch = kShareList / (n + 1);
  cudaError_t e = cudaSuccess;
  int done = 0;
  do {  // the rings go with the first launch
    c.shared = done == 0 ? shared : 0;
    c.page0 = shared + done;
    c.npages = std::min(per_launch, copied - done);
    c.ring_rows = done > 0 || !rings ? -1
                  : static_cast<int>(longest <= P->S ? longest : P->S + std::min<int64_t>(longest, P->W));
    for (int i = 0; i < c.npages; ++i) {
      c.list[i] = src[c.page0 + i];
      for (int d = 0; d < n; ++d) c.list[c.npages + i * n + d] = lists[d][c.page0 + i];
    }
    auto blocks = [&](int rows) {
      const int ring = c.ring_rows >= 0 ? (P->S + P->W + rows - 1) / rows : 1;
      c.pieces = std::max({c.npages * (kPoolTile / rows), ring, 1});
      return static_cast<int64_t>(P->layers) * c.heads2 * c.pieces;
    };
    // 64 rows a piece stream best (32900 tokens of 8 layers 167 us, 200 with 32); where that
    // is less than twice what the GPU holds at once, pieces of 32 share the work more
    // evenly (eight children of 4200 tokens 15.8 us for 17.5, one of 333 tokens 3.5 for 3.9)
    constexpr int64_t kFew = 2 * 8 * 148;
    const bool few = blocks(64) < kFew;
    const int64_t grid = blocks(few ? 32 : 64);
    e = grid > INT32_MAX ? cudaErrorInvalidValue : launch_via_hook([&] {
      return launch_overlapped(few ? pool_share_kernel<32> : pool_share_kernel<64>, grid, 256, 0, st, c);
    });
    done += c.npages;
  } while (e == cudaSuccess && done < copied);
  if (e != cudaSuccess) {  // nothing that is open was written: the pages go back
    for (auto &l : lists)
      for (size_t i = shared; i < l.size(); ++i) Q->drop_page(l[i]);
    return DUO_ERR_CUDA;
  }
  for (int d = 0; d < n; ++d) {
    for (int i = 0; i < shared; ++i) ++Q->refs[lists[d][i]];
    Q->open[slots[d]] = 1;
    Q->pages[slots[d]].swap(lists[d]);
    Q->len[slots[d]].swap(new_lens[d]);
    out[d] = slots[d];
  }
  return DUO_OK;
}

}  // namespace

}  // namespace duo

using namespace duo;

extern "C" {

duo_status duo_pool_fork(duo_pool *P, int seq, int n, void *stream, int *children) {
  DUO_NVTX_RANGE("duo_pool_fork");
  if (!P || !P->is_open(seq) || n < 1 || n > kPoolMaxSeqs || !children) return DUO_ERR_INVALID;
  const std::vector<int64_t> &len = P->len[seq];
  const int64_t shortest = *std::min_element(len.begin(), len.end());
  try {
    return share_sequence(P, seq, P, static_cast<int>(shortest / kPoolTile), n, static_cast<cudaStream_t>(stream),
                          children);
  } catch (const std::exception &) {  // out of host memory, before anything was taken
    return DUO_ERR_INVALID;
  }
}

duo_status duo_pool_copy(const duo_pool *src, int seq, duo_pool *dst, void *stream, int *new_seq) {
  DUO_NVTX_RANGE("duo_pool_copy");
  if (!src || !dst || !src->is_open(seq) || !new_seq) return DUO_ERR_INVALID;
  if (src->layers != dst->layers || src->Hkv != dst->Hkv || src->S != dst->S || src->W != dst->W)
    return DUO_ERR_INVALID;
  for (int l = 0; l < src->layers; ++l)
    for (int g = 0; g < src->Hkv; ++g)
      if (src->h_layers[l].hm.is_retr[g] != dst->h_layers[l].hm.is_retr[g]) return DUO_ERR_INVALID;
  try {
    return share_sequence(src, seq, dst, 0, 1, static_cast<cudaStream_t>(stream), new_seq);
  } catch (const std::exception &) {
    return DUO_ERR_INVALID;
  }
}

}  // extern "C"
