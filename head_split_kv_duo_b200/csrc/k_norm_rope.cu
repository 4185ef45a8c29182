// k_norm_rope.cu -- per-head RMS norm and rotary positions of queries and keys in one
// pass, reading the projection's packed rows and writing the dense rows that the append,
// pre-fill and decode calls take (values ride along).
//
// For token t and a head row x of d elements, with weight w:
//     y = x * rsqrt(mean(x^2) + eps) * w                     (y = x without a weight)
// and for pair i < rot/2, (u, v) = (y_i, y_{i+rot/2}) or, interleaved, (y_2i, y_2i+1):
//     a = position[axis(i)][t] * inv_freq[i]
//     (u, v) <- scale * (u cos a - v sin a, u sin a + v cos a)
// elements from rot on stay y.  All of it in fp32, rounded once, at the store.
//
// The angle in turns is position * f with f = inv_freq / 2 pi, and only its fraction
// matters.  f enters as a 64-bit fixed-point fraction F = frac(f) 2^64, so that
// position * F mod 2^64 -- one wrapping integer product -- is the fraction of a turn to
// |position| 2^-64 whatever the position, where an fp32 product would be off by 0.06 rad
// a million tokens in.  Its top 32 bits, as a signed number of half turns, go to
// sincospif.
//
// Bound: HBM (every element read once and written once; a row is 256 bytes at bf16, d
// 128); for one token, the launch.  A row belongs to 16-byte x 2 lanes: the lane that
// holds elements of a pair's first half holds those of the second too, so the rotation
// needs no exchange, and 32 / lanes rows make one group, a warp iteration.  A warp works
// on one token: its lanes evaluate each angle once (two per lane at rot 128), share them
// through shared memory, and keep them in registers, multiplied by the weights, for all
// of the token's query rows and again for its keys: a pair costs two products, two fused
// multiply-adds and the scaling, on packed fp32 pairs.
// 32768 tokens of 32 + 8 + 8 heads, bf16: 141 us alone, 5.7 TB/s, 87 % of the copy rate (136
// back to back).  What it took: the factors in registers for 190 -> 156 us (before, each row
// unpacked its weights again and multiplied by them and by cos and sin in turn); blocks of
// two warps, ten of them and 160 rows in flight per SM at 96 registers (interleaved pairs:
// 103 and nine), -> 141 us (256 threads: 164; three or four groups per warp: 150 to 162;
// registers capped for more warps: 145 to 166).
#include <cmath>
#include <new>

#include "call_common.h"
#include "device_common.cuh"
#include "nvtx_range.h"

struct duo_rope {
  int head_dim = 0, rot = 0, axes = 0, interleaved = 0;
  float scale = 1.f;
  uint64_t freq[64] = {};  // frac(inv_freq / 2 pi) * 2^64
  uint8_t axis[64] = {};   // position axis of each pair
};

namespace duo {

namespace {

struct NormRopeParams {
  const char *q, *k, *v;               // token t's row of head h: base + t * stride + h * row bytes
  char *qo, *ko, *vo;                  // dense [n][heads][d]
  const char *wq, *wk;                 // [d], or null: that side is not normed
  const int *pos;                      // [axes][n]
  int64_t qs, ks, vs;                  // bytes between tokens
  int64_t n;
  int hq, hk, hv;                      // heads of each kind in this call (0: absent)
  int warps_per_token, iters;          // warps sharing a token, warp iterations of each
  int rot, interleaved;
  float eps, scale;
  uint64_t freq[64];
  uint8_t axis[64];
};

constexpr int kNrThreads = 64;
constexpr int kNrGroups = 2;  // row groups whose loads a warp has in flight

template <typename T>
__device__ __forceinline__ uint4 pack16(const float *f);
template <>
__device__ __forceinline__ uint4 pack16<float>(const float *f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float *f) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t *>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// kInter: pairs are neighbours.
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int VE = 16 / static_cast<int>(sizeof(T));  // elements of a 16-byte vector
  constexpr int LR = D / (2 * VE);                      // lanes of a row (two vectors each)
  constexpr int RW = 32 / LR;                           // rows of a group: one warp iteration
  constexpr int64_t kRow = D * static_cast<int64_t>(sizeof(T));
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float2 table[kNrThreads / 32][D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t w = blockIdx.x * (kNrThreads / 32) + warp;
  const uint32_t t = w / static_cast<uint32_t>(p.warps_per_token);
  if (t >= p.n) return;
  const int g0 = static_cast<int>(w - t * static_cast<uint32_t>(p.warps_per_token)) * p.iters, g1 = g0 + p.iters;

  // vectors of this lane: (a, b) hold the two halves of its pairs; behind the rotated
  // part, two plain vectors
  const int nv = p.rot / (2 * VE);  // lanes that rotate
  const int l = lane % LR, sub = lane / LR;
  const bool rotates = l < nv;
  const int va = rotates ? l : nv + l, vb = rotates ? l + nv : LR + l;

  bool first = true;
  int base = 0;  // groups of the sides before
#pragma unroll 1
  for (int side = 0; side < 3; ++side) {
    const int heads = side == 0 ? p.hq : (side == 1 ? p.hk : p.hv);
    const int lo = max(g0 - base, 0), hi = min(g1 - base, (heads + RW - 1) / RW);
    base += (heads + RW - 1) / RW;
    if (lo >= hi) continue;
    const char *src = (side == 0 ? p.q : (side == 1 ? p.k : p.v)) +
                      t * (side == 0 ? p.qs : (side == 1 ? p.ks : p.vs));
    char *dst = (side == 0 ? p.qo : (side == 1 ? p.ko : p.vo)) + static_cast<int64_t>(t) * heads * kRow;
    const char *weight = side == 0 ? p.wq : p.wk;
    // Per pair, weights folded into the rotation: u' = u ca - v sb, v' = u sa + v cb.  A
    // plain vector pair uses ca and cb alone.
    float ca[VE], cb[VE], sa[VE], sb[VE];
    bool ready = false;
#pragma unroll 1
    for (int i0 = lo; i0 < hi; i0 += kNrGroups) {
      uint4 xa[kNrGroups], xb[kNrGroups];
#pragma unroll
      for (int u = 0; u < kNrGroups; ++u) {
        const int r = (i0 + u) * RW + sub;
        xa[u] = xb[u] = make_uint4(0, 0, 0, 0);
        if (i0 + u < hi && r < heads) {
          const uint4 *at = reinterpret_cast<const uint4 *>(src + r * kRow);
          xa[u] = at[va];
          xb[u] = at[vb];
        }
      }
      if (side < 2 && !ready) {  // the side's factors, while its first rows are on their way
        ready = true;
        if (first) {
          first = false;
          for (int i = lane; i < p.rot / 2; i += 32) {
            const int64_t at = p.pos[p.axis[i] * p.n + t];
            const uint64_t turn = static_cast<uint64_t>(at) * p.freq[i];
            float s, c;
            sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &s, &c);
            table[warp][i] = make_float2(c * p.scale, s * p.scale);
          }
          __syncwarp();
        }
        float wa[VE], wb[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) wa[e] = wb[e] = 1.f;
        if (weight) {
          Elem<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(weight) + va), wa);
          Elem<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(weight) + vb), wb);
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          if (kInter) {
            // pair e of the lane: elements 2e, 2e+1 of a, then of b
            const int i = (e < VE / 2 ? va : vb) * (VE / 2) + e % (VE / 2);
            const float2 f = rotates ? table[warp][i] : make_float2(0.f, 0.f);
            const float *g = e < VE / 2 ? wa : wb;
            const float wu = g[2 * (e % (VE / 2))], wv = g[2 * (e % (VE / 2)) + 1];
            ca[e] = f.x * wu;
            cb[e] = f.x * wv;
            sa[e] = f.y * wu;
            sb[e] = -f.y * wv;
          } else {
            const float2 f = rotates ? table[warp][l * VE + e] : make_float2(1.f, 0.f);
            ca[e] = f.x * wa[e];
            cb[e] = f.x * wb[e];
            sa[e] = f.y * wa[e];
            sb[e] = -f.y * wb[e];
          }
        }
        if (kInter && !rotates) {
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            ca[e] = wa[e];
            cb[e] = wb[e];
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kNrGroups; ++u) {
        const int r = (i0 + u) * RW + sub;
        const bool live = i0 + u < hi && r < heads;
        uint4 *to = reinterpret_cast<uint4 *>(dst + r * kRow);
        if (side == 2) {  // values as they are
          if (live) {
            to[va] = xa[u];
            to[vb] = xb[u];
          }
          continue;
        }
        float a[VE], b[VE];
        Elem<T>::unpack(xa[u], a);
        Elem<T>::unpack(xb[u], b);
        if (weight) {
          uint64_t s2 = pack2(0.f, 0.f), s3 = s2;
#pragma unroll
          for (int e = 0; e < VE; e += 2) {
            s2 = ffma2(pack2(a[e], a[e + 1]), pack2(a[e], a[e + 1]), s2);
            s3 = ffma2(pack2(b[e], b[e + 1]), pack2(b[e], b[e + 1]), s3);
          }
          float x, y;
          unpack2(fadd2(s2, s3), x, y);
          float ss = x + y;
#pragma unroll
          for (int o = LR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float inv = rsqrtf(ss * (1.f / D) + p.eps);
          const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
          for (int e = 0; e < VE; e += 2) {
            unpack2(fmul2(pack2(a[e], a[e + 1]), inv2), a[e], a[e + 1]);
            unpack2(fmul2(pack2(b[e], b[e + 1]), inv2), b[e], b[e + 1]);
          }
        }
        if (!rotates) {  // a product with a zero sine would turn infinities into NaN
          if (weight) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
              a[e] *= ca[e];
              b[e] *= cb[e];
            }
          }
        } else if (kInter) {
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            float *x = e < VE / 2 ? a + 2 * e : b + 2 * e - VE;
            const float u0 = x[0], v0 = x[1];
            x[0] = fmaf(u0, ca[e], v0 * sb[e]);
            x[1] = fmaf(v0, cb[e], u0 * sa[e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < VE; e += 2) {
            const uint64_t u2 = pack2(a[e], a[e + 1]), v2 = pack2(b[e], b[e + 1]);
            unpack2(ffma2(u2, pack2(ca[e], ca[e + 1]), fmul2(v2, pack2(sb[e], sb[e + 1]))), a[e], a[e + 1]);
            unpack2(ffma2(v2, pack2(cb[e], cb[e + 1]), fmul2(u2, pack2(sa[e], sa[e + 1]))), b[e], b[e + 1]);
          }
        }
        if (live) {
          to[va] = pack16<T>(a);
          to[vb] = pack16<T>(b);
        }
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_norm_rope(NormRopeParams p, cudaStream_t st) {
  constexpr int RW = 32 / (D * static_cast<int>(sizeof(T)) / 32);
  // warp iterations of one token
  const int groups = (p.hq + RW - 1) / RW + (p.hk + RW - 1) / RW + (p.hv + RW - 1) / RW;
  // Warps that share a token: one when the tokens alone fill the GPU (each angle is then
  // evaluated once), up to one per iteration when there are few tokens and only latency
  // counts.
  constexpr int64_t kWarps = 148 * 32;
  int64_t per = (p.n * groups + kWarps - 1) / kWarps;  // iterations per warp that give kWarps warps
  per = per < 1 ? 1 : (per > groups ? groups : per);
  p.iters = static_cast<int>(per);
  p.warps_per_token = (groups + p.iters - 1) / p.iters;
  const int64_t blocks = (p.n * p.warps_per_token + kNrThreads / 32 - 1) / (kNrThreads / 32);
  const auto kernel = p.interleaved ? norm_rope_kernel<T, D, true> : norm_rope_kernel<T, D, false>;
  return launch_overlapped(kernel, blocks, kNrThreads, 0, st, p);
}

// The fraction of f / 2 pi, 0 <= f <= 2^20, in units of 2^-64, to the nearest: off by at most
// 2^-65 turns, and by 2^-34 turns times any position.  f = m 2^e exactly with a 53-bit m, so
// it is the product of m and the first 128 bits of 1 / 2 pi (at most 2^-108 turns off), an
// integer of three words, shifted; whole turns fall off at the top.  (A quotient in
// floating point loses as many bits of the fraction as there are whole turns per position:
// with 64 bits and f near 10^6, 2^-47 turns, and 1.3e-4 rad at position 2^31.)
uint64_t turn_fraction(double f) {
  constexpr uint64_t kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;  // floor(2^128 / 2 pi)
  int e;
  const uint64_t m = static_cast<uint64_t>(std::ldexp(std::frexp(f, &e), 53));
  const int s = 64 - (e - 53);  // f / 2 pi in units of 2^-64: m (2^128 / 2 pi) 2^-s; e <= 20, so s >= 97
  using u128 = unsigned __int128;
  const u128 lo = static_cast<u128>(m) * kLo, hi = static_cast<u128>(m) * kHi + static_cast<uint64_t>(lo >> 64);
  const uint64_t w[4] = {static_cast<uint64_t>(lo), static_cast<uint64_t>(hi), static_cast<uint64_t>(hi >> 64), 0};
  const int at = (s - 1) / 64, bit = (s - 1) % 64;  // the highest bit that falls off rounds
  if (at > 2) return 0;
  const u128 x = (static_cast<u128>(w[at + 1]) << 64 | w[at]) >> bit;  // that bit and, behind it, 64 or more
  return static_cast<uint64_t>((x >> 1) + (x & 1));
}

}  // namespace

}  // namespace duo

using namespace duo;

extern "C" {

duo_status duo_rope_create(int head_dim, int rot_dim, const double *inv_freq, const uint8_t *pair_axis, int axes,
                           int interleaved, float scale, duo_rope **out) {
  DUO_NVTX_RANGE("duo_rope_create");
  if (!out) return DUO_ERR_INVALID;
  *out = nullptr;
  if ((head_dim != 64 && head_dim != 128) || rot_dim < 16 || rot_dim > head_dim || rot_dim % 16 || !inv_freq ||
      axes < 1 || axes > 8 || (interleaved != 0 && interleaved != 1) || !(scale > 0.f) || !std::isfinite(scale))
    return DUO_ERR_INVALID;
  for (int i = 0; i < rot_dim / 2; ++i)
    if (!(inv_freq[i] >= 0.) || inv_freq[i] > 1e6 || (pair_axis && pair_axis[i] >= axes)) return DUO_ERR_INVALID;
  duo_rope *r = new (std::nothrow) duo_rope();
  if (!r) return DUO_ERR_INVALID;
  r->head_dim = head_dim;
  r->rot = rot_dim;
  r->axes = axes;
  r->interleaved = interleaved;
  r->scale = scale;
  for (int i = 0; i < rot_dim / 2; ++i) {
    r->freq[i] = turn_fraction(inv_freq[i]);
    r->axis[i] = pair_axis ? pair_axis[i] : 0;
  }
  *out = r;
  return DUO_OK;
}

void duo_rope_destroy(duo_rope *rope) { delete rope; }

duo_status duo_qk_norm_rope(const duo_rope *rope, int n, int q_heads, int kv_heads, duo_dtype dtype, const void *q,
                            int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                            const void *q_weight, const void *k_weight, float eps, const int32_t *positions,
                            void *q_out, void *k_out, void *v_out, void *stream) {
  DUO_NVTX_RANGE("duo_qk_norm_rope");
  if (!rope || n < 1 || (!q && !k) || !positions || (dtype != DUO_BF16 && dtype != DUO_FP32)) return DUO_ERR_INVALID;
  if ((q != nullptr) != (q_out != nullptr) || (k != nullptr) != (k_out != nullptr) ||
      (v != nullptr) != (v_out != nullptr))
    return DUO_ERR_INVALID;
  if ((q && (q_heads < 1 || q_heads > 4096)) || ((k || v) && (kv_heads < 1 || kv_heads > 4096))) return DUO_ERR_INVALID;
  if ((!q && q_weight) || (!k && k_weight)) return DUO_ERR_INVALID;
  if ((q_weight || k_weight) && (!(eps > 0.f) || !std::isfinite(eps))) return DUO_ERR_INVALID;
  const int64_t es = dtype == DUO_BF16 ? 2 : 4, row = rope->head_dim * es;
  const void *ins[3] = {q, k, v}, *outs[3] = {q_out, k_out, v_out}, *small[2] = {q_weight, k_weight};
  const int64_t strides[3] = {q_stride, k_stride, v_stride}, heads[3] = {q_heads, kv_heads, kv_heads};
  Span in[3], res[3];
  for (int i = 0; i < 3; ++i) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(ins[i]), b = reinterpret_cast<uintptr_t>(outs[i]);
    in[i] = res[i] = {0, 0};
    if (!ins[i]) continue;
    if ((a | b) & 15u) return DUO_ERR_INVALID;
    if (strides[i] < heads[i] * rope->head_dim || strides[i] > (int64_t(1) << 40) || strides[i] * es % 16)
      return DUO_ERR_INVALID;
    in[i] = {a, a + static_cast<uintptr_t>((n - 1) * strides[i] * es + heads[i] * row)};
    res[i] = {b, b + static_cast<uintptr_t>(n * heads[i] * row)};
  }
  if (((reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight)) & 15u) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u))
    return DUO_ERR_INVALID;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(positions);
  const Span pos = {pa, pa + static_cast<uintptr_t>(n) * rope->axes * 4};
  for (int i = 0; i < 3; ++i) {  // an output overlaps nothing but its own dense input, exactly
    if (!ins[i]) continue;
    for (int j = 0; j < 3; ++j) {
      const bool in_place = i == j && outs[i] == ins[i] && strides[i] == heads[i] * rope->head_dim;
      if (ins[j] && !in_place && res[i].meets(in[j])) return DUO_ERR_INVALID;
      if (j != i && ins[j] && res[i].meets(res[j])) return DUO_ERR_INVALID;
    }
    for (const void *s : small) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(s);
      if (s && res[i].meets({a, a + static_cast<uintptr_t>(row)})) return DUO_ERR_INVALID;
    }
    if (res[i].meets(pos)) return DUO_ERR_INVALID;
  }

  NormRopeParams p{};
  p.q = static_cast<const char *>(q);
  p.k = static_cast<const char *>(k);
  p.v = static_cast<const char *>(v);
  p.qo = static_cast<char *>(q_out);
  p.ko = static_cast<char *>(k_out);
  p.vo = static_cast<char *>(v_out);
  p.wq = static_cast<const char *>(q_weight);
  p.wk = static_cast<const char *>(k_weight);
  p.pos = positions;
  p.qs = q_stride * es;
  p.ks = k_stride * es;
  p.vs = v_stride * es;
  p.n = n;
  p.hq = q ? q_heads : 0;
  p.hk = k ? kv_heads : 0;
  p.hv = v ? kv_heads : 0;
  p.rot = rope->rot;
  p.interleaved = rope->interleaved;
  p.eps = eps;
  p.scale = rope->scale;
  for (int i = 0; i < rope->rot / 2; ++i) {
    p.freq[i] = rope->freq[i];
    p.axis[i] = rope->axis[i];
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_via_hook([&] {
    if (dtype == DUO_BF16)
      return rope->head_dim == 128 ? launch_norm_rope<__nv_bfloat16, 128>(p, st)
                                   : launch_norm_rope<__nv_bfloat16, 64>(p, st);
    return rope->head_dim == 128 ? launch_norm_rope<float, 128>(p, st) : launch_norm_rope<float, 64>(p, st);
  });
  return e == cudaSuccess ? DUO_OK : DUO_ERR_CUDA;
}

}  // extern "C"
