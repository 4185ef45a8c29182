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
// needs no exchange, and 32 / lanes rows make one warp iteration of two 16-byte loads
// per lane.  A warp works on one token: its lanes evaluate each angle once (two per lane
// at rot 128) and share them through shared memory over all of the token's rows.
#include <cmath>
#include <new>

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
  int rows;                            // hq + hk + hv
  int warps_per_token, iters;          // warps sharing a token, warp iterations of each
  int rot, interleaved;
  float eps, scale;
  uint64_t freq[64];
  uint8_t axis[64];
};

constexpr int kNrThreads = 256;
constexpr int kNrUnroll = 2;  // row groups in flight per warp (loads issued before the first use)

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

template <typename T, int D>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int VE = 16 / static_cast<int>(sizeof(T));  // elements of a 16-byte vector
  constexpr int LR = D / (2 * VE);                      // lanes of a row (two vectors each)
  constexpr int RW = 32 / LR;                           // rows of a warp iteration
  constexpr int64_t kRow = D * static_cast<int64_t>(sizeof(T));
  __shared__ float2 table[kNrThreads / 32][D / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kNrThreads / 32) + warp;
  const int64_t t = w / p.warps_per_token;
  if (t >= p.n) return;
  const int slice = static_cast<int>(w - t * p.warps_per_token);

  // vectors of this lane: (a, b) hold the two halves of its pairs; behind the rotated
  // part, two plain vectors
  const int nv = p.rot / (2 * VE);  // lanes that rotate
  const int l = lane % LR;
  const bool rotates = l < nv;
  const int va = rotates ? l : nv + l, vb = rotates ? l + nv : LR + l;

  const int row0 = slice * p.iters * RW + lane / LR;
  auto source = [&](int r) -> const char * {
    if (r < p.hq) return p.q + t * p.qs + r * kRow;
    if (r < p.hq + p.hk) return p.k + t * p.ks + (r - p.hq) * kRow;
    return p.v + t * p.vs + (r - p.hq - p.hk) * kRow;
  };

  float cs[VE], sn[VE];
  bool first = true;
  for (int i0 = 0; i0 < p.iters; i0 += kNrUnroll) {
    uint4 xa[kNrUnroll], xb[kNrUnroll];
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) {
      const int r = row0 + (i0 + u) * RW;
      if (i0 + u < p.iters && r < p.rows) {
        const uint4 *src = reinterpret_cast<const uint4 *>(source(r));
        xa[u] = src[va];
        xb[u] = src[vb];
      } else {
        xa[u] = xb[u] = make_uint4(0, 0, 0, 0);
      }
    }
    if (first) {  // the token's angles, while the first rows are on their way
      first = false;
      for (int i = lane; i < p.rot / 2; i += 32) {
        const int64_t at = p.pos[p.axis[i] * p.n + t];
        const uint64_t turn = static_cast<uint64_t>(at) * p.freq[i];
        float s, c;
        sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &s, &c);
        table[warp][i] = make_float2(c * p.scale, s * p.scale);
      }
      __syncwarp();
      if (rotates) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          // split halves: pair l VE + e; interleaved: VE/2 pairs of vector a, then of b
          const int i = p.interleaved ? (e < VE / 2 ? va * (VE / 2) + e : vb * (VE / 2) + e - VE / 2) : l * VE + e;
          const float2 f = table[warp][i];
          cs[e] = f.x;
          sn[e] = f.y;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) {
      const int r = row0 + (i0 + u) * RW;
      float x[2 * VE];
      Elem<T>::unpack(xa[u], x);
      Elem<T>::unpack(xb[u], x + VE);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * VE; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = LR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (i0 + u >= p.iters || r >= p.rows) continue;
      const char *wt = r < p.hq ? p.wq : (r < p.hq + p.hk ? p.wk : nullptr);
      char *dst;
      if (r < p.hq) dst = p.qo + (t * p.hq + r) * kRow;
      else if (r < p.hq + p.hk) dst = p.ko + (t * p.hk + r - p.hq) * kRow;
      else dst = p.vo + (t * p.hv + r - p.hq - p.hk) * kRow;
      uint4 *d4 = reinterpret_cast<uint4 *>(dst);
      if (r >= p.hq + p.hk) {  // values as they are
        d4[va] = xa[u];
        d4[vb] = xb[u];
        continue;
      }
      if (wt) {
        const float inv = rsqrtf(ss * (1.f / D) + p.eps);
        float g[2 * VE];
        Elem<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(wt) + va), g);
        Elem<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(wt) + vb), g + VE);
#pragma unroll
        for (int e = 0; e < 2 * VE; ++e) x[e] = x[e] * inv * g[e];
      }
      if (rotates) {
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < VE; ++e) {  // pair e: elements 2e, 2e+1 (of a, then of b)
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = a * cs[e] - b * sn[e];
            x[2 * e + 1] = a * sn[e] + b * cs[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const float a = x[e], b = x[VE + e];
            x[e] = a * cs[e] - b * sn[e];
            x[VE + e] = a * sn[e] + b * cs[e];
          }
        }
      }
      d4[va] = pack16<T>(x);
      d4[vb] = pack16<T>(x + VE);
    }
  }
}

template <typename T, int D>
cudaError_t launch_norm_rope(NormRopeParams p, cudaStream_t st) {
  constexpr int RW = 32 / (D * static_cast<int>(sizeof(T)) / 32);
  const int groups = (p.rows + RW - 1) / RW;  // warp iterations of one token
  // Warps that share a token: one when the tokens alone fill the GPU (each angle is then
  // evaluated once), up to one per iteration when there are few tokens and only latency
  // counts.
  constexpr int64_t kWarps = 148 * 32;
  int64_t per = (p.n * groups + kWarps - 1) / kWarps;  // iterations per warp that give kWarps warps
  per = per < 1 ? 1 : (per > groups ? groups : per);
  p.iters = static_cast<int>(per);
  p.warps_per_token = (groups + p.iters - 1) / p.iters;
  const int64_t blocks = (p.n * p.warps_per_token + kNrThreads / 32 - 1) / (kNrThreads / 32);
  norm_rope_kernel<T, D><<<static_cast<unsigned>(blocks), kNrThreads, 0, st>>>(p);
  return cudaGetLastError();
}

// Byte ranges of the call's tensors, for the overlap check.
struct Span {
  uintptr_t lo, hi;
  bool meets(const Span &o) const { return lo < o.hi && o.lo < hi; }
};

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
    // 64 significant bits: |position| < 2^31 leaves the angle better than 2^-31 turns
    const long double turns = static_cast<long double>(inv_freq[i]) / 6.283185307179586476925286766559L;
    const long double f = turns - std::floor(turns);
    r->freq[i] = static_cast<uint64_t>(f * 0x1p64L);
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
  p.rows = p.hq + p.hk + p.hv;
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
