// qk_rotary: per-head RMS norm (optional) and rotation by position of a step's queries and keys, in
// one pass between the projection and kv_write / attention.
//
// Mathematics: y = x * rsqrt(mean x^2 + eps) * w; the pair (a, b) of frequency i turns by the angle
// t = position * f_i into (a cos t - b sin t, b cos t + a sin t).  The angle is kept in turns as a
// 64-bit fraction: position * (f_i / 2 pi in units of 2^-64) modulo 2^64 is exact modulo one turn,
// where a 32-bit product would lose the angle of far positions (half an ulp of 2^20 radians is
// 0.06).  The top 32 bits, as a signed part of half a turn, go to sincospi.
//
// Bound by HBM: 2 * (Hq + Hkv) * D * 2 bytes per token are moved, a few operations per element.  A
// CTA takes one token, so that its rot / 2 angles are computed once for all heads: each thread holds
// the sines and cosines of its 8 elements in registers while it walks the heads.  Its rows are on their
// way, kBatch at a time, while it waits for the position and computes the angles.
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = 256;
constexpr int kBatch = 4;                // rows in flight per thread

struct RotaryParams {
  uint8_t* q_out;
  const uint8_t* q;
  uint8_t* k_out;
  const uint8_t* k;
  int64_t q_out_stride, q_stride, k_out_stride, k_stride;   // elements
  const int32_t* positions;
  const uint64_t* table;
  const void* q_weight;
  const void* k_weight;
  int num_heads;
  int num_kv_heads;
  int head_dim;
  int rotary_dim;
  float magnitude;
  float eps;
};

template <bool kBF16>
__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<kBF16>(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

// kLanes threads share a row, 8 consecutive elements each (lanes past head_dim / 8 idle).
template <bool kBF16, bool kInterleaved, int kLanes>
__global__ void __launch_bounds__(kThreads) qk_rotary_kernel(const RotaryParams p) {
  __shared__ float2 turn[kMaxDim / 2];                      // magnitude * (cos, sin) of each frequency
  griddep_launch_dependents();
  griddep_wait();
  const int64_t t = blockIdx.x;
  constexpr int kRowsAtOnce = kThreads / kLanes;
  const int sub = threadIdx.x % kLanes, e0 = 8 * sub;
  const bool live = e0 < p.head_dim;
  const int rows = p.num_heads + p.num_kv_heads, half = p.rotary_dim / 2;

  auto src = [&](int r) -> const uint4* {
    const bool isk = r >= p.num_heads;
    const int64_t off = isk ? t * p.k_stride + int64_t(r - p.num_heads) * p.head_dim
                            : t * p.q_stride + int64_t(r) * p.head_dim;
    return reinterpret_cast<const uint4*>((isk ? p.k : p.q) + 2 * (off + e0));
  };
  int r0 = threadIdx.x / kLanes;                            // the batch's first row
  uint4 batch[kBatch];
  auto load_batch = [&]() {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int r = r0 + b * kRowsAtOnce;
      batch[b] = live && r < rows ? *src(r) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  load_batch();
  const int position = p.positions[t];
  if (position < 0) return;                                 // padding token

  if (threadIdx.x < half) {
    const uint64_t phase = uint64_t(int64_t(position)) * p.table[threadIdx.x];
    float sn, cs;
    sincospif(float(int32_t(phase >> 32)) * 4.656612873077393e-10f, &sn, &cs);   // 2^-31: half turns
    turn[threadIdx.x] = make_float2(cs * p.magnitude, sn * p.magnitude);
  }
  __syncthreads();
  // This thread's rotation: element e of the half layout belongs to frequency e mod half, of the
  // interleaved one to e / 2.  Outside the rotated part: cos 1, sin 0.
  const bool rotated = live && e0 < p.rotary_dim;
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = e0 + i;
    float2 cssn = make_float2(1.f, 0.f);
    if (rotated) cssn = turn[kInterleaved ? e >> 1 : (e < half ? e : e - half)];
    const bool first = kInterleaved ? (i & 1) == 0 : e < half;
    cs[i] = cssn.x;
    sn[i] = first ? -cssn.y : cssn.y;
  }
  const int lane = threadIdx.x & 31;
  const int partner = kInterleaved || !rotated ? lane : (e0 < half ? lane + half / 8 : lane - half / 8);

  // Every thread of a warp walks the same number of rows: the norm and the partner's elements come
  // by shuffles.
  auto rotate = [&](int r, const uint4 in) {
    float x[8];
    unpack8<kBF16>(in, x);
    const bool isk = r >= p.num_heads;
    const void* wp = isk ? p.k_weight : p.q_weight;
    if (p.q_weight || p.k_weight) {                         // uniform: the shuffles need the whole warp
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (wp && live) {
        const float inv = rsqrtf(ss / float(p.head_dim) + p.eps);
        float w[8];
        unpack8<kBF16>(__ldg(reinterpret_cast<const uint4*>(wp) + sub), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
      }
    }
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = kInterleaved ? x[i ^ 1] : __shfl_sync(0xffffffffu, x[i], partner);
      y[i] = rotated ? x[i] * cs[i] + other * sn[i] : x[i];
    }
    if (live && r < rows) {
      const int64_t off = isk ? t * p.k_out_stride + int64_t(r - p.num_heads) * p.head_dim
                              : t * p.q_out_stride + int64_t(r) * p.head_dim;
      *reinterpret_cast<uint4*>((isk ? p.k_out : p.q_out) + 2 * (off + e0)) =
          make_uint4(pack2<kBF16>(y[0], y[1]), pack2<kBF16>(y[2], y[3]), pack2<kBF16>(y[4], y[5]),
                     pack2<kBF16>(y[6], y[7]));
    }
  };
  const int last = (rows - 1) / kRowsAtOnce * kRowsAtOnce;  // first row of the last step
  for (int s = 0; s <= last; s += kBatch * kRowsAtOnce, r0 += kBatch * kRowsAtOnce) {
    if (s > 0) load_batch();
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (s + b * kRowsAtOnce > last) break;                // uniform over the CTA
      rotate(r0 + b * kRowsAtOnce, batch[b]);
    }
  }
}

template <bool kBF16, bool kInterleaved>
cudaError_t launch(const RotaryParams& p, int num_tokens, cudaStream_t s) {
  const dim3 grid(num_tokens), block(kThreads);
  if (p.head_dim <= 64) return launch_pdl(qk_rotary_kernel<kBF16, kInterleaved, 8>, grid, block, 0, s, p);
  if (p.head_dim <= 128) return launch_pdl(qk_rotary_kernel<kBF16, kInterleaved, 16>, grid, block, 0, s, p);
  return launch_pdl(qk_rotary_kernel<kBF16, kInterleaved, 32>, grid, block, 0, s, p);
}

}  // namespace
}  // namespace pkv

extern "C" {

pkv_status pkv_rope_table(uint64_t* table, int rotary_dim, double base, pkv_rope_scaling scaling, double factor,
                          double original_context, double alpha, double beta) {
  if (!table || rotary_dim <= 0 || rotary_dim % 2 || !(base > 1.0) || !isfinite(base)) return PKV_ERR_INVALID_ARG;
  if (scaling != PKV_ROPE_NONE && scaling != PKV_ROPE_LINEAR && scaling != PKV_ROPE_NTK && scaling != PKV_ROPE_PARTS)
    return PKV_ERR_INVALID_ARG;
  if (scaling != PKV_ROPE_NONE && (!(factor >= 1.0) || !isfinite(factor))) return PKV_ERR_INVALID_ARG;
  if (scaling == PKV_ROPE_NTK && rotary_dim < 4) return PKV_ERR_INVALID_ARG;
  if (scaling == PKV_ROPE_PARTS && (!(original_context > 0.0) || !isfinite(original_context) || !(alpha < beta) ||
                                    !isfinite(alpha) || !isfinite(beta)))
    return PKV_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  if (scaling == PKV_ROPE_NTK) base *= pow(factor, double(rotary_dim) / double(rotary_dim - 2));
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rotary_dim);
    if (scaling == PKV_ROPE_LINEAR) f /= factor;
    if (scaling == PKV_ROPE_PARTS) {
      const double r = original_context * f / two_pi;
      const double w = fmin(fmax((r - alpha) / (beta - alpha), 0.0), 1.0);
      f = w * f + (1.0 - w) * f / factor;
    }
    // f / 2 pi < 0.16 turns: below 2^62 in units of 2^-64, no overflow.
    table[i] = uint64_t(llrint(ldexp(f / two_pi, 64)));
  }
  return PKV_OK;
}

pkv_status pkv_qk_rotary(void* q_out, const void* q, void* k_out, const void* k, pkv_dtype dtype, int num_tokens,
                         int num_heads, int num_kv_heads, int head_dim, int64_t q_out_stride, int64_t q_stride,
                         int64_t k_out_stride, int64_t k_stride, const int32_t* positions, const uint64_t* table,
                         int rotary_dim, pkv_rope_layout layout, float magnitude, const void* q_weight,
                         const void* k_weight, float eps, pkv_stream_t stream) {
  using namespace pkv;
  if (num_tokens < 0 || num_heads < 0 || num_kv_heads < 0 || head_dim <= 0 || rotary_dim <= 0 ||
      rotary_dim > head_dim)
    return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (layout != PKV_ROPE_HALF && layout != PKV_ROPE_INTERLEAVED) return PKV_ERR_INVALID_ARG;
  if (head_dim % 16 || rotary_dim % 16 || head_dim > kMaxDim) return PKV_ERR_UNSUPPORTED;
  if (num_heads > (1 << 20) || num_kv_heads > (1 << 20)) return PKV_ERR_UNSUPPORTED;
  if (num_tokens == 0 || num_heads + num_kv_heads == 0) return PKV_OK;
  auto bad_side = [&](const void* o, const void* i, int64_t os, int64_t is, int heads, const void* w) {
    if (heads == 0) return false;
    return !o || !i || !aligned16(o) || !aligned16(i) || os % 8 || is % 8 || os < int64_t(heads) * head_dim ||
           is < int64_t(heads) * head_dim || !aligned16(w);
  };
  if (bad_side(q_out, q, q_out_stride, q_stride, num_heads, q_weight) ||
      bad_side(k_out, k, k_out_stride, k_stride, num_kv_heads, k_weight))
    return PKV_ERR_INVALID_ARG;
  if (!positions || !table || (reinterpret_cast<uintptr_t>(positions) & 3u) ||
      (reinterpret_cast<uintptr_t>(table) & 7u))
    return PKV_ERR_INVALID_ARG;
  if ((q_weight || k_weight) && !(eps >= 0.f)) return PKV_ERR_INVALID_ARG;
  RotaryParams p;
  p.q_out = static_cast<uint8_t*>(q_out);
  p.q = static_cast<const uint8_t*>(q);
  p.k_out = static_cast<uint8_t*>(k_out);
  p.k = static_cast<const uint8_t*>(k);
  p.q_out_stride = q_out_stride;
  p.q_stride = q_stride;
  p.k_out_stride = k_out_stride;
  p.k_stride = k_stride;
  p.positions = positions;
  p.table = table;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.rotary_dim = rotary_dim;
  p.magnitude = magnitude;
  p.eps = eps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool inter = layout == PKV_ROPE_INTERLEAVED;
  const cudaError_t e = dtype == PKV_BF16
                            ? (inter ? launch<true, true>(p, num_tokens, s) : launch<true, false>(p, num_tokens, s))
                            : (inter ? launch<false, true>(p, num_tokens, s) : launch<false, false>(p, num_tokens, s));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // extern "C"
