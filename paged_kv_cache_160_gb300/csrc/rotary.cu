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
// CTA takes one token at a time, so that its rot / 2 angles are computed once for all heads: each thread
// holds the sines and cosines of its 8 elements in registers while it walks the heads.  CTAs stay for the
// next token, whose rows (kBatch of them per thread) and position are on their way while this one's are
// turned.  16,381 tokens x 40 heads of 128: 83.6 us with a row in flight per thread, 70.4 with four,
// 58.5 across tokens (5.7 TB/s, 0.85 of the measured copy).
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = 256;
constexpr int kBatch = 4;                // rows in flight per thread
constexpr int kCtasPerSm = 3;

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
  int num_tokens;
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
__global__ void __launch_bounds__(kThreads, kCtasPerSm) qk_rotary_kernel(const RotaryParams p) {
  __shared__ float2 turn[2][kMaxDim / 2];                   // [token parity] magnitude * (cos, sin) of each frequency
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kRowsAtOnce = kThreads / kLanes, kRowsPerBatch = kBatch * kRowsAtOnce;
  const int sub = threadIdx.x % kLanes, e0 = 8 * sub, row_in_step = threadIdx.x / kLanes;
  const bool live = e0 < p.head_dim;
  const int rows = p.num_heads + p.num_kv_heads, half = p.rotary_dim / 2;
  const bool rotated = live && e0 < p.rotary_dim;
  const int lane = threadIdx.x & 31;
  const int partner = kInterleaved || !rotated ? lane : (e0 < half ? lane + half / 8 : lane - half / 8);

  // Row r of token t in the inputs and outputs: byte r * head_dim * 2 behind the token's q (k: the row
  // before its first head would be there).
  const int row_bytes = 2 * p.head_dim;
  const int64_t k_back = int64_t(p.num_heads) * row_bytes;
  auto load_batch = [&](int64_t t, int s, uint4 (&batch)[kBatch]) {   // rows s .. of token t
    const uint8_t* q = p.q + 2 * (t * p.q_stride + e0);
    const uint8_t* k = p.k + 2 * (t * p.k_stride + e0) - k_back;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int r = s + row_in_step + b * kRowsAtOnce;
      batch[b] = live && r < rows ? *reinterpret_cast<const uint4*>((r < p.num_heads ? q : k) + int64_t(r) * row_bytes)
                                  : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  int64_t t = blockIdx.x;
  uint4 batch[kBatch];
  load_batch(t, 0, batch);
  int position = p.positions[t];
  const uint64_t freq = threadIdx.x < half ? p.table[threadIdx.x] : 0;
  auto angles = [&](int at, float2* tn) {
    if (threadIdx.x < half) {
      const uint64_t phase = uint64_t(int64_t(at)) * freq;
      float sine, cosine;
      sincospif(float(int32_t(phase >> 32)) * 4.656612873077393e-10f, &sine, &cosine);   // 2^-31: half turns
      tn[threadIdx.x] = make_float2(cosine * p.magnitude, sine * p.magnitude);
    }
  };
  angles(position, turn[0]);
  float cs[8], sn[8];

  // Every thread of a warp walks the same number of rows: the norm and the partner's elements come
  // by shuffles.
  auto rotate = [&](uint8_t* q_to, uint8_t* k_to, int r, const uint4 in) {
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
      *reinterpret_cast<uint4*>((isk ? k_to : q_to) + int64_t(r) * row_bytes) =
          make_uint4(pack2<kBF16>(y[0], y[1]), pack2<kBF16>(y[2], y[3]), pack2<kBF16>(y[4], y[5]),
                     pack2<kBF16>(y[6], y[7]));
    }
  };
  for (int n = 0, s = 0;;) {
    // The next batch: of this token, or the first of the CTA's next one.
    const bool token_ends = s + kRowsPerBatch >= rows;
    const int64_t t_next = token_ends ? t + gridDim.x : t;
    const int s_next = token_ends ? 0 : s + kRowsPerBatch;
    const bool more = t_next < p.num_tokens;
    uint4 next[kBatch];
    int position_next = position;
    if (more) {
      load_batch(t_next, s_next, next);
      if (token_ends) position_next = p.positions[t_next];
    }
    if (s == 0) {                                           // a token starts
      __syncthreads();                                      // its angles are there; the token before last is done with
      const float2* tn = turn[n & 1];
      // This thread's rotation: element e of the half layout belongs to frequency e mod half, of the
      // interleaved one to e / 2.
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        const float2 cssn = rotated ? tn[kInterleaved ? e >> 1 : (e < half ? e : e - half)] : make_float2(1.f, 0.f);
        const bool first = kInterleaved ? (i & 1) == 0 : e < half;
        cs[i] = cssn.x;
        sn[i] = first ? -cssn.y : cssn.y;
      }
    }
    if (position >= 0) {                                    // else a padding token
      uint8_t* q_to = p.q_out + 2 * (t * p.q_out_stride + e0);
      uint8_t* k_to = p.k_out + 2 * (t * p.k_out_stride + e0) - k_back;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (s + b * kRowsAtOnce >= rows) break;             // uniform over the CTA
        rotate(q_to, k_to, s + row_in_step + b * kRowsAtOnce, batch[b]);
      }
    }
    if (token_ends && more) angles(position_next, turn[(n + 1) & 1]);
    if (!more) break;
    n += token_ends;
    t = t_next;
    s = s_next;
    position = position_next;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) batch[b] = next[b];
  }
}

template <bool kBF16, bool kInterleaved>
cudaError_t launch(const RotaryParams& p, cudaStream_t s) {
  const int most = num_sms() > 0 ? num_sms() * kCtasPerSm : 1024;
  const dim3 grid(p.num_tokens < most ? p.num_tokens : most), block(kThreads);
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
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.rotary_dim = rotary_dim;
  p.magnitude = magnitude;
  p.eps = eps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool inter = layout == PKV_ROPE_INTERLEAVED;
  const cudaError_t e = dtype == PKV_BF16
                            ? (inter ? launch<true, true>(p, s) : launch<true, false>(p, s))
                            : (inter ? launch<false, true>(p, s) : launch<false, false>(p, s));
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // extern "C"
