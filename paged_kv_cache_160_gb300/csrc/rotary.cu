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
// CTA takes tiles of a few tokens: it works their angles out once for all heads, into shared memory, and
// walks their rows (of q and k alike) with kBatch rows per thread in flight, the next tile's first ones
// while this one's last are turned.  A thread has both elements of its pairs, so that nothing but the
// norm's sum crosses threads.
//   16,381 tokens x 40 heads of 128, half of each turned: 52.8 us, 6.4 TB/s, 0.94 of the measured copy.  The same
// with the norm and all of it turned is as much bound by instructions: 4096 tokens take 18.8 us (0.66).  A CTA
// per token, which leaves most of its threads idle where a token has few heads, took 58.5, 31.8 and, for 16,381
// tokens x 3 heads, 74.6 us (10.3 now).
#include <math.h>

#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = 256;
constexpr int kBatch = 2;                // rows in flight per thread
constexpr int kCtasPerSm = 3;
constexpr int kMaxAngles = 2048;         // of a tile

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
  int head_dim;
  int rotary_dim;
  int tile;               // tokens
  Divisor rows;           // heads of q and k together
  Divisor half;           // rotary_dim / 2
  float magnitude;
  float eps;
};

template <bool kBF16>
__device__ __forceinline__ void unpack8(const uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<kBF16>(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
template <bool kBF16>
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack2<kBF16>(f[0], f[1]), pack2<kBF16>(f[2], f[3]), pack2<kBF16>(f[4], f[5]),
                    pack2<kBF16>(f[6], f[7]));
}

// kLanes threads share a row, two runs of 8 elements each (lanes past head_dim / 16 idle): in the half
// layout runs l and l + rotary_dim / 16, whose elements are paired, else l and l + head_dim / 16.
template <bool kBF16, bool kInterleaved, int kLanes, bool kNorm>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) qk_rotary_kernel(const RotaryParams p) {
  extern __shared__ __align__(16) float smem[];
  constexpr int kRowsAtOnce = kThreads / kLanes, kRowsPerStep = kBatch * kRowsAtOnce;
  const int half = int(p.half.d), rows = int(p.rows.d), num_angles = p.tile * half;
  // [tile parity][token][angle], scaled by the magnitude; the half layout keeps angles 8l .. 8l + 3 of all
  // lanes l before their angles 8l + 4 .. 8l + 7, so that a quarter warp reads neighbouring 16 bytes.
  float* cosines = smem;
  float* sines = smem + 2 * num_angles;
  int* place = reinterpret_cast<int*>(smem + 4 * num_angles);   // [tile parity][token] positions
  const int l = threadIdx.x % kLanes, row_in_step = threadIdx.x / kLanes;
  const bool live = 16 * l < p.head_dim;
  const int pairs = p.rotary_dim / 16;                      // lanes with paired runs (half layout)
  int run0 = l, run1 = l + p.head_dim / 16;
  if (!kInterleaved) {
    run0 = l < pairs ? l : 2 * l;
    run1 = l < pairs ? l + pairs : 2 * l + 1;
  }
  const bool turn0 = live && 8 * run0 < p.rotary_dim, turn1 = live && 8 * run1 < p.rotary_dim;

  griddep_launch_dependents();
  griddep_wait();
  const int tiles = (p.num_tokens - 1) / p.tile + 1;
  auto tokens_of = [&](int tile) -> int { return min(p.tile, p.num_tokens - tile * p.tile); };
  auto work_angles_out = [&](int tile, int parity) {        // from the positions in `place`
    const int n = tokens_of(tile) * half;
    float* c = cosines + parity * num_angles;
    float* s = sines + parity * num_angles;
    for (int a = threadIdx.x; a < n; a += kThreads) {
      const int tt = int(p.half.quotient(a)), i = a - tt * half;
      const uint64_t phase = uint64_t(int64_t(place[parity * p.tile + tt])) * __ldg(p.table + i);
      float sine, cosine;
      sincospif(float(int32_t(phase >> 32)) * 4.656612873077393e-10f, &sine, &cosine);   // 2^-31: half turns
      const int at = tt * half + (kInterleaved ? i : (i >> 2 & 1) * (half / 2) + (i >> 3) * 4 + (i & 3));
      c[at] = cosine * p.magnitude;
      s[at] = sine * p.magnitude;
    }
  };
  // Row f of a tile, counted over its tokens: the address of its first element.
  auto row_at = [&](const uint8_t* q, int64_t qs, const uint8_t* k, int64_t ks, int tile, int f, int& tt, bool& isk) -> int64_t {
    tt = int(p.rows.quotient(f));
    const int r = f - tt * rows;
    isk = r >= p.num_heads;
    const int64_t t = int64_t(tile) * p.tile + tt;
    return reinterpret_cast<int64_t>(isk ? k : q) +
           2 * (t * (isk ? ks : qs) + int64_t(isk ? r - p.num_heads : r) * p.head_dim);
  };
  auto load_batch = [&](int tile, int f0, uint4 (&batch)[kBatch][2]) {   // rows f0 ..
    const int n = tokens_of(tile) * rows;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int f = f0 + row_in_step + b * kRowsAtOnce;
      batch[b][0] = batch[b][1] = make_uint4(0u, 0u, 0u, 0u);
      if (live && f < n) {
        int tt;
        bool isk;
        const uint8_t* from = reinterpret_cast<const uint8_t*>(row_at(p.q, p.q_stride, p.k, p.k_stride, tile, f, tt, isk));
        batch[b][0] = __ldcs(reinterpret_cast<const uint4*>(from + 16 * run0));
        batch[b][1] = __ldcs(reinterpret_cast<const uint4*>(from + 16 * run1));
      }
    }
  };
  auto turn_row = [&](int tile, int parity, int f, const uint4 (&in)[2]) {
    float x[16];
    unpack8<kBF16>(in[0], x);
    unpack8<kBF16>(in[1], x + 8);
    const bool there = live && f < tokens_of(tile) * rows;
    int tt = 0;
    bool isk = false;
    const int64_t to = there ? row_at(p.q_out, p.q_out_stride, p.k_out, p.k_out_stride, tile, f, tt, isk) : 0;
    if constexpr (kNorm) {                                  // the shuffles need the whole warp
      uint64_t ss2 = 0;
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const uint64_t v = pack_f32x2(x[i], x[i + 1]);
        ss2 = fma_f32x2(v, v, ss2);
      }
      float ss = lo_f32(ss2) + hi_f32(ss2);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const uint4* wp = static_cast<const uint4*>(isk ? p.k_weight : p.q_weight);
      if (there && wp) {
        const float inv = rsqrtf(ss / float(p.head_dim) + p.eps);
        float w[16];
        unpack8<kBF16>(__ldg(wp + run0), w);
        unpack8<kBF16>(__ldg(wp + run1), w + 8);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const uint64_t v = mul_f32x2(mul_f32x2(pack_f32x2(x[i], x[i + 1]), pack_f32x2(inv, inv)), pack_f32x2(w[i], w[i + 1]));
          x[i] = lo_f32(v);
          x[i + 1] = hi_f32(v);
        }
      }
    }
    if (!there || place[parity * p.tile + tt] < 0) return;  // (negative: a padding token)
    const float* c = cosines + parity * num_angles + tt * half;
    const float* s = sines + parity * num_angles + tt * half;
    if constexpr (kInterleaved) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (!(u ? turn1 : turn0)) continue;
        const float4 cc = *reinterpret_cast<const float4*>(c + 4 * (u ? run1 : run0));
        const float4 sv = *reinterpret_cast<const float4*>(s + 4 * (u ? run1 : run0));
        const float cs[4] = {cc.x, cc.y, cc.z, cc.w}, sn[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[8 * u + 2 * i], b = x[8 * u + 2 * i + 1];
          x[8 * u + 2 * i] = a * cs[i] - b * sn[i];
          x[8 * u + 2 * i + 1] = b * cs[i] + a * sn[i];
        }
      }
    } else if (turn0) {                                     // both runs or neither
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 cc = *reinterpret_cast<const float4*>(c + u * (half / 2) + 4 * l);
        const float4 sv = *reinterpret_cast<const float4*>(s + u * (half / 2) + 4 * l);
        const float cs[4] = {cc.x, cc.y, cc.z, cc.w}, sn[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[4 * u + i], b = x[8 + 4 * u + i];
          x[4 * u + i] = a * cs[i] - b * sn[i];
          x[8 + 4 * u + i] = b * cs[i] + a * sn[i];
        }
      }
    }
    uint8_t* out = reinterpret_cast<uint8_t*>(to);
    *reinterpret_cast<uint4*>(out + 16 * run0) = pack8<kBF16>(x);
    *reinterpret_cast<uint4*>(out + 16 * run1) = pack8<kBF16>(x + 8);
  };

  int tile = blockIdx.x, parity = 0;
  uint4 batch[kBatch][2];
  load_batch(tile, 0, batch);
  if (int(threadIdx.x) < tokens_of(tile)) place[threadIdx.x] = p.positions[int64_t(tile) * p.tile + threadIdx.x];
  __syncthreads();
  work_angles_out(tile, 0);
  while (true) {
    __syncthreads();                                        // the tile's angles are there
    const int next = tile + gridDim.x, n = tokens_of(tile) * rows;
    const bool more = next < tiles;
    int position = 0;
    if (more && int(threadIdx.x) < tokens_of(next)) position = p.positions[int64_t(next) * p.tile + threadIdx.x];
    for (int f = 0; f < n; f += kRowsPerStep) {
      uint4 ahead[kBatch][2];
      if (f + kRowsPerStep < n) load_batch(tile, f + kRowsPerStep, ahead);
      else if (more) load_batch(next, 0, ahead);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) turn_row(tile, parity, f + row_in_step + b * kRowsAtOnce, batch[b]);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        batch[b][0] = ahead[b][0];
        batch[b][1] = ahead[b][1];
      }
    }
    if (!more) break;
    parity ^= 1;
    if (int(threadIdx.x) < tokens_of(next)) place[parity * p.tile + threadIdx.x] = position;
    __syncthreads();                                        // the positions are there
    work_angles_out(next, parity);
    tile = next;
  }
}

// Tokens of a tile: the fewest whose rows fill the threads' steps to nine tenths, as long as there are
// tiles for every CTA and the angles fit.
int tile_of(int num_tokens, int rows, int half, int lanes, int ctas) {
  const int step = kBatch * kThreads / lanes;
  const int most = std::min(std::min(kThreads, std::max(1, kMaxAngles / half)), (num_tokens - 1) / ctas + 1);
  int best = 1;
  double fill = 0;
  for (int n = 1; n <= most && fill < 0.9; ++n) {
    const double full = double(n) * rows / (double((int64_t(n) * rows - 1) / step + 1) * step);
    if (full > fill) {
      fill = full;
      best = n;
    }
  }
  return best;
}

template <bool kBF16, bool kInterleaved, int kLanes>
cudaError_t launch(RotaryParams p, cudaStream_t s) {
  const int ctas = num_sms() > 0 ? num_sms() * kCtasPerSm : 1024;
  p.tile = tile_of(p.num_tokens, int(p.rows.d), int(p.half.d), kLanes, ctas);
  const dim3 grid(std::min(ctas, (p.num_tokens - 1) / p.tile + 1)), block(kThreads);
  const size_t smem = size_t(p.tile) * (4 * p.half.d * sizeof(float) + 2 * sizeof(int));   // at most 34 KB
  return p.q_weight || p.k_weight
             ? launch_pdl(qk_rotary_kernel<kBF16, kInterleaved, kLanes, true>, grid, block, smem, s, p)
             : launch_pdl(qk_rotary_kernel<kBF16, kInterleaved, kLanes, false>, grid, block, smem, s, p);
}
template <bool kBF16, bool kInterleaved>
cudaError_t launch(const RotaryParams& p, cudaStream_t s) {
  if (p.head_dim <= 64) return launch<kBF16, kInterleaved, 4>(p, s);
  if (p.head_dim <= 128) return launch<kBF16, kInterleaved, 8>(p, s);
  return launch<kBF16, kInterleaved, 16>(p, s);
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
  RotaryParams p = {.rows = Divisor(num_heads + num_kv_heads), .half = Divisor(rotary_dim / 2)};
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
