// kv_write (scatter of the step's new K/V rows into their slots), kv_read (a sequence's rows back
// out of its blocks, dequantised) and copy_blocks (the copy step of copy-on-write).  All move
// bytes with 16-byte vector loads/stores where the layout allows; all are bound by HBM traffic
// and, at serving sizes, by launch latency.
//
// Sources: "PagedAttention: manage the KV cache like virtual memory" §3.3 (each new token
// fills its sequence's last block); "Lecture 33 — KV Cache management" §2.2 (slot =
// block * block_size + offset) and §2.4 (copy-on-write copies the shared block).
#include <algorithm>
#include <numeric>
#include <type_traits>

#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;

// Same dtype in and out: every (token, kv head) row is `chunks` 16-byte vectors.
__global__ void __launch_bounds__(kThreads) kv_write_copy_kernel(const uint4* __restrict__ k_new,
                                                                 const uint4* __restrict__ v_new,
                                                                 const int64_t* __restrict__ slots,
                                                                 uint4* __restrict__ k_cache,
                                                                 uint4* __restrict__ v_cache, int num_tokens,
                                                                 int num_kv_heads, int chunks, int block_size,
                                                                 int64_t num_slots, unsigned* err) {
  griddep_launch_dependents();   // a following decode may start its length-only prologue
  griddep_wait();                // the previous kernel (which may read this cache) is done
  const int64_t total = int64_t(num_tokens) * num_kv_heads * chunks;
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < total; i += int64_t(gridDim.x) * blockDim.x) {
    const int c = int(i % chunks);
    const int64_t r = i / chunks;
    const int h = int(r % num_kv_heads);
    const int64_t t = r / num_kv_heads;
    const int64_t slot = slots[t];
    if (slot < 0) continue;                       // padding token
    if (slot >= num_slots) {
      if (c == 0 && h == 0) set_error(err, PKV_DEVERR_SLOT);
      continue;
    }
    const int64_t blk = slot / block_size, off = slot % block_size;
    const int64_t dst = ((blk * num_kv_heads + h) * block_size + off) * chunks + c;
    k_cache[dst] = __ldg(k_new + i);
    v_cache[dst] = __ldg(v_new + i);
  }
}

template <bool kBF16>
__device__ __forceinline__ float2 load2(const void* p) {
  if constexpr (kBF16) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(p));
  }
}

// f16/bf16 rows into an e4m3 cache: code = e4m3(x / scale[h]); 16 codes per thread.
template <bool kBF16>
__global__ void __launch_bounds__(kThreads) kv_write_quant_kernel(
    const uint8_t* __restrict__ k_new, const uint8_t* __restrict__ v_new, const int64_t* __restrict__ slots,
    uint4* __restrict__ k_cache, uint4* __restrict__ v_cache, const float* __restrict__ k_scale,
    const float* __restrict__ v_scale, int num_tokens, int num_kv_heads, int chunks, int block_size,
    int64_t num_slots, unsigned* err) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t total = int64_t(num_tokens) * num_kv_heads * chunks;
  for (int64_t i = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; i < total; i += int64_t(gridDim.x) * blockDim.x) {
    const int c = int(i % chunks);
    const int64_t r = i / chunks;
    const int h = int(r % num_kv_heads);
    const int64_t t = r / num_kv_heads;
    const int64_t slot = slots[t];
    if (slot < 0) continue;
    if (slot >= num_slots) {
      if (c == 0 && h == 0) set_error(err, PKV_DEVERR_SLOT);
      continue;
    }
    const int64_t blk = slot / block_size, off = slot % block_size;
    const int64_t dst = ((blk * num_kv_heads + h) * block_size + off) * chunks + c;
    const float ks = k_scale[h], vs = v_scale[h];
    uint32_t kw[4], vw[4];
    const uint8_t* kp = k_new + i * 32;           // 16 input elements of 2 bytes
    const uint8_t* vp = v_new + i * 32;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float2 a = load2<kBF16>(kp + 8 * w), b = load2<kBF16>(kp + 8 * w + 4);
      kw[w] = f32x2_to_e4m3x2(__fdiv_rn(a.x, ks), __fdiv_rn(a.y, ks)) |
              (f32x2_to_e4m3x2(__fdiv_rn(b.x, ks), __fdiv_rn(b.y, ks)) << 16);
      a = load2<kBF16>(vp + 8 * w);
      b = load2<kBF16>(vp + 8 * w + 4);
      vw[w] = f32x2_to_e4m3x2(__fdiv_rn(a.x, vs), __fdiv_rn(a.y, vs)) |
              (f32x2_to_e4m3x2(__fdiv_rn(b.x, vs), __fdiv_rn(b.y, vs)) << 16);
    }
    k_cache[dst] = make_uint4(kw[0], kw[1], kw[2], kw[3]);
    v_cache[dst] = make_uint4(vw[0], vw[1], vw[2], vw[3]);
  }
}

// f16/bf16 rows into a 4-bit cache; 16 elements (one scale) of K and of V per thread and step.  The grid's
// threads are a whole number of tokens (grid_of_tokens), so that a thread keeps its head and its place in
// the head and works its head's scale out once; the next step's rows and slot are on their way meanwhile.
//   Bound by the instructions of the quantising as much as by memory.  32,768 tokens of 8 heads, D 128, with
// head scales: 34.6 us, 172 MB at 5.0 TB/s; a thread per 16 elements without the loop took 38.4, and K after V
// instead of both at once 37.8.  More CTAs per SM leave a thread too few registers for both (3: 38.5 us).
constexpr int kFp4Ctas = 2;      // resident per SM

// Elements that are not ordinary (quant16_e2m1_ordinary), out of the way of those that are.
template <bool kBF16>
__device__ __noinline__ uint2 quant16_any(const uint4 a, const uint4 b, const HeadScale hs, uint32_t& scale_code) {
  return quant16_e2m1<kBF16>(a, b, hs, scale_code);
}

template <bool kBF16, bool kScaled>
__global__ void __launch_bounds__(kThreads, kFp4Ctas) kv_write_fp4_kernel(
    const uint4* __restrict__ k_new, const uint4* __restrict__ v_new, const int64_t* __restrict__ slots,
    uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache, const float* __restrict__ k_scale,
    const float* __restrict__ v_scale, int num_tokens, int num_kv_heads, const Divisor groups_of, const Divisor per_token_of,
    const Divisor block_size_of, int64_t num_slots, unsigned* err) {
  griddep_launch_dependents();
  griddep_wait();
  const int per_token = int(per_token_of.d), groups = int(groups_of.d), block_size = int(block_size_of.d);
  const int64_t first = blockIdx.x * int64_t(kThreads) + threadIdx.x, threads = int64_t(gridDim.x) * kThreads;
  const bool narrow = threads <= 0x7fffffff;
  int64_t t = narrow ? int64_t(per_token_of.quotient(uint32_t(first))) : first / per_token;
  if (t >= num_tokens) return;
  const int64_t step = narrow ? int64_t(per_token_of.quotient(uint32_t(threads))) : threads / per_token;   // tokens; no remainder
  const int c = int(first - t * per_token), h = int(groups_of.quotient(uint32_t(c))), g = c - h * groups;
  const uint4 *ks = k_new + 2 * first, *vs = v_new + 2 * first;
  uint4 k0 = __ldcs(ks), k1 = __ldcs(ks + 1), v0 = __ldcs(vs), v1 = __ldcs(vs + 1);
  int64_t slot = slots[t];
  const HeadScale hk(k_scale, h), hv(v_scale, h);
  while (true) {
    const uint4 a0 = k0, a1 = k1, b0 = v0, b1 = v1;
    const int64_t at_slot = slot;
    t += step;
    const bool more = t < num_tokens;
    if (more) {
      ks += 2 * threads;
      vs += 2 * threads;
      k0 = __ldcs(ks);
      k1 = __ldcs(ks + 1);
      v0 = __ldcs(vs);
      v1 = __ldcs(vs + 1);
      slot = slots[t];
    }
    if (at_slot >= num_slots) {
      if (c == 0) set_error(err, PKV_DEVERR_SLOT);
    } else if (at_slot >= 0) {                                     // (negative: a padding token)
      const int64_t blk = num_slots <= 0x7fffffff ? int64_t(block_size_of.quotient(uint32_t(at_slot))) : at_slot / block_size;
      const int64_t row = (blk * num_kv_heads + h) * block_size + (at_slot - blk * block_size);
      const int64_t base = (row >> 4) * 144 * groups;              // 9 * head_dim bytes per tile
      const int rr = int(row & 15);
      const int64_t at = base + (rr * groups + g) * 8, sat = base + 128 * groups + rr * groups + g;
      uint2 kc, vc;
      uint32_t ksc, vsc;
      const bool k_ok = quant16_e2m1_ordinary<kBF16, kScaled>(a0, a1, hk, kc, ksc);
      const bool v_ok = quant16_e2m1_ordinary<kBF16, kScaled>(b0, b1, hv, vc, vsc);
      if (!(k_ok && v_ok)) {
        kc = quant16_any<kBF16>(a0, a1, hk, ksc);
        vc = quant16_any<kBF16>(b0, b1, hv, vsc);
      }
      *reinterpret_cast<uint2*>(k_cache + at) = kc;
      k_cache[sat] = uint8_t(ksc);
      *reinterpret_cast<uint2*>(v_cache + at) = vc;
      v_cache[sat] = uint8_t(vsc);
    }
    if (!more) break;
  }
}

// ---------------------------------------------------------------------------------------
// kv_read
// ---------------------------------------------------------------------------------------
struct ReadParams {
  uint8_t* k_out;
  uint8_t* v_out;
  const int32_t* cu_lens;
  const int32_t* block_tables;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  int total_tokens;
  int num_seqs;
  int max_blocks;
  int num_blocks;
  int num_kv_heads;
  int block_size;
  int head_dim;
  int rows;               // output rows per CTA, at most kReadRows
  unsigned* err;
};

constexpr int kReadRows = 32;    // output rows per CTA at most

// Eight elements (8 c .. of a row) as stored, and as 16 output bytes.  Eight and not more, so that a
// warp's stores are runs of whole sectors.
template <pkv_dtype KV>
struct Stored8 {
  static constexpr int kWords = KV == PKV_FP4_E2M1 ? 1 : KV == PKV_FP8_E4M3 ? 2 : 4;
  uint32_t w[kWords];
  uint32_t scale;         // 4-bit: the e4m3 code

  __device__ __forceinline__ void load(const uint8_t* cache, int D, int64_t row, int c) {
    if constexpr (KV == PKV_FP4_E2M1) {
      const uint8_t* tile = cache + (row >> 4) * 9 * D;
      const int rr = int(row & 15);
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(tile + rr * (D / 2) + 4 * c));
      scale = __ldg(tile + 8 * D + rr * (D / 16) + (c >> 1));
    } else if constexpr (KV == PKV_FP8_E4M3) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(cache + row * D + 8 * c));
      w[0] = v.x;
      w[1] = v.y;
    } else {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(cache + (row * D + 8 * c) * 2));
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    }
  }
  template <bool kBF16>
  __device__ __forceinline__ uint4 value(float head_scale) const {
    if constexpr (KV == PKV_F16 || KV == PKV_BF16) {
      return make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      uint32_t half[4];                                    // fp16 pairs, exact
      if constexpr (KV == PKV_FP8_E4M3) {
        half[0] = e4m3x2_to_f16x2(w[0]);
        half[1] = e4m3x2_to_f16x2(w[0] >> 16);
        half[2] = e4m3x2_to_f16x2(w[1]);
        half[3] = e4m3x2_to_f16x2(w[1] >> 16);
      } else {
        const uint32_t s2 = e4m3x2_to_f16x2(scale * 0x101u);
        e2m1x8_to_f16x8(w[0], half);
#pragma unroll
        for (int k = 0; k < 4; ++k) half[k] = hmul2(half[k], s2);
      }
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2<false>(half[k]);
        o[k] = pack2<kBF16>(f.x * head_scale, f.y * head_scale);
      }
      return make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
};

// A CTA takes p.rows output rows: the first warp finds each one's sequence and pool row, then all
// threads move 8 elements of K and of V at a time, kAhead of them on their way at once as stored.  The host
// picks a number of threads that whole rows of all kv heads divide, so that a thread keeps its place in
// the row.
template <pkv_dtype KV, bool kBF16, bool kFull>              // kFull: p.rows is kReadRows
__global__ void __launch_bounds__(1024) kv_read_kernel(const ReadParams p) {
  const int rows = kFull ? kReadRows : p.rows;
  __shared__ int64_t src_row[kReadRows];                   // row of kv head 0 in the pool, -1: leave the row
  griddep_launch_dependents();
  griddep_wait();
  const int t0 = blockIdx.x * rows, S = p.num_seqs;
  if (blockIdx.x == 0) {                                   // cu_lens ascends from 0 to at most total_tokens
    bool bad = threadIdx.x == 0 && (p.cu_lens[0] != 0 || p.cu_lens[S] > p.total_tokens);
    for (int i = threadIdx.x; i < S; i += blockDim.x) bad |= p.cu_lens[i + 1] < p.cu_lens[i];
    if (bad) set_error(p.err, PKV_DEVERR_CHUNK);
  }
  if (threadIdx.x < 32) {
    static_assert(kReadRows == 32, "a row per lane");
    const int lane = threadIdx.x, t = t0 + lane;
    // The largest i with cu_lens[i] <= t0, 32 probes a round; then each lane walks on to its own row's.
    int lo = 0, n = S;
    while (n > 1) {
      const int step = (n + 31) >> 5, at = lane * step;
      const unsigned b = __ballot_sync(0xffffffffu, at < n && p.cu_lens[lo + at] <= t0);
      const int k = b ? 31 - __clz(b) : 0;
      lo += k * step;
      n = min(step, n - k * step);
    }
    int64_t row = -1;
    if (lane < rows && t < p.total_tokens && t < p.cu_lens[S]) {
      int end = p.cu_lens[lo + 1];
      while (t >= end && lo + 1 < S) end = p.cu_lens[++lo + 1];
      const int j = t - p.cu_lens[lo];
      if (j < 0 || t >= end || j / p.block_size >= p.max_blocks) {
        set_error(p.err, PKV_DEVERR_CHUNK);
      } else {
        const int blk = p.block_tables[int64_t(lo) * p.max_blocks + j / p.block_size];
        if (blk < 0 || blk >= p.num_blocks) set_error(p.err, PKV_DEVERR_BLOCK_ID);
        else row = int64_t(blk) * p.num_kv_heads * p.block_size + j % p.block_size;
      }
    }
    src_row[lane] = row;
  }
  __syncthreads();
  constexpr int kAhead = KV == PKV_F16 || KV == PKV_BF16 ? 2 : 8;
  const int D = p.head_dim, chunks = D / 8, per_row = p.num_kv_heads * chunks;
  const int at_once = max(1, int(blockDim.x) / per_row);   // rows per pass
  const int r0 = threadIdx.x / per_row;
  if (r0 >= at_once) return;
  for (int c = threadIdx.x - r0 * per_row; c < per_row; c += blockDim.x) {   // (once, unless a row is longer than the CTA)
    const int h = c / chunks, chunk = c - h * chunks;
    const float ks = p.k_scale ? __ldg(p.k_scale + h) : 1.f, vs = p.v_scale ? __ldg(p.v_scale + h) : 1.f;
    uint4* ko = reinterpret_cast<uint4*>(p.k_out) + int64_t(t0) * per_row + c;
    uint4* vo = reinterpret_cast<uint4*>(p.v_out) + int64_t(t0) * per_row + c;
    for (int r = r0; r < rows; r += kAhead * at_once) {
      Stored8<KV> k[kAhead], v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int ru = r + u * at_once;
        if (ru >= rows || src_row[ru] < 0) continue;
        const int64_t row = src_row[ru] + int64_t(h) * p.block_size;
        k[u].load(p.k_cache, D, row, chunk);
        v[u].load(p.v_cache, D, row, chunk);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int ru = r + u * at_once;
        if (ru >= rows || src_row[ru] < 0) continue;
        ko[int64_t(ru) * per_row] = k[u].template value<kBF16>(ks);
        vo[int64_t(ru) * per_row] = v[u].template value<kBF16>(vs);
      }
    }
  }
}

// One CTA per (pair, K or V): copies the whole block of `chunks` 16-byte vectors.
__global__ void __launch_bounds__(kThreads) copy_blocks_kernel(uint4* __restrict__ k_cache,
                                                               uint4* __restrict__ v_cache,
                                                               const int32_t* __restrict__ pairs, int num_pairs,
                                                               int num_blocks, int64_t chunks, unsigned* err) {
  griddep_launch_dependents();
  griddep_wait();
  const int pair = blockIdx.x;
  const int32_t src = pairs[2 * pair], dst = pairs[2 * pair + 1];
  // A pair is applied only when both ids are in the pool, its dst is nobody's src and no
  // other pair writes the same dst.
  bool bad = src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks;
  for (int j = threadIdx.x; j < num_pairs && !bad; j += blockDim.x) {
    if (pairs[2 * j] == dst || (j != pair && pairs[2 * j + 1] == dst)) bad = true;
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (threadIdx.x == 0 && blockIdx.y == 0) set_error(err, PKV_DEVERR_COPY_PAIR);
    return;
  }
  uint4* cache = blockIdx.y == 0 ? k_cache : v_cache;
  const uint4* s = cache + int64_t(src) * chunks;
  uint4* d = cache + int64_t(dst) * chunks;
  for (int64_t i = threadIdx.x; i < chunks; i += blockDim.x) d[i] = s[i];
}

// One CTA per (pair, K or V) between two pools of the same block layout, either of which may
// be pinned host memory (Grace reaches it over NVLink-C2C).  Each thread keeps four 16-byte
// loads in flight, so a block is read with few round trips even from host memory.
__global__ void __launch_bounds__(kThreads) swap_blocks_kernel(uint4* __restrict__ dst_k, uint4* __restrict__ dst_v,
                                                               const uint4* __restrict__ src_k,
                                                               const uint4* __restrict__ src_v,
                                                               const int32_t* __restrict__ pairs, int num_pairs,
                                                               int src_blocks, int dst_blocks, int64_t chunks,
                                                               unsigned* err) {
  griddep_launch_dependents();
  griddep_wait();
  const int pair = blockIdx.x;
  const int32_t src = pairs[2 * pair], dst = pairs[2 * pair + 1];
  // Applied only when both ids are inside their pools and no other pair writes the same dst.
  bool bad = src < 0 || src >= src_blocks || dst < 0 || dst >= dst_blocks;
  for (int j = threadIdx.x; j < num_pairs && !bad; j += blockDim.x) {
    if (j != pair && pairs[2 * j + 1] == dst) bad = true;
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (threadIdx.x == 0 && blockIdx.y == 0) set_error(err, PKV_DEVERR_COPY_PAIR);
    return;
  }
  const uint4* sp = (blockIdx.y == 0 ? src_k : src_v) + int64_t(src) * chunks;
  uint4* dp = (blockIdx.y == 0 ? dst_k : dst_v) + int64_t(dst) * chunks;
  constexpr int kUnroll = 4;
  int64_t i = threadIdx.x;
  for (; i + (kUnroll - 1) * int64_t(blockDim.x) < chunks; i += kUnroll * int64_t(blockDim.x)) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = sp[i + u * int64_t(blockDim.x)];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) dp[i + u * int64_t(blockDim.x)] = v[u];
  }
  for (; i < chunks; i += blockDim.x) dp[i] = sp[i];
}

// CTAs for tokens of `per_token` threads' work, whose threads are a whole number of tokens: about `resident`
// of them, fewer where there is less to do.
unsigned grid_of_tokens(int num_tokens, int64_t per_token, int64_t resident) {
  const int64_t unit = per_token / std::gcd(per_token, int64_t(kThreads));   // below 2^24
  const int64_t needed = (num_tokens * per_token - 1) / kThreads + 1;
  return unsigned(std::min((needed - 1) / unit + 1, std::max<int64_t>(1, resident / unit)) * unit);
}

// One 16-byte chunk per thread: these kernels are latency-bound at serving sizes, so every
// thread should issue its loads once rather than loop.
int grid_for(int64_t work) {
  const int64_t per = kThreads;
  int64_t g = (work + per - 1) / per;
  const int cap = num_sms() > 0 ? num_sms() * 64 : 8192;
  if (g > cap) g = cap;
  return g < 1 ? 1 : int(g);
}

}  // namespace
}  // namespace pkv

extern "C" {

pkv_status pkv_kv_write(const void* k_new, const void* v_new, pkv_dtype in_dtype, int num_tokens,
                        const int64_t* slot_mapping, void* k_cache, void* v_cache, const pkv_cache_desc* cache,
                        pkv_stream_t stream) {
  using namespace pkv;
  pkv_status st = check_cache_desc(cache);
  if (st != PKV_OK) return st;
  if (num_tokens < 0) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (!k_new || !v_new || !slot_mapping || !k_cache || !v_cache) return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return PKV_ERR_INVALID_ARG;
  if (in_dtype == PKV_FP4_E2M1) return PKV_ERR_UNSUPPORTED;
  if (in_dtype != PKV_F16 && in_dtype != PKV_BF16 && in_dtype != PKV_FP8_E4M3) return PKV_ERR_INVALID_ARG;
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  const int64_t num_slots = int64_t(cache->num_blocks) * cache->block_size;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (in_dtype == cache->kv_dtype) {
    const int chunks = cache->head_dim * dtype_bytes(in_dtype) / 16;
    const int64_t work = int64_t(num_tokens) * cache->num_kv_heads * chunks;
    if (launch_pdl(kv_write_copy_kernel, dim3(grid_for(work)), dim3(kThreads), 0, s,
                   static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), slot_mapping,
                   static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), num_tokens, cache->num_kv_heads,
                   chunks, cache->block_size, num_slots, err) != cudaSuccess)
      return PKV_ERR_CUDA;
  } else if (cache->kv_dtype == PKV_FP8_E4M3 && (in_dtype == PKV_F16 || in_dtype == PKV_BF16)) {
    const int chunks = cache->head_dim / 16;
    const int64_t work = int64_t(num_tokens) * cache->num_kv_heads * chunks;
    auto kern = in_dtype == PKV_BF16 ? kv_write_quant_kernel<true> : kv_write_quant_kernel<false>;
    if (launch_pdl(kern, dim3(grid_for(work)), dim3(kThreads), 0, s, static_cast<const uint8_t*>(k_new),
                   static_cast<const uint8_t*>(v_new), slot_mapping, static_cast<uint4*>(k_cache),
                   static_cast<uint4*>(v_cache), cache->k_scale, cache->v_scale, num_tokens, cache->num_kv_heads,
                   chunks, cache->block_size, num_slots, err) != cudaSuccess)
      return PKV_ERR_CUDA;
  } else if (cache->kv_dtype == PKV_FP4_E2M1 && (in_dtype == PKV_F16 || in_dtype == PKV_BF16)) {
    const int groups = cache->head_dim / 16;
    const int64_t per_token = int64_t(cache->num_kv_heads) * groups;
    if (per_token >= (int64_t(1) << 24)) return PKV_ERR_UNSUPPORTED;
    const bool scaled = cache->k_scale || cache->v_scale;
    auto kern = in_dtype == PKV_BF16 ? (scaled ? kv_write_fp4_kernel<true, true> : kv_write_fp4_kernel<true, false>)
                                     : (scaled ? kv_write_fp4_kernel<false, true> : kv_write_fp4_kernel<false, false>);
    if (launch_pdl(kern, dim3(grid_of_tokens(num_tokens, per_token, kFp4Ctas * num_sms())), dim3(kThreads), 0, s,
                   static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), slot_mapping,
                   static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), cache->k_scale, cache->v_scale,
                   num_tokens, cache->num_kv_heads, Divisor(groups), Divisor(int(per_token)), Divisor(cache->block_size), num_slots,
                   err) != cudaSuccess)
      return PKV_ERR_CUDA;
  } else {
    return PKV_ERR_UNSUPPORTED;
  }
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_kv_read(void* k_out, void* v_out, pkv_dtype out_dtype, int total_tokens, const int32_t* cu_lens,
                       int num_seqs, const int32_t* block_tables, int max_blocks_per_seq, const void* k_cache,
                       const void* v_cache, const pkv_cache_desc* cache, pkv_stream_t stream) {
  using namespace pkv;
  pkv_status st = check_cache_desc(cache);
  if (st != PKV_OK) return st;
  if (total_tokens < 0 || num_seqs < 0 || max_blocks_per_seq < 0) return PKV_ERR_INVALID_ARG;
  if (out_dtype != PKV_F16 && out_dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  const bool wide = cache->kv_dtype == PKV_F16 || cache->kv_dtype == PKV_BF16;
  if (wide && out_dtype != cache->kv_dtype) return PKV_ERR_UNSUPPORTED;
  if (cache->head_dim % 16) return PKV_ERR_UNSUPPORTED;
  if (total_tokens == 0 || num_seqs == 0) return PKV_OK;
  if (!k_out || !v_out || !cu_lens || !block_tables || !k_cache || !v_cache || max_blocks_per_seq == 0)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(cu_lens) & 3u) || (reinterpret_cast<uintptr_t>(block_tables) & 3u))
    return PKV_ERR_INVALID_ARG;
  if (int64_t(cache->num_kv_heads) * cache->head_dim >= (int64_t(1) << 24))
    return PKV_ERR_UNSUPPORTED;              // the rows of one CTA are indexed in 32 bits
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  ReadParams prm;
  prm.k_out = static_cast<uint8_t*>(k_out);
  prm.v_out = static_cast<uint8_t*>(v_out);
  prm.cu_lens = cu_lens;
  prm.block_tables = block_tables;
  prm.k_cache = static_cast<const uint8_t*>(k_cache);
  prm.v_cache = static_cast<const uint8_t*>(v_cache);
  prm.k_scale = cache->k_scale;
  prm.v_scale = cache->v_scale;
  prm.total_tokens = total_tokens;
  prm.num_seqs = num_seqs;
  prm.max_blocks = max_blocks_per_seq;
  prm.num_blocks = cache->num_blocks;
  prm.num_kv_heads = cache->num_kv_heads;
  prm.block_size = cache->block_size;
  prm.head_dim = cache->head_dim;
  prm.err = err;
  const bool bf = out_dtype == PKV_BF16;
  // Whole rows of all kv heads, 256 threads or more, in full warps; longer rows are walked.
  const int per_row = cache->num_kv_heads * (cache->head_dim / 8);
  const int threads = per_row >= 1024 ? 1024 : std::min(1024, (per_row * std::max(1, kThreads / per_row) + 31) / 32 * 32);
  // A CTA takes 32 rows, fewer where that leaves SMs with less than four CTAs; whole passes of its threads.
  // 4096 tokens of 4 heads, D 128, from 4 bits: 4.1 us, 5.9 by 32 rows.
  const int pass = std::max(1, threads / per_row), share = (total_tokens - 1) / (4 * std::max(1, num_sms())) + 1;
  prm.rows = std::min(kReadRows, (share + pass - 1) / pass * pass);
  const int grid = (total_tokens - 1) / prm.rows + 1;
  auto pick = [&](auto full) {
    constexpr bool kFull = decltype(full)::value;
    return wide ? (bf ? kv_read_kernel<PKV_BF16, true, kFull> : kv_read_kernel<PKV_F16, false, kFull>)
           : cache->kv_dtype == PKV_FP8_E4M3
               ? (bf ? kv_read_kernel<PKV_FP8_E4M3, true, kFull> : kv_read_kernel<PKV_FP8_E4M3, false, kFull>)
               : (bf ? kv_read_kernel<PKV_FP4_E2M1, true, kFull> : kv_read_kernel<PKV_FP4_E2M1, false, kFull>);
  };
  auto kern = prm.rows == kReadRows ? pick(std::true_type{}) : pick(std::false_type{});
  return launch_pdl(kern, dim3(grid), dim3(threads), 0, reinterpret_cast<cudaStream_t>(stream), prm) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

pkv_status pkv_copy_blocks(void* k_cache, void* v_cache, const pkv_cache_desc* cache, const int32_t* block_pairs,
                           int num_pairs, pkv_stream_t stream) {
  using namespace pkv;
  pkv_status st = check_cache_desc(cache);
  if (st != PKV_OK) return st;
  if (num_pairs < 0) return PKV_ERR_INVALID_ARG;
  if (num_pairs == 0) return PKV_OK;
  if (!k_cache || !v_cache || !block_pairs) return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || (reinterpret_cast<uintptr_t>(block_pairs) & 7u))
    return PKV_ERR_INVALID_ARG;
  if (num_pairs > 65535) return PKV_ERR_UNSUPPORTED;
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  const int64_t chunks = cache_block_bytes(cache) / 16;
  dim3 grid(num_pairs, 2);
  if (launch_pdl(copy_blocks_kernel, grid, dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream),
                 static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), block_pairs, num_pairs,
                 cache->num_blocks, chunks, err) != cudaSuccess)
    return PKV_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_swap_blocks(void* dst_k, void* dst_v, int dst_num_blocks, const void* src_k, const void* src_v,
                           int src_num_blocks, const pkv_cache_desc* layout, const int32_t* block_pairs,
                           int num_pairs, pkv_stream_t stream) {
  using namespace pkv;
  pkv_status st = check_cache_desc(layout);
  if (st != PKV_OK) return st;
  if (num_pairs < 0 || dst_num_blocks <= 0 || src_num_blocks <= 0) return PKV_ERR_INVALID_ARG;
  if (num_pairs == 0) return PKV_OK;
  if (!dst_k || !dst_v || !src_k || !src_v || !block_pairs) return PKV_ERR_INVALID_ARG;
  if (!aligned16(dst_k) || !aligned16(dst_v) || !aligned16(src_k) || !aligned16(src_v) ||
      (reinterpret_cast<uintptr_t>(block_pairs) & 7u))
    return PKV_ERR_INVALID_ARG;
  if (num_pairs > 65535) return PKV_ERR_UNSUPPORTED;
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  const int64_t block_bytes = cache_block_bytes(layout);
  if (launch_pdl(swap_blocks_kernel, dim3(num_pairs, 2), dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream),
                 static_cast<uint4*>(dst_k), static_cast<uint4*>(dst_v), static_cast<const uint4*>(src_k),
                 static_cast<const uint4*>(src_v), block_pairs, num_pairs, src_num_blocks, dst_num_blocks,
                 block_bytes / 16, err) != cudaSuccess)
    return PKV_ERR_CUDA;
  return PKV_OK;
}

}  // extern "C"
