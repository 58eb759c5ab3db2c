// What the paged-decode kernels share: their parameters, the split of the (sequence, kv head, tile) list
// over worker warps, and the launch of the merge that follows.
#pragma once

#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {

enum { KV_F16 = 0, KV_BF16 = 1, KV_E4M3 = 2 };

constexpr int kBS = 16;        // tokens per tile: a 16-token block, or half of a 32-token one
constexpr int kMaxWarps = 12;  // worker warps per CTA (3 per SM sub-partition)
constexpr int kMaxGroup = 8;   // query heads per kv head handled by one n=8 MMA tile

struct DecodeParams {
  void* out;
  const void* q;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const float* k_scale;
  const float* v_scale;
  int num_seqs;
  int num_kv_heads;
  int group;
  int max_blocks;
  int max_len;            // min(max_blocks * block_size, max_context_len): lengths are clamped to it
  int num_blocks;
  int block_size;         // tokens per pool block: 16 or 32 (1 or 2 tiles)
  int tile_shift;         // log2(block_size / 16)
  int part_blocks;        // tiles per partition; 0 = balanced split
  int num_workers;        // gridDim.x * worker warps per CTA
  int defer_dependents;   // 1: the merge kernel launches when this grid completes, not at its start
  float scale_log2;       // softmax scale * log2(e)
  float2* ml;             // [slots][group] (running max in log2 units, sum of exponentials)
  float* po;              // [slots][group][D] unnormalised partial outputs
  unsigned* err;
  // Fused append (null k_new: plain decode): each sequence's new K/V row, [num_seqs][num_kv_heads][D]
  // in the q dtype, belongs at position context_len - 1; it is written to the caches and attended.
  const void* k_new;
  const void* v_new;
  void* k_cache;
  void* v_cache;
};

struct Tile {
  int s, h, b, nb, len;
};

// Largest s in [lo, hi] with mult * cum[s] <= t, given mult * cum[lo] <= t.  cum is a
// non-decreasing prefix array whose scaled entries stay below 2^31 (checked on the host).
__device__ __forceinline__ int find_seq(const int* cum, int lo, int hi, int t, int mult) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (mult * cum[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The same search over [0, S) done by a whole warp for one t: each round the 32 lanes probe
// 32 evenly spaced candidates and a ballot keeps the chunk holding the answer, so S entries
// take ceil(log32 S) rounds instead of log2 S dependent probes.
__device__ __forceinline__ int find_seq_warp(const int* cum, int S, int t, int mult, int lane) {
  int lo = 0, n = S;                         // the answer lies in [lo, lo + n); mult * cum[lo] <= t
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int pos = lo + lane * step;
    const bool ok = lane * step < n && mult * cum[pos] <= t;
    const unsigned b = __ballot_sync(0xffffffffu, ok);   // lane 0 always holds: b != 0
    const int k = 31 - __clz(b);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

__device__ __forceinline__ int clamp_len(int L, int max_len) { return min(max(L, 0), max_len); }

// Workers that share `units` tiles of `segments` (sequence, kv head) pairs in the decode over 4 bits.  More
// workers shorten each one's walk, by about 0.3 us a tile, and lengthen the merge, by 6 ns a piece: the sum
// is least at sqrt(48 units segments).  One sequence of 131,072 tokens, 8 heads over one: 20 us, and 45 with
// every worker.
__device__ __forceinline__ int workers_wide(int64_t units, int num_workers, int segments) {
  const int64_t most = min(int64_t(num_workers), units);
  const float best = __fsqrt_rn(48.f * float(units) * float(segments));
  return best < float(most) ? max(1, int(best)) : int(most);
}

// Dynamic shared memory a launch of `kern` may request: the device's per-CTA opt-in limit
// less the kernel's static arrays.
template <typename K>
size_t dynamic_smem_limit(K kern) {
  int dev = 0, optin = 0;
  cudaFuncAttributes fa = {};
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
      cudaFuncGetAttributes(&fa, kern) != cudaSuccess || size_t(optin) <= fa.sharedSizeBytes)
    return 0;
  return size_t(optin) - fa.sharedSizeBytes;
}

// Launches the split-KV merge behind a decode kernel that ran with prm.num_workers worker warps.
// wide: workers_wide was the split, and a head whose sum of exponentials is NaN gives NaN (else zeros).
pkv_status launch_merge(const DecodeParams& prm, bool q_bf16, int head_dim, bool wide, cudaStream_t stream);

// The decode kernel over 4-bit caches, with its merge.
pkv_status launch_decode_fp4(DecodeParams prm, bool q_bf16, int head_dim, int grid, cudaStream_t stream);

}  // namespace pkv
