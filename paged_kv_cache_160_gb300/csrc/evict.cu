// evict_select and evict_compact: which tokens of a sequence each kv head keeps, and their move to the front of
// the sequence's blocks.
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

// ---------------------------------------------------------------------------------------
// select
// ---------------------------------------------------------------------------------------
constexpr int kSelThreads = 1024;

struct SelectParams {
  int32_t* kept;
  const float* weights;
  const int32_t* rows;
  const int32_t* lens;
  const int32_t* keep;
  int max_keep, num_rows, max_len, num_seqs, num_kv_heads, first, recent;
  unsigned* err;
};

// Weights as unsigned numbers of the same order: -0 equals 0, NaN is below everything.
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sum over the CTA's threads; total in `total`.  Two barriers.
__device__ __forceinline__ uint32_t scan_cta(uint32_t v, uint32_t* sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  uint32_t s = sums[lane], t = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += y;
  }
  total = __shfl_sync(0xffffffffu, t, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, t - s, warp);
  __syncthreads();
  return before + x - v;
}

// A CTA per (sequence, kv head): the rank of the last one kept is found 8 bits at a time, then one ordered pass
// writes the positions.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
  __shared__ uint32_t hist[256], sums[32], found[2];
  griddep_launch_dependents();
  griddep_wait();
  const int i = blockIdx.x / p.num_kv_heads, h = blockIdx.x % p.num_kv_heads, tid = threadIdx.x;
  int32_t* kept = p.kept + int64_t(blockIdx.x) * p.max_keep;
  const int L = p.lens[i], want = p.keep[i], row = p.rows ? p.rows[i] : i;
  int n = 0;
  if (L < 0 || L > p.max_len || want < 0 || want > p.max_keep) {
    if (tid == 0) set_error(p.err, PKV_DEVERR_CONTEXT_LEN);
  } else if (row >= p.num_rows) {
    if (tid == 0) set_error(p.err, PKV_DEVERR_SLOT);
  } else if (row >= 0) {
    n = min(L, want);
  }
  for (int j = n + tid; j < p.max_keep; j += kSelThreads) kept[j] = -1;
  if (n == 0) return;
  const int r = min(p.recent, n), f = min(p.first, n - r), rest = n - r - f;
  for (int j = tid; j < f; j += kSelThreads) kept[j] = j;
  for (int j = tid; j < r; j += kSelThreads) kept[n - r + j] = L - r + j;
  if (rest == 0) return;
  const float* w = p.weights + (int64_t(row) * p.num_kv_heads + h) * p.max_len;
  const int lo = f, hi = L - r;
  uint32_t prefix = 0, need = rest;                          // the threshold's leading bits; how many from there on
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int j = lo + tid; j < hi; j += kSelThreads) {
      const uint32_t k = rank_of(w[j]);
      if (shift == 24 || k >> (shift + 8) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1u);
    }
    __syncthreads();
    uint32_t total;                                          // bins from the top down
    const uint32_t c = tid < 256 ? hist[255 - tid] : 0, before = scan_cta(c, sums, total);
    if (tid < 256 && before < need && need <= before + c) {
      found[0] = prefix << 8 | (255 - tid);
      found[1] = need - before;
    }
    __syncthreads();
    prefix = found[0];
    need = found[1];
    __syncthreads();
  }
  // prefix: the least rank kept; `need` of its holders, the lowest positions.
  uint32_t above = 0, equal = 0;                             // among the positions walked
  for (int j0 = lo; j0 < hi; j0 += kSelThreads) {
    const int j = j0 + tid;
    const uint32_t k = j < hi ? rank_of(w[j]) : 0;
    const bool a = j < hi && k > prefix, e = j < hi && k == prefix;
    uint32_t total;
    const uint32_t before = scan_cta(uint32_t(a) | uint32_t(e) << 16, sums, total);
    const uint32_t na = above + (before & 0xffffu), ne = equal + (before >> 16);
    if (a || (e && ne < need)) kept[f + na + min(ne, need)] = j;
    above += total & 0xffffu;
    equal += total >> 16;
  }
}

// ---------------------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------------------
constexpr int kMoveThreads = 256;

struct CompactParams {
  uint8_t* cache[2];
  const int32_t* kept;
  const int32_t* keep;
  const int32_t* src_tables;
  const int32_t* dst_tables;
  float* weights;
  const int32_t* rows;
  const int32_t* dst_rows;
  int max_keep, src_blocks, dst_blocks, num_rows, max_len, num_kv_heads, num_blocks, block_size, head_dim, kv;
  unsigned* err;
};

// A CTA per (sequence, kv head) and K, V or the weights: a thread per kept row, as many rows at a time as threads.
// Rows only move forward to lower positions, so a step's reads are all that its writes have to wait for.
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const CompactParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int i = blockIdx.x / p.num_kv_heads, h = blockIdx.x % p.num_kv_heads, which = blockIdx.y;
  const int32_t* kept = p.kept + int64_t(blockIdx.x) * p.max_keep;
  int n = p.keep[i];
  if (n < 0 || n > p.max_keep) {
    if (threadIdx.x == 0) set_error(p.err, PKV_DEVERR_CONTEXT_LEN);
    return;
  }
  const int D = p.head_dim;
  for (int j0 = 0; j0 < n; j0 += kMoveThreads) {
    const int j = j0 + threadIdx.x, q = j < n ? kept[j] : -1;
    bool ok = q >= 0;
    if (ok && (q < j || (j > 0 && kept[j - 1] >= q))) {
      set_error(p.err, PKV_DEVERR_CHUNK);
      ok = false;
    }
    if (which == 2) {
      const int from = p.rows ? p.rows[i] : i, to = p.dst_rows ? p.dst_rows[i] : from;
      ok = ok && from >= 0 && to >= 0;
      if (ok && (from >= p.num_rows || to >= p.num_rows || q >= p.max_len)) {
        set_error(p.err, q >= p.max_len ? PKV_DEVERR_CONTEXT_LEN : PKV_DEVERR_SLOT);
        ok = false;
      }
      const float v = ok ? p.weights[(int64_t(from) * p.num_kv_heads + h) * p.max_len + q] : 0.f;
      __syncthreads();
      if (ok) p.weights[(int64_t(to) * p.num_kv_heads + h) * p.max_len + j] = v;
      continue;
    }
    int64_t src = 0, dst = 0;
    if (ok && (q / p.block_size >= p.src_blocks || j / p.block_size >= p.dst_blocks)) {
      set_error(p.err, PKV_DEVERR_CHUNK);
      ok = false;
    }
    if (ok) {
      const int sb = p.src_tables[int64_t(i) * p.src_blocks + q / p.block_size];
      const int db = p.dst_tables[int64_t(i) * p.dst_blocks + j / p.block_size];
      if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
        set_error(p.err, PKV_DEVERR_BLOCK_ID);
        ok = false;
      }
      src = (int64_t(sb) * p.num_kv_heads + h) * p.block_size + q % p.block_size;
      dst = (int64_t(db) * p.num_kv_heads + h) * p.block_size + j % p.block_size;
    }
    uint8_t* cache = p.cache[which];
    const bool fp4 = p.kv == PKV_FP4_E2M1;
    const int bytes = fp4 ? D / 2 : p.kv == PKV_FP8_E4M3 ? D : 2 * D;
    auto code_of = [&](int64_t row) { return fp4 ? (row >> 4) * 9 * D + (row & 15) * (D / 2) : row * bytes; };
    auto scale_of = [&](int64_t row) { return (row >> 4) * 9 * D + 8 * D + (row & 15) * (D / 16); };
    for (int b = 0; b < bytes; b += 64) {                    // 64 bytes of the row at a time, the whole CTA's rows
      uint2 v[8];
      for (int c = 0; c < 8 && ok; ++c)
        if (b + 8 * c < bytes) v[c] = *reinterpret_cast<const uint2*>(cache + code_of(src) + b + 8 * c);
      __syncthreads();
      for (int c = 0; c < 8 && ok; ++c)
        if (b + 8 * c < bytes) *reinterpret_cast<uint2*>(cache + code_of(dst) + b + 8 * c) = v[c];
    }
    for (int c = 0; fp4 && c < D / 16; ++c) {
      const uint8_t v = ok ? cache[scale_of(src) + c] : 0;
      __syncthreads();
      if (ok) cache[scale_of(dst) + c] = v;
    }
  }
}

}  // namespace
}  // namespace pkv

extern "C" {

pkv_status pkv_evict_select(int32_t* kept, int max_keep, const float* weights, int num_rows, int max_len,
                            const int32_t* rows, const int32_t* context_lens, const int32_t* keep_lens, int num_seqs,
                            int num_kv_heads, int first, int recent, pkv_stream_t stream) {
  using namespace pkv;
  if (max_keep < 0 || num_rows < 0 || max_len < 0 || num_seqs < 0 || num_kv_heads <= 0 || first < 0 || recent < 0)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || max_keep == 0) return PKV_OK;
  if (!kept || !weights || !context_lens || !keep_lens || num_rows == 0 || max_len == 0) return PKV_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(kept), static_cast<const void*>(weights),
                        static_cast<const void*>(rows), static_cast<const void*>(context_lens),
                        static_cast<const void*>(keep_lens)})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return PKV_ERR_INVALID_ARG;
  if (int64_t(num_seqs) * num_kv_heads >= (int64_t(1) << 31)) return PKV_ERR_UNSUPPORTED;
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  SelectParams prm = {kept,    weights, rows,     context_lens, keep_lens, max_keep, num_rows,
                      max_len, num_seqs, num_kv_heads, first,     recent,   err};
  return launch_pdl(select_kernel, dim3(unsigned(num_seqs * num_kv_heads)), dim3(kSelThreads), 0,
                    reinterpret_cast<cudaStream_t>(stream), prm) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

pkv_status pkv_evict_compact(void* k_cache, void* v_cache, const pkv_cache_desc* cache, const int32_t* kept,
                             int max_keep, const int32_t* keep_lens, const int32_t* src_tables, int src_max_blocks,
                             const int32_t* dst_tables, int dst_max_blocks, float* weights, int num_rows, int max_len,
                             const int32_t* rows, const int32_t* dst_rows, int num_seqs, pkv_stream_t stream) {
  using namespace pkv;
  pkv_status st = check_cache_desc(cache);
  if (st != PKV_OK) return st;
  if (max_keep < 0 || src_max_blocks < 0 || dst_max_blocks < 0 || num_rows < 0 || max_len < 0 || num_seqs < 0)
    return PKV_ERR_INVALID_ARG;
  if (cache->head_dim % 16) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || max_keep == 0) return PKV_OK;
  if (!k_cache || !v_cache || !kept || !keep_lens || !src_tables || !dst_tables || src_max_blocks == 0 ||
      dst_max_blocks == 0 || (weights && (num_rows == 0 || max_len == 0)))
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(kept), static_cast<const void*>(weights),
                        static_cast<const void*>(rows), static_cast<const void*>(dst_rows),
                        static_cast<const void*>(keep_lens), static_cast<const void*>(src_tables),
                        static_cast<const void*>(dst_tables)})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return PKV_ERR_INVALID_ARG;
  if (int64_t(num_seqs) * cache->num_kv_heads >= (int64_t(1) << 31)) return PKV_ERR_UNSUPPORTED;
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  CompactParams prm = {{static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache)},
                       kept, keep_lens, src_tables, dst_tables, weights, rows, dst_rows, max_keep, src_max_blocks,
                       dst_max_blocks, num_rows, max_len, cache->num_kv_heads, cache->num_blocks, cache->block_size,
                       cache->head_dim, cache->kv_dtype, err};
  return launch_pdl(compact_kernel, dim3(unsigned(num_seqs * cache->num_kv_heads), weights ? 3 : 2), dim3(kMoveThreads),
                    0, reinterpret_cast<cudaStream_t>(stream), prm) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

}  // extern "C"
