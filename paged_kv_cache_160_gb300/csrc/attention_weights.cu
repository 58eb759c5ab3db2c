// attention_weights: the attention weight that each cached token gets from a chunk's rows, summed over the rows and
// over the query heads of its kv head, and added to what it had.
//
// Mathematics: with the rows' log-sum-exp known, p = exp(scale q . k - lse) needs no other key: a key's sum is
// its own, and nothing is exchanged between keys.
#include "cache_row.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

struct WeightsParams {
  float* out;
  const float* in;
  float decay;
  const int32_t* rows;
  const uint8_t* q;
  const float* lse;
  const int32_t* cu_q;
  const int32_t* start;
  const int32_t* tables;
  const uint8_t* k_cache;
  const float* k_scale;
  int num_rows, max_len, num_chunks, total_q, num_heads, num_kv_heads, max_blocks, num_blocks, block_size;
  pkv_dtype kv;
  float scale;
  unsigned* err;
};

// A warp per (chunk, kv head, key).
template <bool kBF16, int D>
__global__ void __launch_bounds__(256) weights_kernel(const WeightsParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, g = blockIdx.y, G = p.num_heads / p.num_kv_heads;
  for (int i = blockIdx.z; i < p.num_chunks; i += gridDim.z) {
    const int64_t q0 = p.cu_q[i], n = p.cu_q[i + 1] - q0, start = p.start[i];
    const bool one = threadIdx.x == 0 && blockIdx.x == 0 && g == 0;
    if (one && i == 0 && p.cu_q[0] != 0) set_error(p.err, PKV_DEVERR_CHUNK);
    if (q0 < 0 || n < 0 || q0 + n > p.total_q || start < 0 || (n > 0 && start + n > int64_t(p.max_blocks) * p.block_size)) {
      if (one) set_error(p.err, PKV_DEVERR_CHUNK);
      continue;
    }
    const int row = p.rows ? p.rows[i] : i;
    if (n == 0 || row < 0) continue;
    if (row >= p.num_rows || start + n > p.max_len) {
      if (one) set_error(p.err, row >= p.num_rows ? PKV_DEVERR_SLOT : PKV_DEVERR_CONTEXT_LEN);
      continue;
    }
    constexpr int kPairs = D / 64;
    const float ks = (p.k_scale ? p.k_scale[g] : 1.f) * p.scale;
    for (int64_t j = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); j < start + n; j += int64_t(gridDim.x) * 8) {
      const int blk = p.tables[int64_t(i) * p.max_blocks + j / p.block_size];
      const bool there = blk >= 0 && blk < p.num_blocks;
      if (!there && lane == 0) set_error(p.err, PKV_DEVERR_BLOCK_ID);
      const int64_t at = (int64_t(blk) * p.num_kv_heads + g) * p.block_size + j % p.block_size;
      float2 k[kPairs];
      for (int c = 0; c < kPairs; ++c)
        k[c] = there ? cache_pair(p.k_cache, p.kv, D, at, 32 * c + lane) : make_float2(0.f, 0.f);
      float sum = 0.f;
      for (int64_t r = j > start ? j - start : 0; r < n; ++r) {
        for (int h = g * G; h < (g + 1) * G; ++h) {
          const int64_t unit = (q0 + r) * p.num_heads + h;
          float s = 0.f;
          for (int c = 0; c < kPairs; ++c) {
            const float2 q = unpack2<kBF16>(reinterpret_cast<const uint32_t*>(p.q)[unit * (D / 2) + 32 * c + lane]);
            s += q.x * k[c].x + q.y * k[c].y;
          }
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          sum += expf(s * ks - p.lse[unit]);
        }
      }
      if (lane == 0) {
        const int64_t w = (int64_t(row) * p.num_kv_heads + g) * p.max_len + j;
        p.out[w] = p.in && j < start ? p.decay * p.in[w] + sum : sum;
      }
    }
  }
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_attention_weights(float* out, const float* weights, float decay, int num_rows, int max_len,
                                            const int32_t* rows, const void* q, pkv_dtype q_dtype, const float* lse,
                                            const int32_t* cu_q_lens, const int32_t* q_start_pos, int num_chunks,
                                            int total_q, int num_heads, const void* k_cache,
                                            const pkv_cache_desc* cache, const int32_t* block_tables,
                                            int max_blocks_per_seq, float scale, pkv_stream_t stream) {
  using namespace pkv;
  pkv_status st = check_cache_desc(cache);
  if (st != PKV_OK) return st;
  if (num_chunks < 0 || total_q < 0 || num_heads <= 0 || max_blocks_per_seq < 0 || num_rows < 0 || max_len < 0 ||
      num_heads % cache->num_kv_heads)
    return PKV_ERR_INVALID_ARG;
  if (q_dtype != PKV_F16 && q_dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale > 3.4e38f || !(decay >= 0.f) || decay > 3.4e38f) return PKV_ERR_INVALID_ARG;
  if ((cache->kv_dtype == PKV_F16 || cache->kv_dtype == PKV_BF16) && cache->kv_dtype != q_dtype)
    return PKV_ERR_UNSUPPORTED;
  if (cache->head_dim != 64 && cache->head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (cache->block_size != 16 && cache->block_size != 32) return PKV_ERR_UNSUPPORTED;
  if (!chunk_work_fits(num_chunks, total_q, num_heads, max_blocks_per_seq, cache)) return PKV_ERR_UNSUPPORTED;
  if (num_chunks == 0 || total_q == 0) return PKV_OK;
  if (!out || !q || !lse || !cu_q_lens || !q_start_pos || !k_cache || !block_tables || max_blocks_per_seq == 0 ||
      num_rows == 0 || max_len == 0)
    return PKV_ERR_INVALID_ARG;
  auto misaligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
  if (!aligned16(q) || !aligned16(k_cache) || misaligned(out) || misaligned(weights) || misaligned(lse) ||
      misaligned(rows) || misaligned(cu_q_lens) || misaligned(q_start_pos) || misaligned(block_tables))
    return PKV_ERR_INVALID_ARG;
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  WeightsParams prm;
  prm.out = out;
  prm.in = weights;
  prm.decay = decay;
  prm.rows = rows;
  prm.q = static_cast<const uint8_t*>(q);
  prm.lse = lse;
  prm.cu_q = cu_q_lens;
  prm.start = q_start_pos;
  prm.tables = block_tables;
  prm.k_cache = static_cast<const uint8_t*>(k_cache);
  prm.k_scale = cache->k_scale;
  prm.num_rows = num_rows;
  prm.max_len = max_len;
  prm.num_chunks = num_chunks;
  prm.total_q = total_q;
  prm.num_heads = num_heads;
  prm.num_kv_heads = cache->num_kv_heads;
  prm.max_blocks = max_blocks_per_seq;
  prm.num_blocks = cache->num_blocks;
  prm.block_size = cache->block_size;
  prm.kv = cache->kv_dtype;
  prm.scale = scale;
  prm.err = err;
  auto kern = q_dtype == PKV_BF16 ? (cache->head_dim == 128 ? weights_kernel<true, 128> : weights_kernel<true, 64>)
                                  : (cache->head_dim == 128 ? weights_kernel<false, 128> : weights_kernel<false, 64>);
  const dim3 grid(unsigned(max_len < 8 * 1024 ? (max_len + 7) / 8 : 1024), unsigned(cache->num_kv_heads),
                  unsigned(num_chunks < 65535 ? num_chunks : 65535));
  return launch_pdl(kern, grid, dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), prm) == cudaSuccess ? PKV_OK
                                                                                                         : PKV_ERR_CUDA;
}
