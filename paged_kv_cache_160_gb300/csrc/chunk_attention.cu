// paged_chunk_attention: causal attention of each sequence's new rows over its paged cache of any type.
//
// Mathematics: row r of a chunk at positions start .. start + L - 1 attends keys 0 .. start + r, in one pass with
// the running maximum m and sum l of the softmax: out = O / l, lse = m + log l.
#include "cache_row.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

struct ChunkParams {
  uint8_t* out;
  float* lse;
  const uint8_t* q;
  const int32_t* cu_q;
  const int32_t* start;
  const int32_t* tables;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  int num_chunks, total_q, num_heads, num_kv_heads, max_blocks, num_blocks, block_size;
  pkv_dtype kv;
  float scale;
  unsigned* err;
};

// A warp per (query row, head).
template <bool kBF16, int D>
__global__ void __launch_bounds__(256) chunk_kernel(const ChunkParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t unit = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int t = int(unit / p.num_heads), h = int(unit % p.num_heads), g = h / (p.num_heads / p.num_kv_heads);
  if (blockIdx.x == 0) {
    bool bad = threadIdx.x == 0 && p.cu_q[0] != 0;
    for (int i = threadIdx.x; i < p.num_chunks; i += blockDim.x) {
      const int64_t q0 = p.cu_q[i], n = p.cu_q[i + 1] - q0, s = p.start[i];
      bad |= q0 < 0 || n < 0 || q0 + n > p.total_q || s < 0 || (n > 0 && s + n > int64_t(p.max_blocks) * p.block_size);
    }
    if (bad) set_error(p.err, PKV_DEVERR_CHUNK);
  }
  if (t >= p.total_q) return;
  int lo = 0, hi = p.num_chunks;                             // the chunk of row t
  while (lo + 1 < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_q[mid] <= t) lo = mid; else hi = mid;
  }
  const int q0 = p.cu_q[lo], n = p.cu_q[lo + 1] - q0, start = p.start[lo];
  if (q0 < 0 || t < q0 || t - q0 >= n || int64_t(q0) + n > p.total_q || start < 0 ||
      int64_t(start) + n > int64_t(p.max_blocks) * p.block_size)
    return;
  constexpr int kPairs = D / 64;                             // of this lane
  const float ks = p.k_scale ? p.k_scale[g] : 1.f, vs = p.v_scale ? p.v_scale[g] : 1.f;
  float2 q[kPairs], o[kPairs];
  for (int c = 0; c < kPairs; ++c) {
    q[c] = unpack2<kBF16>(reinterpret_cast<const uint32_t*>(p.q)[unit * (D / 2) + 32 * c + lane]);
    o[c] = make_float2(0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j <= start + t - q0; ++j) {
    const int blk = p.tables[int64_t(lo) * p.max_blocks + j / p.block_size];
    const bool there = blk >= 0 && blk < p.num_blocks;
    if (!there && lane == 0) set_error(p.err, PKV_DEVERR_BLOCK_ID);
    const int64_t row = (int64_t(blk) * p.num_kv_heads + g) * p.block_size + j % p.block_size;
    float s = 0.f;
    for (int c = 0; c < kPairs && there; ++c) {
      const float2 k = cache_pair(p.k_cache, p.kv, D, row, 32 * c + lane);
      s += q[c].x * k.x + q[c].y * k.y;
    }
    for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    s *= ks * p.scale;
    const float m_new = s > m ? s : m, a = m == -INFINITY ? 0.f : expf(m - m_new), e = expf(s - m_new);
    l = l * a + e;
    for (int c = 0; c < kPairs; ++c) {
      const float2 v = there ? cache_pair(p.v_cache, p.kv, D, row, 32 * c + lane) : make_float2(0.f, 0.f);
      o[c].x = o[c].x * a + e * v.x;
      o[c].y = o[c].y * a + e * v.y;
    }
    m = m_new;
  }
  for (int c = 0; c < kPairs; ++c)
    reinterpret_cast<uint32_t*>(p.out)[unit * (D / 2) + 32 * c + lane] = pack2<kBF16>(o[c].x * vs / l, o[c].y * vs / l);
  if (p.lse && lane == 0) p.lse[unit] = m + logf(l);
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_chunk_workspace_bytes(int total_q, int num_heads, int num_kv_heads, int head_dim) {
  return total_q > 0 && num_heads > 0 && num_kv_heads > 0 && head_dim > 0 ? 256 : 0;
}

extern "C" pkv_status pkv_paged_chunk_attention(void* out, float* lse, const void* q, pkv_dtype q_dtype,
                                                const int32_t* cu_q_lens, const int32_t* q_start_pos, int num_chunks,
                                                int total_q, int num_heads, const void* k_cache, const void* v_cache,
                                                const pkv_cache_desc* cache, const int32_t* block_tables,
                                                int max_blocks_per_seq, float scale, void* workspace,
                                                size_t workspace_bytes, pkv_stream_t stream) {
  using namespace pkv;
  pkv_status st = check_cache_desc(cache);
  if (st != PKV_OK) return st;
  if (num_chunks < 0 || total_q < 0 || num_heads <= 0 || max_blocks_per_seq < 0 || num_heads % cache->num_kv_heads)
    return PKV_ERR_INVALID_ARG;
  if (q_dtype != PKV_F16 && q_dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (!(scale > 0.f) || scale > 3.4e38f) return PKV_ERR_INVALID_ARG;
  if ((cache->kv_dtype == PKV_F16 || cache->kv_dtype == PKV_BF16) && cache->kv_dtype != q_dtype)
    return PKV_ERR_UNSUPPORTED;
  if (cache->head_dim != 64 && cache->head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (cache->block_size != 16 && cache->block_size != 32) return PKV_ERR_UNSUPPORTED;
  if (!chunk_work_fits(num_chunks, total_q, num_heads, max_blocks_per_seq, cache)) return PKV_ERR_UNSUPPORTED;
  if (num_chunks == 0 || total_q == 0) return PKV_OK;
  if (!out || !q || !cu_q_lens || !q_start_pos || !k_cache || !v_cache || !block_tables || max_blocks_per_seq == 0)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) || (reinterpret_cast<uintptr_t>(cu_q_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(q_start_pos) & 3u) || (reinterpret_cast<uintptr_t>(block_tables) & 3u))
    return PKV_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < pkv_chunk_workspace_bytes(total_q, num_heads, cache->num_kv_heads, cache->head_dim))
    return PKV_ERR_WORKSPACE;
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  ChunkParams prm;
  prm.out = static_cast<uint8_t*>(out);
  prm.lse = lse;
  prm.q = static_cast<const uint8_t*>(q);
  prm.cu_q = cu_q_lens;
  prm.start = q_start_pos;
  prm.tables = block_tables;
  prm.k_cache = static_cast<const uint8_t*>(k_cache);
  prm.v_cache = static_cast<const uint8_t*>(v_cache);
  prm.k_scale = cache->k_scale;
  prm.v_scale = cache->v_scale;
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
  const int64_t grid = (int64_t(total_q) * num_heads + 7) / 8;
  auto kern = q_dtype == PKV_BF16 ? (cache->head_dim == 128 ? chunk_kernel<true, 128> : chunk_kernel<true, 64>)
                                  : (cache->head_dim == 128 ? chunk_kernel<false, 128> : chunk_kernel<false, 64>);
  return launch_pdl(kern, dim3(unsigned(grid)), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), prm) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}
