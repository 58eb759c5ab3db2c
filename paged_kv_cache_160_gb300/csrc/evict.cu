// evict_select and evict_compact: which tokens of a sequence each kv head keeps, and their move to the front of
// the sequence's blocks.
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

// ---------------------------------------------------------------------------------------
// select
// ---------------------------------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMostPositions = 1 << 30;       // of a row: loops step past the end of one in 32 bits
constexpr int kDigits = 3;                    // of 11, 11 and 10 bits, from the top
constexpr int kBins = 2048;

struct SelectParams {
  int32_t* kept;
  const float* weights;
  const int32_t* rows;
  const int32_t* lens;
  const int32_t* keep;
  int max_keep, num_rows, max_len, num_kv_heads, first, recent;
  unsigned* err;
};

// Weights as unsigned numbers of the same order: -0 equals 0, NaN is below everything.
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// What lies at the place of `p` (shared memory) in the CTA of the given rank of the cluster.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t peer_word(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void add_to_peer(const void* p, uint32_t rank, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(peer_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A cluster of 1 to 8 CTAs per (sequence, kv head).  Every warp has a run of consecutive positions, so that
// counts and ballots alone give the order of the output.
//   The rank of the last one kept is found a digit at a time: each CTA counts its own positions' digits and
// adds the counts that are not zero to every CTA's totals.  (Reading all counts of all CTAs took 4 to 8
// thousand cycles a digit.  11 bits: the first digit holds the exponent and two bits of the mantissa, which
// spreads weights of similar size over several counters.)
//   kStored: the ranks stay in shared memory, one pass over the weights; else (longer rows) the weights are
// read again for each digit.
// Bound: launch, and three rounds of counting, a barrier and a scan.  Measured: 64 sequences of up to 2,048
// positions, 4 heads: 7.8 us (in rows of 131,072: 53, clusters of eight for what one CTA could do); 8 of 32K to 128K, 8
// heads: 39.6 us (512 CTAs of which 304 run at once; 58 us with the weights read again for each digit and
// twice the CTAs).  All weights equal: 7.9 and 35.7 us; all within a fifth of each other 7.8 and 46.2.
template <bool kStored>
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(const SelectParams p, int ctas) {
  extern __shared__ uint32_t ranks[];                        // [warp][run]
  __shared__ __align__(16) uint32_t hist[kBins], totals[kDigits][kBins];       // of this CTA (0 between digits); of the cluster
  __shared__ uint32_t warp_sum[kSelWarps], found[2];
  __shared__ uint32_t warp_above[kSelWarps], warp_equal[kSelWarps], cta_above, cta_equal;
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int job = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const int i = job / p.num_kv_heads, h = job % p.num_kv_heads;
  int32_t* kept = p.kept + int64_t(job) * p.max_keep;
  const int L = p.lens[i], want = p.keep[i], row = p.rows ? p.rows[i] : i;
  const int all_tid = rank * kSelThreads + tid, all_threads = ctas * kSelThreads;
  int n = 0;
  if (L < 0 || L > p.max_len || want < 0 || want > p.max_keep) {
    if (all_tid == 0) set_error(p.err, PKV_DEVERR_CONTEXT_LEN);
  } else if (row >= p.num_rows) {
    if (all_tid == 0) set_error(p.err, PKV_DEVERR_SLOT);
  } else if (row >= 0) {
    n = min(L, want);
  }
  const int r = min(p.recent, n), f = min(p.first, n - r), rest = n - r - f;
  for (int j = n + all_tid; j < p.max_keep; j += all_threads) kept[j] = -1;
  for (int j = all_tid; j < f; j += all_threads) kept[j] = j;
  for (int j = all_tid; j < r; j += all_threads) kept[n - r + j] = L - r + j;
  if (rest == 0) return;                                     // (the same for the whole cluster)
  const int lo = f, hi = L - r;
  if (rest == hi - lo) {
    for (int j = all_tid; j < rest; j += all_threads) kept[f + j] = lo + j;
    return;
  }
  const float* w = p.weights + (int64_t(row) * p.num_kv_heads + h) * p.max_len;
  // This warp's positions: run of them from `from` on, lane + 32 k.
  const int run = ((hi - lo + ctas * kSelWarps - 1) / (ctas * kSelWarps) + 31) & ~31;
  const int64_t from64 = lo + int64_t(rank * kSelWarps + warp) * run;
  const int from = int(min(from64, int64_t(hi))), to = int(min(from64 + run, int64_t(hi)));
  for (int b = tid; b < kDigits * kBins; b += kSelThreads) (&totals[0][0])[b] = 0;
  for (int b = tid; b < kBins; b += kSelThreads) hist[b] = 0;
  if (ctas > 1) cluster_arrive();
  uint32_t* mine = ranks + warp * run;
  if constexpr (kStored) {
#pragma unroll 8
    for (int j = from + lane; j < to; j += 32) mine[j - from] = rank_of(__ldg(w + j));
  }
  // Calls body(rank, there, position) for this thread's positions in ascending order; whole warps.
  auto each = [&](auto body) {
#pragma unroll 4
    for (int j = from + lane; j < to + lane; j += 32)
      body(j >= to ? 0u : kStored ? mine[j - from] : rank_of(__ldg(w + j)), j < to, j);
  };
  __syncthreads();
  uint32_t prefix = 0, need = rest;                          // the threshold's leading bits; how many from there on
#pragma unroll 1
  for (int d = 0; d < kDigits; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bits = d == 2 ? 10 : 11, bins = 1 << bits;
    each([&](uint32_t k, bool there, int) {
      if (there && (d == 0 || k >> (shift + bits) == prefix)) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
    });
    __syncthreads();
    if (ctas > 1) {
      if (d == 0) cluster_wait();                            // everyone's totals are zero
      for (int b = tid; b < bins; b += kSelThreads) {
        const uint32_t v = hist[b];
        if (v == 0) continue;
        hist[b] = 0;
        for (int q = 0; q < ctas; ++q) add_to_peer(&totals[d][b], q, v);
      }
      cluster_sync();
    }
    // Four bins a thread, from the top down: bins - 1 - 4 tid ...
    uint32_t c[4] = {0, 0, 0, 0}, sum = 0;
    if (4 * tid < bins) {
      uint32_t* at = &(ctas > 1 ? totals[d] : hist)[bins - 4 - 4 * tid];
      const uint4 v = *reinterpret_cast<const uint4*>(at);
      if (ctas == 1) *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
      c[0] = v.w;
      c[1] = v.z;
      c[2] = v.y;
      c[3] = v.x;
      sum = c[0] + c[1] + c[2] + c[3];
    }
    uint32_t before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    if (lane == 31) warp_sum[warp] = before;
    before -= sum;
    __syncthreads();
    for (int q = 0; q < warp; ++q) before += warp_sum[q];
    if (before < need && need <= before + sum) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (before < need && need <= before + c[u]) {
          found[0] = prefix << bits | uint32_t(bins - 1 - 4 * tid - u);
          found[1] = need - before;
        }
        before += c[u];
      }
    }
    __syncthreads();
    prefix = found[0];
    need = found[1];
    __syncthreads();
  }
  // prefix: the least rank kept; `need` of its holders, those of the lowest positions.
  uint32_t above = 0, equal = 0;                             // before this warp
  {
    uint32_t a = 0, e = 0;
    each([&](uint32_t k, bool there, int) {
      a += there && k > prefix;
      e += there && k == prefix;
    });
    a = __reduce_add_sync(0xffffffffu, a);
    e = __reduce_add_sync(0xffffffffu, e);
    if (lane == 0) {
      warp_above[warp] = a;
      warp_equal[warp] = e;
    }
    __syncthreads();
    uint32_t ta = 0, te = 0;
    for (int q = 0; q < kSelWarps; ++q) {
      if (q == warp) {
        above = ta;
        equal = te;
      }
      ta += warp_above[q];
      te += warp_equal[q];
    }
    if (ctas > 1) {
      if (tid == 0) {
        cta_above = ta;
        cta_equal = te;
      }
      cluster_sync();
      const bool before = lane < rank;                       // a lane for each of the CTAs before this one
      above += __reduce_add_sync(0xffffffffu, before ? peer_word(&cta_above, lane) : 0u);
      equal += __reduce_add_sync(0xffffffffu, before ? peer_word(&cta_equal, lane) : 0u);
    }
  }
  const unsigned below = (1u << lane) - 1;
  each([&](uint32_t k, bool there, int j) {
    const unsigned ma = __ballot_sync(0xffffffffu, there && k > prefix), me = __ballot_sync(0xffffffffu, there && k == prefix);
    const uint32_t na = above + __popc(ma & below), ne = equal + __popc(me & below);
    if (there && (k > prefix || (k == prefix && ne < need))) kept[f + na + min(ne, need)] = j;
    above += __popc(ma);
    equal += __popc(me);
  });
  if (ctas > 1) cluster_sync();                              // the others have read this CTA's counts
}

// ---------------------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kMoveAhead = 8;                 // pieces of a row that a thread has in flight
constexpr int kMoveRows = 512;                // rows of a round at most
constexpr int kMoveCtas = 4;                  // resident per SM

struct CompactParams {
  uint8_t* cache[2];
  const int32_t* kept;
  const int32_t* keep;
  const int32_t* src_tables;
  const int32_t* dst_tables;
  float* weights;
  const int32_t* rows;
  const int32_t* dst_rows;
  int max_keep, src_blocks, dst_blocks, num_rows, max_len, num_kv_heads, num_blocks, block_size, head_dim;
  int round_rows;         // rows that a CTA moves between two barriers
  Divisor pieces;         // of a row: 16 bytes each (8 where kUnit8), and in a 4-bit cache one more for its scales
  unsigned* err;
};

// A cluster of CTAs per (sequence, kv head) and K, V or the weights (blockIdx.y).
//   In place: kept positions ascend, so a row only ever moves to a lower position, and what a row at
// position d overwrites is needed by rows up to d alone.  A round reads the sources of consecutive
// destinations, all CTAs of the cluster meet, and then it writes; rounds ascend.  The next round's reads
// lie behind everything that this one writes.
// Bound: HBM, by reads and writes in flight: rows are `pieces` of 16 bytes, eight of them in flight per
// thread, and the next round's moves are looked up beside them.
// Measured: 512 rows of 64 sequences, 4 heads of 128 in bf16: 27.9 us, 0.68 of the measured copy; 8,192 of
// 3 sequences, 8 heads in e4m3, in clusters of 8: 27.5 us, 0.56.
template <bool kFp4, bool kUnit8>
__global__ void __launch_bounds__(kMoveThreads, kMoveCtas) compact_kernel(const CompactParams p, int ctas) {
  __shared__ int64_t src_at[2][kMoveRows], dst_at[2][kMoveRows];             // rows of the pool; -1: no move
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, job = blockIdx.x / ctas, rank = blockIdx.x % ctas, which = blockIdx.y;
  const int i = job / p.num_kv_heads, h = job % p.num_kv_heads;
  const int32_t* kept = p.kept + int64_t(job) * p.max_keep;
  const int n = p.keep[i];
  if (n < 0 || n > p.max_keep) {                             // (the same for the whole cluster)
    if (tid == 0) set_error(p.err, PKV_DEVERR_CONTEXT_LEN);
    return;
  }
  auto meet = [&]() {
    if (ctas > 1) cluster_sync(); else __syncthreads();
  };
  // Entry j of the list, or -1 where there is none or it does not ascend.
  auto entry = [&](int j) -> int {
    if (j >= n) return -1;
    const int q = __ldg(kept + j);
    if (q < 0) return -1;
    if (q < j || (j > 0 && __ldg(kept + j - 1) >= q)) {
      set_error(p.err, PKV_DEVERR_CHUNK);
      return -1;
    }
    return q;
  };
  if (which == 2) {
    const int from = p.rows ? p.rows[i] : i, to = p.dst_rows ? p.dst_rows[i] : from;
    if (from < 0 || to < 0) return;
    if (from >= p.num_rows || to >= p.num_rows) {
      if (tid == 0) set_error(p.err, PKV_DEVERR_SLOT);
      return;
    }
    const float* src = p.weights + (int64_t(from) * p.num_kv_heads + h) * p.max_len;
    float* dst = p.weights + (int64_t(to) * p.num_kv_heads + h) * p.max_len;
    constexpr int kStep = kMoveThreads * kMoveAhead;
    for (int j0 = rank * kStep; j0 - rank * kStep < n; j0 += ctas * kStep) {
      float v[kMoveAhead];
      bool on[kMoveAhead];
#pragma unroll
      for (int u = 0; u < kMoveAhead; ++u) {
        const int q = entry(j0 + u * kMoveThreads + tid);
        on[u] = q >= 0 && q < p.max_len;
        if (q >= p.max_len) set_error(p.err, PKV_DEVERR_CONTEXT_LEN);
        if (on[u]) v[u] = src[q];
      }
      meet();
#pragma unroll
      for (int u = 0; u < kMoveAhead; ++u)
        if (on[u]) dst[j0 + u * kMoveThreads + tid] = v[u];
    }
    return;
  }
  const int D = p.head_dim, R = p.round_rows;
  const int row_bytes = kFp4 ? D / 2 : int(p.pieces.d) * 16; // of codes
  auto place = [&](int64_t row) -> int64_t { return kFp4 ? (row >> 4) * 9 * D + (row & 15) * (D / 2) : row * row_bytes; };
  // The moves of the rows from j0 on.
  auto look_up = [&](int j0, int buf) {
    for (int t = tid; t < R; t += kMoveThreads) {
      const int j = j0 + t, q = entry(j);
      int64_t s = -1, d = -1;
      if (q >= 0) {
        if (q / p.block_size >= p.src_blocks || j / p.block_size >= p.dst_blocks) {
          set_error(p.err, PKV_DEVERR_CHUNK);
        } else {
          const int sb = __ldg(p.src_tables + int64_t(i) * p.src_blocks + q / p.block_size);
          const int db = __ldg(p.dst_tables + int64_t(i) * p.dst_blocks + j / p.block_size);
          if (unsigned(sb) >= unsigned(p.num_blocks) || unsigned(db) >= unsigned(p.num_blocks)) {
            set_error(p.err, PKV_DEVERR_BLOCK_ID);
          } else {
            s = (int64_t(sb) * p.num_kv_heads + h) * p.block_size + q % p.block_size;
            d = (int64_t(db) * p.num_kv_heads + h) * p.block_size + j % p.block_size;
            if (s == d) s = -1;                              // it stays
          }
        }
      }
      src_at[buf][t] = s;
      dst_at[buf][t] = d;
    }
  };
  auto scales = [&](int64_t row) -> int64_t { return (row >> 4) * 9 * D + 8 * D + (row & 15) * (D / 16); };
  uint8_t* cache = p.cache[which];
  const int pieces = int(p.pieces.d), work = R * pieces;
  look_up(rank * R, 0);
  __syncthreads();
  int buf = 0;
  for (int j0 = rank * R; j0 - rank * R < n; j0 += ctas * R, buf ^= 1) {
    uint4 v[kMoveAhead];
#pragma unroll
    for (int u = 0; u < kMoveAhead; ++u) {
      const int k = u * kMoveThreads + tid;
      if (k >= work) continue;
      const int t = int(p.pieces.quotient(k)), c = k - t * pieces;
      const int64_t s = src_at[buf][t];
      if (s < 0) continue;
      if (kFp4 && c == pieces - 1) {
        const uint8_t* sc = cache + scales(s);
        if (D == 128) {
          const uint2 x = *reinterpret_cast<const uint2*>(sc);
          v[u].x = x.x;
          v[u].y = x.y;
        } else if (D == 64) {
          v[u].x = *reinterpret_cast<const uint32_t*>(sc);
        } else {
          uint32_t x[4] = {0, 0, 0, 0};
          for (int b = 0; b < D / 16; ++b) x[b >> 2 & 3] |= uint32_t(sc[b]) << (8 * (b & 3));
          v[u] = make_uint4(x[0], x[1], x[2], x[3]);
        }
      } else if constexpr (kUnit8) {
        const uint2 x = *reinterpret_cast<const uint2*>(cache + place(s) + 8 * c);
        v[u].x = x.x;
        v[u].y = x.y;
      } else {
        v[u] = *reinterpret_cast<const uint4*>(cache + place(s) + 16 * c);
      }
    }
    if (j0 + ctas * R < n + rank * R) look_up(j0 + ctas * R, buf ^ 1);
    meet();
#pragma unroll
    for (int u = 0; u < kMoveAhead; ++u) {
      const int k = u * kMoveThreads + tid;
      if (k >= work) continue;
      const int t = int(p.pieces.quotient(k)), c = k - t * pieces;
      if (src_at[buf][t] < 0) continue;
      const int64_t d = dst_at[buf][t];
      if (kFp4 && c == pieces - 1) {
        uint8_t* sc = cache + scales(d);
        if (D == 128) {
          *reinterpret_cast<uint2*>(sc) = make_uint2(v[u].x, v[u].y);
        } else if (D == 64) {
          *reinterpret_cast<uint32_t*>(sc) = v[u].x;
        } else {
          const uint32_t x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
          for (int b = 0; b < D / 16; ++b) sc[b] = uint8_t(x[b >> 2 & 3] >> (8 * (b & 3)));
        }
      } else if constexpr (kUnit8) {
        *reinterpret_cast<uint2*>(cache + place(d) + 8 * c) = make_uint2(v[u].x, v[u].y);
      } else {
        *reinterpret_cast<uint4*>(cache + place(d) + 16 * c) = v[u];
      }
    }
    __syncthreads();                                         // the addresses just used may be overwritten
  }
}

// Launches `kern` with clusters of `ctas` along x, as a programmatic dependent.
template <typename... Params, typename... Args>
cudaError_t launch_clusters(void (*kern)(Params...), dim3 grid, int threads, int ctas, int smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, args...);
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
  if (int64_t(num_seqs) * num_kv_heads >= (int64_t(1) << 31) / kMaxCluster || max_keep > kMostPositions ||
      max_len > kMostPositions)
    return PKV_ERR_UNSUPPORTED;
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  SelectParams prm = {kept, weights, rows, context_lens, keep_lens, max_keep, num_rows, max_len, num_kv_heads, first, recent, err};
  // One CTA for up to 4096 positions, then up to eight, then more positions for each as far as two CTAs of an SM have
  // shared memory for their ranks.  The positions are those of a row, not of the sequences, which the host does not know.
  //   64 sequences x 4 heads of 4,096 positions: 9.1 us with one CTA each, 21.1 with two; 8,192: 23.7 with two, 12.4 with
  // one; 16,384: 43.8 with four, 18.8 with one.  8 x 8 of 16,384: 13.1 with four, 16.0 with two, 18.8 with one; 65,536: 34.8
  // with eight, 24.8 with four.  So 4,096 is right where the lists are few; many lists of 8K and more would rather have
  // one CTA each.
  //   Ranks stored or read again, 16,384 a CTA (8 x 8 of 131,072): 39.7 us and 73; 32,768 a CTA (262,144), where one CTA an
  // SM would have room: 144 stored, 197 as here.
  constexpr int kFew = 4096, kMost = 16384;
  int ctas = 1;
  while (ctas < kMaxCluster && int64_t(kFew) * ctas < max_len) ctas *= 2;
  const int64_t per_warp = (((int64_t(max_len) + ctas * kSelWarps - 1) / (ctas * kSelWarps)) + 31) / 32 * 32;
  const bool stored = per_warp * kSelWarps <= kMost;
  const int smem = stored ? int(per_warp) * kSelWarps * 4 : 0;
  auto kern = stored ? select_kernel<true> : select_kernel<false>;
  if (stored && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost * 4) != cudaSuccess) return PKV_ERR_CUDA;
  const int64_t jobs = int64_t(num_seqs) * num_kv_heads;
  return launch_clusters(kern, dim3(unsigned(jobs * ctas)), kSelThreads, ctas, smem, reinterpret_cast<cudaStream_t>(stream), prm, ctas) ==
                 cudaSuccess
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
  if (cache->head_dim % 16 || cache->head_dim > 256) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || max_keep == 0) return PKV_OK;
  if (!k_cache || !v_cache || !kept || !keep_lens || !src_tables || !dst_tables || src_max_blocks == 0 ||
      dst_max_blocks == 0 || (weights && (num_rows == 0 || max_len == 0)))
    return PKV_ERR_INVALID_ARG;
  // One cache as both would be moved by two CTAs at once.
  if (!aligned16(k_cache) || !aligned16(v_cache) || k_cache == v_cache) return PKV_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(kept), static_cast<const void*>(weights),
                        static_cast<const void*>(rows), static_cast<const void*>(dst_rows),
                        static_cast<const void*>(keep_lens), static_cast<const void*>(src_tables),
                        static_cast<const void*>(dst_tables)})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return PKV_ERR_INVALID_ARG;
  if (int64_t(num_seqs) * cache->num_kv_heads >= (int64_t(1) << 31) / kMaxCluster || max_keep > kMostPositions)
    return PKV_ERR_UNSUPPORTED;
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  const bool fp4 = cache->kv_dtype == PKV_FP4_E2M1;
  const int D = cache->head_dim, row_bytes = fp4 ? D / 2 : D * dtype_bytes(cache->kv_dtype);
  const bool unit8 = row_bytes % 16 != 0;                    // (4-bit rows of some head sizes)
  const int pieces = row_bytes / (unit8 ? 8 : 16) + (fp4 ? 1 : 0);
  CompactParams prm = {.pieces = Divisor(pieces)};
  prm.cache[0] = static_cast<uint8_t*>(k_cache);
  prm.cache[1] = static_cast<uint8_t*>(v_cache);
  prm.kept = kept;
  prm.keep = keep_lens;
  prm.src_tables = src_tables;
  prm.dst_tables = dst_tables;
  prm.weights = weights;
  prm.rows = rows;
  prm.dst_rows = dst_rows;
  prm.max_keep = max_keep;
  prm.src_blocks = src_max_blocks;
  prm.dst_blocks = dst_max_blocks;
  prm.num_rows = num_rows;
  prm.max_len = max_len;
  prm.num_kv_heads = cache->num_kv_heads;
  prm.num_blocks = cache->num_blocks;
  prm.block_size = cache->block_size;
  prm.head_dim = D;
  prm.round_rows = std::min(kMoveRows, kMoveThreads * kMoveAhead / pieces);
  prm.err = err;
  // More CTAs for a list while the lists alone do not fill the SMs and each CTA still has rows to move: up to half of the
  // CTAs that can be resident for K, and as many for V.  With one CTA a list 3 x 8 lists of 8,192 e4m3 rows take 112 us in
  // place of 27.5, 8 x 8 of 4,096 bf16 rows 127 in place of 60.5; 64 x 4 of 512 would take 24.9 in place of 27.8.  Half as
  // many: 54.0 for the 8 x 8, 24.9 for the 64 x 4, and 28.6 in place of 32.9 for 16 x 8 of 1,024; twice as many 33.1 for
  // the 64 x 4.
  const int64_t jobs = int64_t(num_seqs) * cache->num_kv_heads;
  int ctas = 1;
  while (ctas < kMaxCluster && 2 * jobs * ctas < int64_t(kMoveCtas) * std::max(1, num_sms()) && max_keep > ctas * prm.round_rows)
    ctas *= 2;
  auto kern = fp4 ? (unit8 ? compact_kernel<true, true> : compact_kernel<true, false>) : compact_kernel<false, false>;
  return launch_clusters(kern, dim3(unsigned(jobs * ctas), weights ? 3 : 2), kMoveThreads, ctas, 0,
                         reinterpret_cast<cudaStream_t>(stream), prm, ctas) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

}  // extern "C"
