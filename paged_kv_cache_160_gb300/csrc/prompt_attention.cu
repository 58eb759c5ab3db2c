// prompt_attention: causal attention of packed prompts over keys and values given as plain rows.
//
// Mathematics: row r of a sequence with Lq query and Lk key rows attends keys 0 .. r + Lk - Lq.  One
// pass over the keys in tiles of 128 with the running maximum m and sum l of the softmax (in units
// of log2): P = 2^(s c - m), O = O 2^(m_old - m) + P V, out = O / l.
//
// GB300 design: a CTA holds two row blocks A and B of 128 query rows that read the same keys, so
// every K/V tile feeds 256 rows: two query heads of a kv head where the group has two left, else two
// adjacent query tiles of one head.  S = Q K^T and O += P V run on tcgen05 with S, P and O in tensor
// memory; Q, K and V arrive by TMA straight from the packed rows (any row stride).
#include "f32x2.cuh"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kTile = 128;                    // query rows of a block, keys of a tile
constexpr int kThreads = 320;
constexpr int kStages = 2;                    // K and V tiles in flight
constexpr uint32_t kTmemCols = 512;           // S_A | S_B | O_A | O_B, 128 columns each
constexpr int kHalfBytes = kTile * 128;       // [128 rows][64 elements] of 2 bytes
constexpr float kRescaleThreshold = 8.f;      // log2 units

struct PromptParams {
  uint8_t* out;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int64_t out_stride;     // elements
  int total_q;
  int total_k;
  int num_heads;
  int num_kv_heads;
  float scale_log2;
  unsigned* err;
};

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Three-input maximum (one instruction on this architecture).
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

//   warp 0   : TMA producer
//   warp 1   : TMEM owner and MMA issuer, in the order S_A(0) S_B(0) | PV_A(t) S_A(t+1) PV_B(t) S_B(t+1) | ...
//   warps 2-5: softmax of block A, warps 6-9: of block B; one query row per thread
template <bool kBF16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv, const PromptParams p) {
  constexpr int kTileBytes = D / 64 * kHalfBytes;            // one 128 x D operand
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t bar_q, bar_k_full[kStages], bar_k_empty[kStages], bar_v_full[kStages],
      bar_v_empty[kStages], bar_s_full[2], bar_p_full[2], bar_pv_done[2];
  __shared__ uint32_t tmem_base_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  griddep_wait();
  // ---- the CTA's two row blocks --------------------------------------------------------
  // The hardware starts CTAs with x fastest and z slowest: the last query tiles, which walk the most
  // keys, come first.
  const int seq = blockIdx.y, qt = gridDim.z - 1 - blockIdx.z;
  const int G = p.num_heads / p.num_kv_heads, slots = (G + 1) / 2;
  const int h = blockIdx.x / slots, sl = blockIdx.x % slots;
  const bool qpair = 2 * sl + 1 >= G;                        // the group's odd head: two query tiles
  const int q0 = p.cu_q[seq], k0 = p.cu_k[seq];
  const int Lq = p.cu_q[seq + 1] - q0, Lk = p.cu_k[seq + 1] - k0;
  const bool bad = q0 < 0 || k0 < 0 || Lq < 0 || Lk < 0 || Lq > p.total_q - q0 || Lk > p.total_k - k0;
  if (threadIdx.x == 0 && qt == int(gridDim.z) - 1 && blockIdx.x == 0 &&
      (bad || Lq > int(gridDim.z) * kTile || (seq == 0 && (q0 != 0 || k0 != 0))))
    set_error(p.err, PKV_DEVERR_CHUNK);
  if (bad || qt * kTile >= Lq || (qpair && (qt & 1)) || (smem_u32(smem) & 1023u)) {
    if ((smem_u32(smem) & 1023u) && threadIdx.x == 0) set_error(p.err, PKV_DEVERR_CHUNK);
    griddep_launch_dependents();
    return;
  }
  const int ra = qt * kTile, rb = qpair ? ra + kTile : ra;   // first query rows of A and B
  const int ha = h * G + 2 * sl, hb = qpair ? ha : ha + 1;
  const int shift = Lk - Lq;
  // Key tiles that the rows of a block starting at r0 attend (0: none, or no such rows).
  auto tiles_of = [&](int r0) -> int {
    if (r0 >= Lq) return 0;
    const int keys = min(Lq, r0 + kTile) + shift;
    return keys > 0 ? (keys + kTile - 1) / kTile : 0;
  };
  const int na = tiles_of(ra), nb = tiles_of(rb), n = max(na, nb);

  uint8_t* sQ = smem;                                        // [block][64-dim half][128 rows]
  uint8_t* sK = smem + 2 * kTileBytes;
  uint8_t* sV = smem + (2 + kStages) * kTileBytes;
  if (threadIdx.x == 0) {
    mbar_init(&bar_q, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar_k_full[i], 1);
      mbar_init(&bar_k_empty[i], 1);
      mbar_init(&bar_v_full[i], 1);
      mbar_init(&bar_v_empty[i], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bar_s_full[x], 1);
      mbar_init(&bar_p_full[x], 4);                          // one arrival per softmax warp
      mbar_init(&bar_pv_done[x], 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;

  if (warp == 0 && lane == 0) {
    // ---------------- TMA producer ----------------
    const uint64_t pol_q = l2_policy_evict_first();
    const uint64_t pol_kv = l2_policy_evict_last();          // re-read by the other heads and query tiles
    bool ok = true;
    if (n > 0) {
      mbar_arrive_expect_tx(&bar_q, 2 * kTileBytes);
      for (int d = 0; d < D / 64; ++d) {
        tma_load_3d(sQ + d * kHalfBytes, &tmq, &bar_q, 64 * d, ha, q0 + ra, pol_q);
        // A missing second query tile loads the first once more (its rows are computed by nobody).
        tma_load_3d(sQ + kTileBytes + d * kHalfBytes, &tmq, &bar_q, 64 * d, hb, q0 + (nb > 0 ? rb : ra), pol_q);
      }
    }
    int t = 0;
    for (; ok && t < n; ++t) {
      const int st = t % kStages;
      const uint32_t par = uint32_t(t / kStages - 1) & 1u;
      if (t >= kStages && !(ok = mbar_wait(&bar_k_empty[st], par))) break;
      mbar_arrive_expect_tx(&bar_k_full[st], kTileBytes);
      for (int d = 0; d < D / 64; ++d)
        tma_load_3d(sK + st * kTileBytes + d * kHalfBytes, &tmk, &bar_k_full[st], 64 * d, h, k0 + t * kTile, pol_kv);
      if (t >= kStages && !(ok = mbar_wait(&bar_v_empty[st], par))) {
        (void)mbar_wait(&bar_k_full[st], uint32_t(t / kStages) & 1u);   // the K tile just started
        break;
      }
      mbar_arrive_expect_tx(&bar_v_full[st], kTileBytes);
      for (int d = 0; d < D / 64; ++d)
        tma_load_3d(sV + st * kTileBytes + d * kHalfBytes, &tmv, &bar_v_full[st], 64 * d, h, k0 + t * kTile, pol_kv);
    }
    // Drain: the last loads of each stage have landed and the commits that release the stages have
    // arrived before the CTA may leave (each wait bounded).
    if (!ok) {
      set_error(p.err, PKV_DEVERR_TIMEOUT);
      (void)mbar_wait(&bar_q, 0);
    }
    for (int u = max(0, t - kStages); u < t; ++u) {
      const int st = u % kStages;
      const uint32_t par = uint32_t(u / kStages) & 1u;
      (void)mbar_wait(&bar_k_full[st], par);
      (void)mbar_wait(&bar_v_full[st], par);
      if (ok) ok = mbar_wait(&bar_k_empty[st], par) && mbar_wait(&bar_v_empty[st], par);
    }
  } else if (warp == 1 && lane == 0) {
    // ---------------- MMA issuer ----------------
    const uint32_t idesc_s = umma_idesc_f16(kBF16, 128, 128, false, false);
    const uint32_t idesc_o = umma_idesc_f16(kBF16, 128, D, false, true);
    const uint32_t aQ = smem_u32(sQ), aK = smem_u32(sK), aV = smem_u32(sV);
    bool ok = n == 0 || mbar_wait(&bar_q, 0);
    // S_x(t) = Q_x K_t^T into TMEM columns 128x .. 128x + 127.
    auto issue_s = [&](int x, int t) -> bool {
      const int st = t % kStages;
      if (!mbar_wait(&bar_k_full[st], uint32_t(t / kStages) & 1u)) return false;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
        umma_f16(tmem + 128 * x, umma_sdesc_sw128(aQ + x * kTileBytes + off, 16, 1024),
                 umma_sdesc_sw128(aK + st * kTileBytes + off, 16, 1024), idesc_s, kk > 0);
      }
      umma_commit(&bar_s_full[x]);
      return true;
    };
    // O_x += P_x(t) V_t, P_x in the first 64 columns of S_x.
    auto issue_pv = [&](int x, int t) -> bool {
      const int st = t % kStages;
      if (!mbar_wait(&bar_p_full[x], uint32_t(t) & 1u)) return false;
      if (!mbar_wait(&bar_v_full[st], uint32_t(t / kStages) & 1u)) return false;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < kTile / 16; ++kk)
        umma_f16_ts(tmem + 256 + 128 * x, tmem + 128 * x + 8 * kk,
                    umma_sdesc_sw128(aV + st * kTileBytes + kk * 2048, kHalfBytes, 1024), idesc_o, t > 0 || kk > 0);
      umma_commit(&bar_pv_done[x]);
      return true;
    };
    // One block may walk fewer tiles than the other.  A stage is released once both have read it.
    if (ok && n > 0) {
      ok = (na == 0 || issue_s(0, 0)) && (nb == 0 || issue_s(1, 0));
      umma_commit(&bar_k_empty[0]);
    }
    for (int t = 0; ok && t < n; ++t) {
      if (t < na) ok = issue_pv(0, t);
      if (ok && t + 1 < na) ok = issue_s(0, t + 1);
      if (ok && t < nb) ok = issue_pv(1, t);
      umma_commit(&bar_v_empty[t % kStages]);
      if (ok && t + 1 < nb) ok = issue_s(1, t + 1);
      if (t + 1 < n) umma_commit(&bar_k_empty[(t + 1) % kStages]);
    }
    if (!ok) set_error(p.err, PKV_DEVERR_TIMEOUT);
  } else if (warp >= 2) {
    // ---------------- softmax: one query row per thread ----------------
    const int x = (warp - 2) >> 2;                           // row block
    const int r = 32 * (warp & 3) + lane;                    // TMEM lane == row of the block
    const uint32_t lane_off = uint32_t(32 * (warp & 3)) << 16;
    const int row = (x == 0 ? ra : rb) + r;
    const int nx = x == 0 ? na : nb;
    const float slog = p.scale_log2;                         // > 0, so max(s) * slog = max(s * slog)
    const uint32_t tS = tmem + 128 * x + lane_off, tO = tmem + 256 + 128 * x + lane_off;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int t = 0; t < nx; ++t) {
      if (!(ok = mbar_wait(&bar_s_full[x], uint32_t(t) & 1u))) break;
      // Waiting for PV(t - 1) on every tile keeps that barrier at most one phase ahead of this wait.
      if (t >= 1 && !(ok = mbar_wait(&bar_pv_done[x], uint32_t(t - 1) & 1u))) break;
      __syncwarp();
      tc_fence_after();
      const int lim = min(row + shift + 1, Lk) - t * kTile;  // keys 0 .. lim - 1 of the tile are attended
      float s[kTile];
#pragma unroll
      for (int cc = 0; cc < kTile / 32; ++cc) tmem_ld32(tS + 32 * cc, *reinterpret_cast<float(*)[32]>(s + 32 * cc));
      tmem_wait_ld();
      if (lim < kTile) {
#pragma unroll
        for (int i = 0; i < kTile; ++i) s[i] = i < lim ? s[i] : -INFINITY;
      }
      float mraw;
      {
        float c4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < kTile; i += 8) {
#pragma unroll
          for (int u = 0; u < 4; ++u) c4[u] = fmax3(c4[u], s[i + 2 * u], s[i + 2 * u + 1]);
        }
        mraw = fmaxf(fmaxf(c4[0], c4[1]), fmaxf(c4[2], c4[3]));
      }
      const float mt = mraw * slog;
      const bool grow = mt > m + kRescaleThreshold;          // also true for the first tile
      const float m_prev = m;
      if (grow) m = mt;
      // The sequence's last tile may reach past its keys: zero those V rows, so that 0 * whatever
      // the rows behind hold cannot turn into NaN (both blocks write the same zeros).
      const int kb = t * kTile;
      if (kb + kTile > Lk) {
        if (!(ok = mbar_wait(&bar_v_full[t % kStages], uint32_t(t / kStages) & 1u))) break;
        if (kb + r >= Lk) {
          const uint32_t vrow = smem_u32(sV + (t % kStages) * kTileBytes) + r * 128;
#pragma unroll
          for (int d = 0; d < D / 64; ++d)
#pragma unroll
            for (int cc = 0; cc < 8; ++cc) sts128(vrow + d * kHalfBytes + cc * 16, 0u, 0u, 0u, 0u);
        }
      }
      // P over S (keys 2e, 2e + 1 in column e).  A row without keys so far has m = -inf and every
      // s = -inf: m = 0 then gives P = 0.
      const float mu = m == -INFINITY ? 0.f : m;
      const uint64_t sl2 = pack_f32x2(slog, slog), nm2 = pack_f32x2(-mu, -mu);
      uint64_t acc0 = pack_f32x2(0.f, 0.f), acc1 = acc0;
#pragma unroll
      for (int hb4 = 0; hb4 < 4; ++hb4) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int c0 = 32 * hb4 + 2 * e;
          const uint64_t x2 = fma_f32x2(pack_f32x2(s[c0], s[c0 + 1]), sl2, nm2);
          const float pa = fast_exp2(lo_f32(x2)), pb = fast_exp2(hi_f32(x2));
          const uint64_t p2 = pack_f32x2(pa, pb);
          if (e & 1) acc1 = add_f32x2(acc1, p2);
          else acc0 = add_f32x2(acc0, p2);
          w[e] = pack2<kBF16>(pa, pb);
        }
        tmem_st16u(tS + 16 * hb4, w);
      }
      const uint64_t acc = add_f32x2(acc0, acc1);
      const float lsum = lo_f32(acc) + hi_f32(acc);
      if (__any_sync(0xffffffffu, grow && t >= 1)) {
        const float alpha = (grow && m_prev != -INFINITY) ? fast_exp2(m_prev - m) : 1.f;
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          float v[32];
          tmem_ld32(tO + 32 * cc, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] *= alpha;
          tmem_st32(tO + 32 * cc, v);
        }
        if (grow) l *= alpha;
      }
      tmem_wait_st();
      l += lsum;
      if (kb + kTile > Lk) fence_proxy_async_smem();         // the zeroed V rows, to the tensor cores
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_p_full[x]);
    }
    if (ok && nx > 0) ok = mbar_wait(&bar_pv_done[x], uint32_t(nx - 1) & 1u);
    if (!ok && r == 0) set_error(p.err, PKV_DEVERR_TIMEOUT);
    __syncwarp();
    tc_fence_after();
    // ---------------- output ----------------
    const int first = x == 0 ? ra : rb;
    if (ok && first < Lq) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int hq = x == 0 ? ha : hb;
      uint4* dst = reinterpret_cast<uint4*>(p.out + ((int64_t(q0) + row) * p.out_stride + int64_t(hq) * D) * 2);
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        float v[32];
        if (nx > 0) {
          tmem_ld32(tO + 32 * cc, v);
          tmem_wait_ld();
        }
        if (row < Lq) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint4 o = make_uint4(0u, 0u, 0u, 0u);
            if (l > 0.f)
              o = make_uint4(pack2<kBF16>(v[i] * inv, v[i + 1] * inv), pack2<kBF16>(v[i + 2] * inv, v[i + 3] * inv),
                             pack2<kBF16>(v[i + 4] * inv, v[i + 5] * inv), pack2<kBF16>(v[i + 6] * inv, v[i + 7] * inv));
            dst[4 * cc + i / 8] = o;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  griddep_launch_dependents();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool kBF16, int D>
pkv_status launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PromptParams& prm,
                  int num_seqs, int max_q_len, cudaStream_t stream) {
  auto kern = prompt_kernel<kBF16, D>;
  constexpr int smem = (2 + 2 * kStages) * (D / 64) * kHalfBytes;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return PKV_ERR_CUDA;
  const int G = prm.num_heads / prm.num_kv_heads;
  const dim3 grid(prm.num_kv_heads * ((G + 1) / 2), num_seqs, (max_q_len - 1) / kTile + 1);
  return launch_pdl(kern, grid, dim3(kThreads), smem, stream, tq, tk, tv, prm) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_prompt_attention(void* out, const void* q, const void* k, const void* v, pkv_dtype dtype,
                                           const int32_t* cu_q_lens, const int32_t* cu_k_lens, int num_seqs,
                                           int total_q, int total_k, int max_q_len, int num_heads, int num_kv_heads,
                                           int head_dim, int64_t out_stride, int64_t q_stride, int64_t k_stride,
                                           int64_t v_stride, float scale, pkv_stream_t stream) {
  using namespace pkv;
  if (num_seqs < 0 || total_q < 0 || total_k < 0 || max_q_len < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
      head_dim <= 0 || num_heads % num_kv_heads)
    return PKV_ERR_INVALID_ARG;
  if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
  if (!(scale > 0.f)) return PKV_ERR_INVALID_ARG;            // the softmax takes max(s) * scale
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || num_heads > 65535 || (max_q_len - 1) / kTile + 1 > 65535) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || total_q == 0 || max_q_len == 0) return PKV_OK;
  if (!out || !q || !cu_q_lens || !cu_k_lens || (total_k > 0 && (!k || !v))) return PKV_ERR_INVALID_ARG;
  auto bad_rows = [&](const void* t, int64_t stride, int heads) {
    return !aligned16(t) || stride % 8 || stride < int64_t(heads) * head_dim;
  };
  if (bad_rows(out, out_stride, num_heads) || bad_rows(q, q_stride, num_heads) || bad_rows(k, k_stride, num_kv_heads) ||
      bad_rows(v, v_stride, num_kv_heads) || (reinterpret_cast<uintptr_t>(cu_q_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(cu_k_lens) & 3u))
    return PKV_ERR_INVALID_ARG;
  const int64_t kMaxStride = int64_t(1) << 38;               // a tensor map's strides end at 2^40 bytes
  if (q_stride >= kMaxStride || k_stride >= kMaxStride || v_stride >= kMaxStride) return PKV_ERR_UNSUPPORTED;
  if (!on_current_device(q) || (total_k > 0 && (!on_current_device(k) || !on_current_device(v))))
    return PKV_ERR_INVALID_ARG;
  unsigned* err = error_word_ptr();
  if (!err) return PKV_ERR_CUDA;
  // Rows as (dims, heads, rows): a box is 64 dims of one head of 128 rows.
  auto encode = [&](CUtensorMap* m, const void* base, int heads, int rows, int64_t stride) {
    return encode_tmap_3d(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, base, uint64_t(head_dim), uint64_t(heads), uint64_t(rows),
                          uint64_t(head_dim) * 2, uint64_t(stride) * 2, 64, 1, kTile, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  CUtensorMap tq, tk = {}, tv = {};
  if (!encode(&tq, q, num_heads, total_q, q_stride)) return PKV_ERR_CUDA;
  if (total_k > 0 && (!encode(&tk, k, num_kv_heads, total_k, k_stride) || !encode(&tv, v, num_kv_heads, total_k, v_stride)))
    return PKV_ERR_CUDA;
  PromptParams prm;
  prm.out = static_cast<uint8_t*>(out);
  prm.cu_q = cu_q_lens;
  prm.cu_k = cu_k_lens;
  prm.out_stride = out_stride;
  prm.total_q = total_q;
  prm.total_k = total_k;
  prm.num_heads = num_heads;
  prm.num_kv_heads = num_kv_heads;
  prm.scale_log2 = scale * 1.4426950408889634f;
  prm.err = err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == PKV_BF16)
    return head_dim == 128 ? launch<true, 128>(tq, tk, tv, prm, num_seqs, max_q_len, s)
                           : launch<true, 64>(tq, tk, tv, prm, num_seqs, max_q_len, s);
  return head_dim == 128 ? launch<false, 128>(tq, tk, tv, prm, num_seqs, max_q_len, s)
                         : launch<false, 64>(tq, tk, tv, prm, num_seqs, max_q_len, s);
}
