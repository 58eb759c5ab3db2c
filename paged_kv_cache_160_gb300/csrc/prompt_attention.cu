// prompt_attention: causal attention of packed prompts over keys and values given as plain rows.
//
// Mathematics: row r of a sequence with Lq query and Lk key rows attends keys 0 .. r + Lk - Lq.  One
// pass over the keys in tiles of 128 with the running maximum m and sum l of the softmax (in units
// of log2): P = 2^(s c - m), O = O 2^(m_old - m) + P V, out = O / l.
//
// GB300 design: a CTA holds two row blocks of 128 query rows that read the same keys, so every K/V
// tile feeds 256 rows.  S = Q K^T and O += P V run on tcgen05 with S, P and O in tensor memory; Q, K
// and V arrive by TMA straight from the packed rows (any row stride).
#include "f32x2.cuh"
#include "pkv_device.cuh"
#include "pkv_host.h"

namespace pkv {
namespace {

constexpr int kTile = 128;                    // query rows of a block, keys of a tile
constexpr int kThreads = 576;
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
  int max_q_len;
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

// tcgen05 issued by a whole warp of which one lane (`lead` != 0) takes effect: control flow and operands
// stay uniform over the warp, so descriptors live in uniform registers.  Issued from a branch that only
// one lane takes, every product waited for its operands to be moved there: a prompt of 8192 tokens took
// 434 us instead of 392.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// One arrival on `bar` once every product issued so far is done.
__device__ __forceinline__ void commit(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}
// 1 in one lane of a converged warp, 0 in the others.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
  return r;
}

// ---------------------------------------------------------------------------------------
// A CTA holds two row blocks A and B of 128 query rows that read the same keys.
//   warp 0   : TMA producer of Q, K and V
//   warp 1   : TMEM owner and MMA issuer, in the order S_A(0) S_B(0) | PV_A(t) S_A(t+1) PV_B(t) S_B(t+1) | ...
//              so that one block's softmax overlaps the other's products
//   warps 2-9: softmax of block A, warps 10-17: of block B; two threads per query row, one for each half
//              of the tile's keys.  A tile's way from its scores to its product with V is a chain that
//              only the other block's products cover, so the softmax is spread over twice the threads:
//              one thread per row took 390 us for a prompt of 8192 tokens.
// ---------------------------------------------------------------------------------------
template <int D>
struct Cfg {
  static constexpr int kTileBytes = D / 64 * kHalfBytes;          // 128 rows of Q, K or V
  static constexpr int kStages = D == 128 ? 2 : 4;                // K and V tiles in flight
  static constexpr int kSmem = (2 + 2 * kStages) * kTileBytes;
};

template <bool kBF16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv, const PromptParams p) {
  using C = Cfg<D>;
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t bar_q, bar_k_full[kStages], bar_k_empty[kStages], bar_v_full[kStages],
      bar_v_empty[kStages], bar_s_full[2], bar_p_full[2], bar_pv_done[2];
  __shared__ uint32_t tmem_base_sh;
  __shared__ float exchange[2][2][2][kTile];                 // [block][tile parity][key half][row]
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform in the warp

  griddep_wait();
  // ---- the row blocks --------------------------------------------------------------------
  // A sequence's blocks of a kv head are numbered query tile by query tile, its query heads inside a
  // tile; a CTA takes the next two of them.  The hardware starts CTAs with x fastest and
  // z slowest: the last tiles, which walk the most keys, come first.
  const int seq = blockIdx.y, group = gridDim.z - 1 - blockIdx.z, h = blockIdx.x;
  const int G = p.num_heads / p.num_kv_heads;
  const int q0 = p.cu_q[seq], k0 = p.cu_k[seq];
  const int Lq = p.cu_q[seq + 1] - q0, Lk = p.cu_k[seq + 1] - k0;
  const bool bad = q0 < 0 || k0 < 0 || Lq < 0 || Lk < 0 || Lq > p.total_q - q0 || Lk > p.total_k - k0;
  if (threadIdx.x == 0 && blockIdx.z == 0 && blockIdx.x == 0 &&
      (bad || Lq > p.max_q_len || (seq == 0 && (q0 != 0 || k0 != 0))))
    set_error(p.err, PKV_DEVERR_CHUNK);
  const int rows = min(Lq, p.max_q_len);                     // rows past the promised bound stay unwritten
  if (bad || group * 2 >= (rows + kTile - 1) / kTile * G || (smem_u32(smem) & 1023u)) {
    if ((smem_u32(smem) & 1023u) && threadIdx.x == 0) set_error(p.err, PKV_DEVERR_CHUNK);
    griddep_launch_dependents();
    return;
  }
  const int shift = Lk - Lq;
  // First row and head of block e, and the key tiles its rows attend (0: none, or no such rows).
  auto first_row = [&](int e) -> int { return e / G * kTile; };
  auto head_of = [&](int e) -> int { return h * G + e % G; };
  auto tiles_of = [&](int e) -> int {
    const int r0 = first_row(e);
    if (r0 >= rows) return 0;
    const int keys = min(Lq, r0 + kTile) + shift;
    return keys > 0 ? (keys + kTile - 1) / kTile : 0;
  };
  const int e0 = 2 * group;                                  // A is block e0, B the next one
  const int na = tiles_of(e0), nb = tiles_of(e0 + 1), n = max(na, nb);

  uint8_t* sQ = smem;                                        // [block][64-dim half][128 rows]
  uint8_t* sK = smem + 2 * C::kTileBytes;                    // [stage][64-dim half][128 rows]
  uint8_t* sV = sK + kStages * C::kTileBytes;
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
      mbar_init(&bar_p_full[x], 8);                          // one arrival per softmax warp
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
      mbar_arrive_expect_tx(&bar_q, 2 * C::kTileBytes);
      for (int x = 0; x < 2; ++x) {
        // A block past the sequence's end reads rows that nobody stores: its own first ones.
        const int e = e0 + x, r0 = first_row(e) < rows ? first_row(e) : 0;
        for (int d = 0; d < D / 64; ++d)
          tma_load_3d(sQ + x * C::kTileBytes + d * kHalfBytes, &tmq, &bar_q, 64 * d, head_of(e), q0 + r0, pol_q);
      }
    }
    int t = 0;
    for (; ok && t < n; ++t) {
      const int st = t % kStages;
      const uint32_t par = uint32_t(t / kStages - 1) & 1u;
      if (t >= kStages && !(ok = mbar_wait(&bar_k_empty[st], par))) break;
      mbar_arrive_expect_tx(&bar_k_full[st], C::kTileBytes);
      for (int d = 0; d < D / 64; ++d)
        tma_load_3d(sK + st * C::kTileBytes + d * kHalfBytes, &tmk, &bar_k_full[st], 64 * d, h, k0 + t * kTile, pol_kv);
      if (t >= kStages && !(ok = mbar_wait(&bar_v_empty[st], par))) {
        (void)mbar_wait(&bar_k_full[st], uint32_t(t / kStages) & 1u);   // the K tile just started
        break;
      }
      mbar_arrive_expect_tx(&bar_v_full[st], C::kTileBytes);
      for (int d = 0; d < D / 64; ++d)
        tma_load_3d(sV + st * C::kTileBytes + d * kHalfBytes, &tmv, &bar_v_full[st], 64 * d, h, k0 + t * kTile, pol_kv);
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
  } else if (warp == 1) {
    // ---------------- MMA issuer (the whole warp; see mma_ss) ----------------
    const uint32_t lead = elect_one();
    const uint32_t idesc_s = umma_idesc_f16(kBF16, 128, 128, false, false);
    const uint32_t idesc_o = umma_idesc_f16(kBF16, 128, D, false, true);
    const uint64_t dQ = umma_sdesc_sw128(smem_u32(sQ), 16, 1024), dK = umma_sdesc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dV = umma_sdesc_sw128(smem_u32(sV), kHalfBytes, 1024);
    auto all = [](bool v) -> bool { return __all_sync(0xffffffffu, v); };
    bool ok = n == 0 || all(mbar_wait(&bar_q, 0));
    auto landed = [&](uint64_t* bar, int t) -> bool { return all(mbar_wait(bar, uint32_t(t / kStages) & 1u)); };
    // S_x(t) = Q_x K_t^T into TMEM columns 128x .. 128x + 127.  A descriptor advances by bytes / 16.
    auto issue_s = [&](int x, int t) -> bool {
      const int st = t % kStages;
      if (!landed(&bar_k_full[st], t)) return false;
      tc_fence_after();
      const uint64_t a = dQ + uint32_t(x * C::kTileBytes / 16), b = dK + uint32_t(st * C::kTileBytes / 16);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss(lead, tmem + 128 * x, a + ((kk >> 2) * kHalfBytes + (kk & 3) * 32) / 16,
                      b + ((kk >> 2) * kHalfBytes + (kk & 3) * 32) / 16, idesc_s, kk > 0);
      commit(lead, &bar_s_full[x]);
      return true;
    };
    // O_x += P_x(t) V_t; P_x of each half of the keys in the first 32 columns of that half's scores.
    auto issue_pv = [&](int x, int t) -> bool {
      const int st = t % kStages;
      if (!landed(&bar_v_full[st], t)) return false;         // (long before P)
      if (!all(mbar_wait(&bar_p_full[x], uint32_t(t) & 1u))) return false;
      tc_fence_after();
      const uint64_t b = dV + uint32_t(st * C::kTileBytes / 16);
#pragma unroll
      for (int kk = 0; kk < kTile / 16; ++kk)
        mma_ts(lead, tmem + 256 + 128 * x, tmem + 128 * x + (kk >> 2) * 64 + (kk & 3) * 8, b + kk * 2048 / 16, idesc_o, t > 0 || kk > 0);
      commit(lead, &bar_pv_done[x]);
      return true;
    };
    // One block may walk fewer tiles than the other.  A stage is released once both have read it.
    if (ok && n > 0) {
      ok = (na == 0 || issue_s(0, 0)) && (nb == 0 || issue_s(1, 0));
      commit(lead, &bar_k_empty[0]);
    }
    for (int t = 0; ok && t < n; ++t) {
      if (t < na) ok = issue_pv(0, t);
      if (ok && t + 1 < na) ok = issue_s(0, t + 1);
      if (ok && t < nb) ok = issue_pv(1, t);
      commit(lead, &bar_v_empty[t % kStages]);
      if (ok && t + 1 < nb) ok = issue_s(1, t + 1);
      if (t + 1 < n) commit(lead, &bar_k_empty[(t + 1) % kStages]);
    }
    if (!ok && lane == 0) set_error(p.err, PKV_DEVERR_TIMEOUT);
  } else if (warp >= 2) {
    // ---------------- softmax: two threads per query row ----------------
    const int x = (warp - 2) >> 3, hf = ((warp - 2) >> 2) & 1;   // row block; half of the keys (and of O)
    const int quarter = warp & 3, r = 32 * quarter + lane;   // TMEM lane == row of the block
    const uint32_t lane_off = uint32_t(32 * quarter) << 16;
    const int e = e0 + x;
    const int row = first_row(e) + r;
    const int nx = x == 0 ? na : nb;
    constexpr int kKeys = kTile / 2, kODims = D / 2;
    const float slog = p.scale_log2;                         // > 0, so max(s) * slog = max(s * slog)
    const uint32_t tS = tmem + 128 * x + lane_off + kKeys * hf;   // scores, and P over them
    const uint32_t tO = tmem + 256 + 128 * x + lane_off + kODims * hf;
    // The two warps of a row quarter meet here, once per tile and once at the end, also after a wait
    // gave up: then they only walk on, so that neither is left waiting for the other.
    auto meet = [&]() {
      asm volatile("bar.sync %0, 64;" ::"r"(1 + 4 * x + quarter) : "memory");
    };
    float m = -INFINITY, l = 0.f;                            // m of the row, l of this thread's keys
    bool ok = true;
    for (int t = 0; t < nx; ++t) {
      // Waiting for PV(t - 1) on every tile keeps that barrier at most one phase ahead of this wait.
      ok = __all_sync(0xffffffffu, ok && mbar_wait(&bar_s_full[x], uint32_t(t) & 1u) &&
                                       (t == 0 || mbar_wait(&bar_pv_done[x], uint32_t(t - 1) & 1u)));
      if (!ok) {
        meet();
        continue;
      }
      tc_fence_after();
      const int lim = min(row + shift + 1, Lk) - t * kTile - kKeys * hf;   // keys 0 .. lim - 1 are attended
      float s[kKeys];
#pragma unroll
      for (int cc = 0; cc < kKeys / 32; ++cc) tmem_ld32(tS + 32 * cc, *reinterpret_cast<float(*)[32]>(s + 32 * cc));
      tmem_wait_ld();
      if (lim < kKeys) {
#pragma unroll
        for (int i = 0; i < kKeys; ++i) s[i] = i < lim ? s[i] : -INFINITY;
      }
      float mine;
      {
        float c4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < kKeys; i += 8) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (i + 2 * u + 1 < kKeys) c4[u] = fmax3(c4[u], s[i + 2 * u], s[i + 2 * u + 1]);
        }
        mine = fmaxf(fmaxf(c4[0], c4[1]), fmaxf(c4[2], c4[3]));
      }
      float* xm = &exchange[x][t & 1][0][r];
      xm[kTile * hf] = mine;
      meet();
      const float mt = fmaxf(mine, xm[kTile * (hf ^ 1)]) * slog;
      const bool grow = mt > m + kRescaleThreshold;          // also true for the first tile
      const float m_prev = m;
      if (grow) m = mt;
      // The sequence's last tile may reach past its keys: zero those V rows, so that 0 * whatever
      // the rows behind hold cannot turn into NaN (both blocks write the same zeros).
      const int kb = t * kTile;
      if (kb + kTile > Lk) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bar_v_full[t % kStages], uint32_t(t / kStages) & 1u));
        if (!ok) continue;
        if (kb + r >= Lk) {
          const uint32_t vrow = smem_u32(sV + (t % kStages) * C::kTileBytes) + r * 128;
#pragma unroll
          for (int d = 0; d < D / 64; ++d)
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) sts128(vrow + d * kHalfBytes + (4 * hf + cc) * 16, 0u, 0u, 0u, 0u);
        }
      }
      // P over S (keys 2e, 2e + 1 in column e).  A row without keys so far has m = -inf and every
      // s = -inf: m = 0 then gives P = 0.
      const float mu = m == -INFINITY ? 0.f : m;
      const uint64_t sl2 = pack_f32x2(slog, slog), nm2 = pack_f32x2(-mu, -mu);
      uint64_t acc0 = pack_f32x2(0.f, 0.f), acc1 = acc0;
#pragma unroll
      for (int hb = 0; hb < kKeys / 32; ++hb) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c0 = 32 * hb + 2 * i;
          const uint64_t x2 = fma_f32x2(pack_f32x2(s[c0], s[c0 + 1]), sl2, nm2);
          const float pa = fast_exp2(lo_f32(x2)), pb = fast_exp2(hi_f32(x2));
          const uint64_t p2 = pack_f32x2(pa, pb);
          if (i & 1) acc1 = add_f32x2(acc1, p2);
          else acc0 = add_f32x2(acc0, p2);
          w[i] = pack2<kBF16>(pa, pb);
        }
        tmem_st16u(tS + 16 * hb, w);
      }
      const uint64_t acc = add_f32x2(acc0, acc1);
      const float lsum = lo_f32(acc) + hi_f32(acc);
      if (__any_sync(0xffffffffu, grow && t >= 1)) {         // rescale this thread's half of O
        const float alpha = (grow && m_prev != -INFINITY) ? fast_exp2(m_prev - m) : 1.f;
#pragma unroll
        for (int cc = 0; cc < kODims / 32; ++cc) {
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
    if (nx == 0 && n > 0) ok = mbar_wait(&bar_q, 0);         // the output is staged where Q lands
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0) set_error(p.err, PKV_DEVERR_TIMEOUT);
    tc_fence_after();
    // ---------------- output ----------------
    // Every product that reads this block's Q is done: its area stages the warp's 32 half rows of
    // 16-bit values, 16-byte chunk c of a row at c ^ (row mod chunks) against bank conflicts, and the
    // warp writes runs of whole half rows.
    exchange[x][nx & 1][hf][r] = l;                          // tile nx - 1 used the other parity
    meet();
    if (ok && first_row(e) + 32 * quarter < rows) {
      constexpr int kRowBytes = D, kChunks = D / 16;         // of a half row
      l += exchange[x][nx & 1][hf ^ 1][r];
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const uint32_t stage = smem_u32(sQ) + x * C::kTileBytes + (hf * 4 + quarter) * 32 * kRowBytes;
#pragma unroll
      for (int cc = 0; cc < kODims / 32; ++cc) {
        float v[32];
        if (nx > 0) {
          tmem_ld32(tO + 32 * cc, v);
          tmem_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 4 * cc + i;
          const uint32_t at = stage + lane * kRowBytes + ((c ^ (lane & (kChunks - 1))) << 4);
          if (l > 0.f)
            sts128(at, pack2<kBF16>(v[8 * i] * inv, v[8 * i + 1] * inv),
                   pack2<kBF16>(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                   pack2<kBF16>(v[8 * i + 4] * inv, v[8 * i + 5] * inv),
                   pack2<kBF16>(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
          else
            sts128(at, 0u, 0u, 0u, 0u);
        }
      }
      __syncwarp();
      uint8_t* dst = p.out + (int64_t(q0) * p.out_stride + int64_t(head_of(e)) * D + kODims * hf) * 2;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int i = 32 * k + lane, rr = i / kChunks, c = i % kChunks;
        const uint4 val = lds128(stage + rr * kRowBytes + ((c ^ (rr & (kChunks - 1))) << 4));
        const int orow = first_row(e) + 32 * quarter + rr;
        if (orow < rows) reinterpret_cast<uint4*>(dst + orow * p.out_stride * 2)[c] = val;
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
  using C = Cfg<D>;
  auto kern = prompt_kernel<kBF16, D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
    return PKV_ERR_CUDA;
  const unsigned groups = (unsigned((max_q_len - 1) / kTile + 1) * unsigned(prm.num_heads / prm.num_kv_heads) + 1) / 2;
  const dim3 grid(prm.num_kv_heads, num_seqs, groups);
  return launch_pdl(kern, grid, dim3(kThreads), C::kSmem, stream, tq, tk, tv, prm) == cudaSuccess ? PKV_OK
                                                                                                  : PKV_ERR_CUDA;
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
  if (num_seqs > 65535 || num_heads > 65535) return PKV_ERR_UNSUPPORTED;
  // The row blocks of a sequence's kv head, two to a CTA, fill one grid dimension.
  if ((int64_t((int64_t(max_q_len) + kTile - 1) / kTile) * (num_heads / num_kv_heads) + 1) / 2 > 65535)
    return PKV_ERR_UNSUPPORTED;
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
                          uint64_t(head_dim) * 2, uint64_t(stride) * 2, 64, 1, kTile,
                          CU_TENSOR_MAP_SWIZZLE_128B);
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
  prm.max_q_len = max_q_len;
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
