// Paged decode over a 4-bit cache: the kernel behind pkv_paged_decode, _append and _noalloc for
// PKV_FP4_E2M1 pools.
//
// Mathematics: as paged_decode.cu (online softmax over a worker's range of 16-token tiles, partials
// merged by log-sum-exp), with K and V as code * scale of 16 elements * scale of the head.  code *
// scale is exact in fp16 (a 2-bit times a 4-bit significand, 2^-10 .. 2688), so the tensor cores
// multiply the stored values themselves; the head's k_scale goes into the softmax scale, its v_scale
// into the output.  P is rounded to fp16 for its product with V (2^-11 of each weight); the sum of the
// weights takes them unrounded.
//
// What bounds it: a 16-token tile of K and V is 18 * head_dim bytes, about 100 SM cycles at the
// measured copy bandwidth, while turning its 32 * head_dim codes into fp16 fragments takes
// head_dim / 2 conversions and as many multiplications per warp, a fixed ~170 instructions with the
// MMAs.  So the kernel has to keep everything else small:
//   * a warp takes up to 4 tiles (64 tokens) of a sequence per step: one wait, one softmax with its
//     shuffles, one refill per 64 tokens instead of per 16.  One tile per step took 463 instructions
//     per tile and ran at 3.1 TB/s;
//   * the tiles of a step are copied by as many lanes at once (a plain bulk copy each for K and V: a
//     4-bit tile is one contiguous run), 2 steps in flight per warp, 12 warps per SM;
//   * all query heads of a kv head (at most 8) share the converted fragments, K as the A operand
//     (S^T = K Q^T), V^T as the A operand (O^T += V^T P^T), as in paged_decode.cu.
//
// Fragment layouts.  Thread (g, t) = (lane / 4, lane % 4).  K: the thread reads elements D/4 t .. of
// rows g and g + 8 (one 16-byte load each at head_dim 128) and feeds 4 of them to each k step; Q is
// laid out to match.  V: it reads elements D/8 g .. of 4 tokens, which belong to one scale group per
// token; pairs of tokens are brought next to each other by merging nibbles.  A score row r stands
// for token row_token(r), so that the 4 V rows a warp reads at once differ modulo 4.
#include <type_traits>

#include "decode_split.cuh"

namespace pkv {
namespace {

constexpr int kSub = 4;                       // tiles per step

template <int D>
struct Fp4Cfg {
  static constexpr int kTileBytes = 9 * D;    // 16 x D/2 bytes of codes, 16 x D/16 scales
  static constexpr int kStageBytes = kSub * 2 * kTileBytes;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kKSteps = D / 16;
  static constexpr int kMTiles = D / 16;
  static constexpr int kGroups = D / 16;      // scale groups of a row
};

// Token of the tile that score row r (0..15) stands for.
__device__ __forceinline__ int row_token(int r) {
  return (r & 8) | ((r & 1) ? 7 - ((r & 7) >> 1) : (r & 7) >> 1);
}

// D += A * B (m16n8k16, fp16 in, fp32 out).  Not volatile, as the loads below are plain ones: the
// compiler may interleave the fragments of different tiles.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with D = A * B: the zero accumulator costs no registers to clear.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Two e4m3 codes (low byte -> low half) to two fp16 values; exact.
__device__ __forceinline__ uint32_t scales_f16x2(uint32_t two_codes) {
  uint32_t out;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(out) : "h"(static_cast<unsigned short>(two_codes)));
  return out;
}

// A pair of fp16 values times the low (high) half of s.
__device__ __forceinline__ uint32_t mul_lo(uint32_t x, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), __low2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul_hi(uint32_t x, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x), __high2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <bool kQBF16, int D, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, 1) paged_decode_fp4_kernel(const DecodeParams p) {
  using C = Fp4Cfg<D>;
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][kStages];
  __shared__ int warp_tot[kWarps * 2];

  const int S = p.num_seqs;
  const int Hkv = p.num_kv_heads;
  const int G = p.group;
  const int PB = p.part_blocks;
  int* cum_nb = reinterpret_cast<int*>(smem + kWarps * kStages * C::kStageBytes);   // [S + 1]
  int* cum_np = cum_nb + (S + 1);                                                    // [S + 1]
  int* lenc = cum_np + (S + 1);                                                      // [S] clamped lengths

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, tq = lane & 3;

  if (lane == 0) {
    for (int st = 0; st < kStages; ++st) mbar_init(&bars[warp][st], 1);
    fence_mbar_init();
  }

  // ---- prefix sums of tiles (and partitions) per sequence -------------------------------
  {
    const int per = (S + blockDim.x - 1) / blockDim.x;
    const int s0 = min(S, int(threadIdx.x) * per), s1 = min(S, s0 + per);
    int a = 0, u = 0;
    for (int s = s0; s < s1; ++s) {
      const int L = p.context_lens[s];
      const int Lc = clamp_len(L, p.max_len);
      if (Lc != L) set_error(p.err, PKV_DEVERR_CONTEXT_LEN);
      lenc[s] = Lc;
      const int nb = (Lc + kBS - 1) / kBS;
      a += nb;
      u += PB ? (nb + PB - 1) / PB : 0;
    }
    int ia = a, iu = u;   // inclusive warp scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int va = __shfl_up_sync(0xffffffffu, ia, o), vu = __shfl_up_sync(0xffffffffu, iu, o);
      if (lane >= o) { ia += va; iu += vu; }
    }
    if (lane == 31) { warp_tot[warp] = ia; warp_tot[kWarps + warp] = iu; }
    __syncthreads();
    int ba = 0, bu = 0;
    for (int w = 0; w < warp; ++w) { ba += warp_tot[w]; bu += warp_tot[kWarps + w]; }
    int ra = ba + ia - a, ru = bu + iu - u;   // exclusive prefix at s0
    for (int s = s0; s < s1; ++s) {
      const int nb = (lenc[s] + kBS - 1) / kBS;
      cum_nb[s] = ra;
      cum_np[s] = ru;
      ra += nb;
      ru += PB ? (nb + PB - 1) / PB : 0;
    }
    if (threadIdx.x == blockDim.x - 1) {
      int ta = 0, tu = 0;
      for (int w = 0; w < kWarps; ++w) { ta += warp_tot[w]; tu += warp_tot[kWarps + w]; }
      cum_nb[S] = ta;
      cum_np[S] = tu;
    }
  }
  __syncthreads();

  // Sequences with nothing to attend produce zeros (their tiles never exist).
  auto zero_empty = [&]() {
    for (int s = blockIdx.x; s < S; s += gridDim.x) {
      if (cum_nb[s + 1] != cum_nb[s]) continue;
      const int n = Hkv * G * D / 8;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + int64_t(s) * n * 16);
      for (int e = threadIdx.x; e < n; e += blockDim.x) dst[e] = make_uint4(0u, 0u, 0u, 0u);
    }
  };

  // Tile and unit counts stay below 2^31 (checked on the host).
  const int T = Hkv * cum_nb[S];
  const int U = Hkv * cum_np[S];
  const int nunits = PB ? U : T;
  const int W = PB ? min(p.num_workers, nunits) : workers_wide(nunits, p.num_workers, S * Hkv);
  const int w = warp * gridDim.x + blockIdx.x;   // a few workers get an SM each
  if (w >= W) {                              // no tiles for this warp
    griddep_wait();
    if (!p.defer_dependents) griddep_launch_dependents();
    zero_empty();
    return;
  }

  auto locate_in = [&](int t, int lo, int hi) -> Tile {
    Tile r;
    r.s = find_seq(cum_nb, lo, hi, t, Hkv);
    r.nb = cum_nb[r.s + 1] - cum_nb[r.s];
    const int off = t - Hkv * cum_nb[r.s];
    r.h = off / r.nb;
    r.b = off - r.h * r.nb;
    r.len = lenc[r.s];
    return r;
  };
  auto locate = [&](int t) -> Tile {         // whole warp, same t
    const int s = find_seq_warp(cum_nb, S, t, Hkv, lane);
    return locate_in(t, s, s);
  };
  // First tile of unit u (partition mode) in the flattened tile order; whole warp.
  auto unit_tile = [&](int u) -> int {
    if (u >= U) return T;
    const int s = find_seq_warp(cum_np, S, u, Hkv, lane);
    const int np = cum_np[s + 1] - cum_np[s];
    const int nb = cum_nb[s + 1] - cum_nb[s];
    const int off = u - Hkv * cum_np[s];
    const int h = off / np, part = off - h * np;
    return Hkv * cum_nb[s] + h * nb + part * PB;
  };
  // Worker wi starts at unit floor(wi * nunits / W), in 32 bits (see paged_decode.cu).
  const unsigned uq = unsigned(nunits) / unsigned(W), ur = unsigned(nunits) % unsigned(W);
  auto start_of = [&](int wi) -> int { return int(unsigned(wi) * uq + unsigned(wi) * ur / unsigned(W)); };
  const int t_begin = PB ? unit_tile(start_of(w)) : start_of(w);
  const int t_end = PB ? unit_tile(start_of(w + 1)) : start_of(w + 1);
  const int n = t_end - t_begin;
  const Tile first = locate(t_begin);
  const Tile last = locate(t_end - 1);

  uint8_t* my_stages = smem + warp * kStages * C::kStageBytes;
  const uint64_t pol = l2_policy_evict_first();

  // A step: the next tiles of one (sequence, kv head), at most kSub.
  auto step_tiles = [&](const Tile& c, int done) -> int { return min(min(kSub, c.nb - c.b), n - done); };
  // Moves a cursor past k tiles of its segment, to the next segment with tiles where that ends it.
  auto advance = [&](Tile& c, int k) {
    c.b += k;
    if (c.b < c.nb) return;
    c.b = 0;
    if (++c.h < Hkv) return;
    c.h = 0;
    do { ++c.s; } while (c.s < S && cum_nb[c.s + 1] == cum_nb[c.s]);
    if (c.s < S) {
      c.nb = cum_nb[c.s + 1] - cum_nb[c.s];
      c.len = lenc[c.s];
    }
  };

  // Block ids of the worker's tiles, 32 per window, loaded one window ahead.
  auto load_window = [&](int win) -> int {
    const int t = t_begin + win * 32 + lane;
    if (t >= t_end) return -1;
    const Tile c = locate_in(t, first.s, last.s);
    return p.block_tables[int64_t(c.s) * p.max_blocks + (c.b >> p.tile_shift)];
  };
  int win = 0;
  int bid_cur = load_window(0);
  int bid_nxt = n > 32 ? load_window(1) : -1;

  // Lane l's tile of the step of k tiles at cursor c, `done` tiles into the range: its index in the
  // pool in tiles, or -1 where the lane has none or the block id is outside the pool.
  auto tile_index = [&](const Tile& c, int done, int k) -> int {
    if ((done >> 5) > win) {
      bid_cur = bid_nxt;
      ++win;
      bid_nxt = load_window(win + 1);
    }
    const int j = done + (lane & (kSub - 1)) - (win << 5);     // up to kSub - 1 past the window
    const int a = __shfl_sync(0xffffffffu, bid_cur, j & 31), b = __shfl_sync(0xffffffffu, bid_nxt, j & 31);
    const int pb = j < 32 ? a : b;
    if (lane >= k) return -1;
    if (pb < 0 || pb >= p.num_blocks) {
      set_error(p.err, PKV_DEVERR_BLOCK_ID);
      return -1;
    }
    return int(((int64_t(pb) * Hkv + c.h) * p.block_size) / kBS) + ((c.b + lane) & ((1 << p.tile_shift) - 1));
  };
  // Starts the copies of a step into stage st; bit 4 st + l of `valid` says whether tile l came.
  uint32_t valid = 0;
  auto launch_step = [&](int index, int st) {
    uint64_t* bar = &bars[warp][st];
    const uint32_t have = __ballot_sync(0xffffffffu, index >= 0);
    valid = (valid & ~(0xFu << (4 * st))) | (have << (4 * st));
    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(have) * 2 * C::kTileBytes);
    __syncwarp();
    if (index >= 0) {
      uint8_t* dst = my_stages + st * C::kStageBytes + lane * 2 * C::kTileBytes;
      const int64_t off = int64_t(index) * C::kTileBytes;
      bulk_load(dst, static_cast<const uint8_t*>(p.k_cache) + off, C::kTileBytes, bar, pol);
      bulk_load(dst + C::kTileBytes, static_cast<const uint8_t*>(p.v_cache) + off, C::kTileBytes, bar, pol);
    }
  };

  // The first kStages steps' pool tiles, so that only the copies themselves follow the wait.
  Tile pc = first;                           // producer cursor
  int pdone = 0;                             // tiles before it
  int y0[kStages];
#pragma unroll
  for (int i = 0; i < kStages; ++i) {
    y0[i] = -1;
    if (pdone < n) {
      const int k = step_tiles(pc, pdone);
      y0[i] = tile_index(pc, pdone, k);
      pdone += k;
      if (pdone < n) advance(pc, k);
    }
  }

  // Up to here the kernel has read only lengths and block tables; the rest waits for the preceding
  // kernel on the stream (typically the KV write of this step).
  griddep_wait();
  if (!p.defer_dependents) griddep_launch_dependents();      // see paged_decode.cu
  {
    Tile c = first;
    int d = 0;
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      if (d < n) {
        launch_step(y0[i], i);
        const int k = step_tiles(c, d);
        d += k;
        if (d < n) advance(c, k);
      }
    }
  }
  zero_empty();

  // The query rows of the segment this range ends in are read late: bring them into L1.
  if (first.s != last.s || first.h != last.h) {
    const uint8_t* qrow0 = static_cast<const uint8_t*>(p.q) + (int64_t(last.s) * Hkv + last.h) * G * D * 2;
    for (int off = lane * 128; off < G * D * 2; off += 32 * 128) prefetch_l1(qrow0 + off);
  }

  Tile tl = first;                           // consumer cursor

  // Per-piece state.
  uint32_t qf[C::kKSteps][2];
  float o[C::kMTiles][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  uint64_t sl2 = 0;                          // softmax factors of heads 2t and 2t + 1
  int piece_b0 = 0;
  const int rt = row_token(gq);              // token of score row g (row g + 8: 8 more)

  int done = 0;
  for (int i = 0; done < n; ++i) {
    const int st = i % kStages;
    const int k = step_tiles(tl, done);
    if (done == 0 || tl.b == 0) {            // a piece starts
      piece_b0 = tl.b;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
#pragma unroll
      for (int mt = 0; mt < C::kMTiles; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
      const float sl = p.scale_log2 * (p.k_scale ? p.k_scale[tl.h] : 1.f);
      // The softmax takes max(s) * sl and -inf * sl, so sl has to be positive: its sign goes to the
      // queries, and 0 becomes the least normal number.
      const uint32_t flip = sl < 0.f ? 0x80008000u : 0u;
      auto positive = [](float v) -> float {                 // (NaN stays)
        return fabsf(v) < 1.17549435e-38f ? 1.17549435e-38f : fabsf(v);
      };
      const int64_t qrow = (int64_t(tl.s) * Hkv * G + int64_t(tl.h) * G + gq) * D + D / 4 * tq;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {     // 8 elements: two k steps
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (gq < G) v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.q) + 2 * (qrow + 8 * c));
        qf[2 * c][0] = v.x;
        qf[2 * c][1] = v.y;
        qf[2 * c + 1][0] = v.z;
        qf[2 * c + 1][1] = v.w;
      }
      if constexpr (!kQBF16) {
        sl2 = pack_f32x2(positive(sl), positive(sl));
#pragma unroll
        for (int c = 0; c < C::kKSteps; ++c) {
          qf[c][0] ^= flip;
          qf[c][1] ^= flip;
        }
      } else {
        // bf16 reaches further than fp16: each row goes into fp16 times the power of two that brings its largest
        // element to 2^14 .. 2^15, and the head's softmax factor takes the inverse.  Elements from 2^-31 of
        // the largest on stay exact, smaller ones are off by at most 2^-39 of it.  (Costs 0.4 us of 20.1 on 64
        // sequences of 128 to 2048 tokens, 28 heads over 4.)
        uint32_t m = 0u, m2 = 0u;
#pragma unroll
        for (int c = 0; c < C::kKSteps; ++c) {
          max_magnitudes<true>(m, qf[c][0]);
          max_magnitudes<true>(m2, qf[c][1]);
        }
        max_magnitudes<true>(m, m2);
        max_magnitudes<true>(m, __shfl_xor_sync(0xffffffffu, m, 1));
        max_magnitudes<true>(m, __shfl_xor_sync(0xffffffffu, m, 2));
        // The largest's biased exponent; from 15 to 254 both powers of two are normal numbers (a row of smaller
        // elements is exact at 15 as well).
        const int e = min(max(int(max(m & 0x7fffu, m >> 16 & 0x7fffu)) >> 7, 15), 254);
        const uint32_t down = (uint32_t(268 - e) * 0x00800080u) ^ flip;      // +-2^(141 - e), twice in bf16
        const float up = __int_as_float((e - 14) << 23);                     // 2^(e - 141)
#pragma unroll
        for (int c = 0; c < C::kKSteps; ++c) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(qf[c][i]) : "r"(down));
            const float2 f = unpack2<true>(qf[c][i]);
            qf[c][i] = pack2<false>(f.x, f.y);
          }
        }
        sl2 = pack_f32x2(positive(sl * __shfl_sync(0xffffffffu, up, 8 * tq)),
                         positive(sl * __shfl_sync(0xffffffffu, up, 8 * tq + 4)));
      }
    }
    const bool ends = tl.b + k == tl.nb;     // the step holds the segment's last tile

    // Fused append: lane l fetches 16 elements of the new token's row (K for the first kGroups lanes,
    // V for the next) while the tiles are still in flight.
    const bool app = p.k_new != nullptr && ends;
    uint4 na = make_uint4(0u, 0u, 0u, 0u), nb2 = na;
    int apb = -1, araw = -1;
    if (app) {
      araw = p.context_lens[tl.s];           // a clamped length has no new row to place
      apb = p.block_tables[int64_t(tl.s) * p.max_blocks + ((tl.len - 1) >> (4 + p.tile_shift))];
      if (lane < 2 * C::kGroups) {
        const uint4* src = static_cast<const uint4*>(lane < C::kGroups ? p.k_new : p.v_new) +
                           (int64_t(tl.s) * Hkv + tl.h) * (D / 8) + 2 * (lane % C::kGroups);
        na = src[0];
        nb2 = src[1];
      }
    }

    if (!mbar_wait(&bars[warp][st], uint32_t(i / kStages) & 1u)) {
      // Give up: report, then wait (bounded) for this warp's copies still in flight.
      if (lane == 0) set_error(p.err, PKV_DEVERR_TIMEOUT);
      for (int s2 = 1; s2 < kStages; ++s2)
        if (valid >> (4 * ((i + s2) % kStages)) & 0xFu)
          (void)mbar_wait(&bars[warp][(i + s2) % kStages], uint32_t((i + s2) / kStages) & 1u);
      return;
    }
    const uint32_t have = (valid >> (4 * st)) & 0xFu;
    uint8_t* stage = my_stages + st * C::kStageBytes;

    if (app && (have >> (k - 1) & 1u) && araw == tl.len) {
      // The new row goes into the staged tile and into the cache, at position len - 1.
      if (lane < 2 * C::kGroups) {
        const bool isv = lane >= C::kGroups;
        const int c = lane % C::kGroups, r = (tl.len - 1) & (kBS - 1);
        uint32_t sc;
        const uint2 v = quant16_e2m1<kQBF16>(na, nb2, HeadScale(isv ? p.v_scale : p.k_scale, tl.h), sc);
        const int at = r * (D / 2) + 8 * c, sat = 8 * D + r * C::kGroups + c;
        uint8_t* tile = stage + ((k - 1) * 2 + (isv ? 1 : 0)) * C::kTileBytes;
        *reinterpret_cast<uint2*>(tile + at) = v;
        tile[sat] = uint8_t(sc);
        fence_proxy_async_smem();            // orders these writes before the stage's next fill
        const int64_t row = (int64_t(apb) * Hkv + tl.h) * p.block_size + ((tl.len - 1) & (p.block_size - 1));
        uint8_t* pool = static_cast<uint8_t*>(isv ? p.v_cache : p.k_cache) + row / kBS * C::kTileBytes;
        *reinterpret_cast<uint2*>(pool + at) = v;
        pool[sat] = uint8_t(sc);
      }
      __syncwarp();
    }

    // ---- the step's tokens ------------------------------------------------------------------
    // Tokens of tile u that are attended (0: the tile is not part of the step, or did not come).
    auto tokens = [&](int u) -> int {
      return u < k && (have >> u & 1u) ? min(kBS, tl.len - (tl.b + u) * kBS) : 0;
    };
    // S^T = K Q^T of tile u: s[0]: (row g, head 2t)  s[1]: (row g, head 2t+1)  s[2]/s[3]: row g + 8.
    auto scores = [&](int u, float (&s)[4]) {
      const uint8_t* kb = stage + u * 2 * C::kTileBytes;
      uint32_t kw[2][D / 32], ks[2];         // codes; scales of the row's two groups here (D = 64: one)
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int row = rt + 8 * rr;
        if constexpr (D == 128) {
          const uint4 c = *reinterpret_cast<const uint4*>(kb + row * 64 + 16 * tq);
          kw[rr][0] = c.x; kw[rr][1] = c.y; kw[rr][2] = c.z; kw[rr][3] = c.w;
          ks[rr] = scales_f16x2(*reinterpret_cast<const uint16_t*>(kb + 8 * D + row * 8 + 2 * tq));
        } else {
          const uint2 c = *reinterpret_cast<const uint2*>(kb + row * 32 + 8 * tq);
          kw[rr][0] = c.x; kw[rr][1] = c.y;
          ks[rr] = scales_f16x2(kb[8 * D + row * 4 + tq]);
        }
      }
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {     // 8 elements of each row: two k steps
        uint32_t x[4], y[4];
        e2m1x8_to_f16x8(kw[0][c], x);
        e2m1x8_to_f16x8(kw[1][c], y);
        const bool hi = D == 128 && c >= 2;
        auto mul = [&](uint32_t v, uint32_t sc) { return hi ? mul_hi(v, sc) : mul_lo(v, sc); };
        const uint32_t a[4] = {mul(x[0], ks[0]), mul(y[0], ks[1]), mul(x[1], ks[0]), mul(y[1], ks[1])};
        if (c == 0) mma_f16_zero(s, a, qf[0][0], qf[0][1]);
        else mma_f16(s, a, qf[2 * c][0], qf[2 * c][1]);
        const uint32_t b[4] = {mul(x[2], ks[0]), mul(y[2], ks[1]), mul(x[3], ks[0]), mul(y[3], ks[1])};
        mma_f16(s, b, qf[2 * c + 1][0], qf[2 * c + 1][1]);
      }
    };
    // O^T += V^T P^T of tile u.  Tokens past nv contribute code 0 and scale 0, whatever their bytes.
    auto values = [&](int u, int nv, uint32_t pb0, uint32_t pb1, auto full) {
      const uint8_t* vb = stage + (u * 2 + 1) * C::kTileBytes;
      uint32_t vw[4][D / 64], sc[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {          // tokens of score rows 2t, 2t + 1, 2t + 8, 2t + 9
        const int vt = (x & 2 ? 8 : 0) + (x & 1 ? 7 - tq : tq);
        if constexpr (D == 128) {
          const uint2 c = *reinterpret_cast<const uint2*>(vb + vt * 64 + 8 * gq);
          vw[x][0] = c.x;
          vw[x][1] = c.y;
          sc[x] = vb[8 * D + vt * 8 + gq];
        } else {
          vw[x][0] = *reinterpret_cast<const uint32_t*>(vb + vt * 32 + 4 * gq);
          sc[x] = vb[8 * D + vt * 4 + (gq >> 1)];
        }
        if (!decltype(full)::value && vt >= nv) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) vw[x][c] = 0u;
          sc[x] = 0u;
        }
      }
      const uint32_t s01 = scales_f16x2(sc[0] | (sc[1] << 8)), s89 = scales_f16x2(sc[2] | (sc[3] << 8));
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {     // 8 elements: four m-tiles
        // Byte m: element 2m (e) / 2m + 1 (o) of the pair's first token (low nibble) and second.
        uint32_t e01[4], o01[4], e89[4], o89[4];
        e2m1x8_to_f16x8((vw[0][c] & 0x0F0F0F0Fu) | ((vw[1][c] << 4) & 0xF0F0F0F0u), e01);
        e2m1x8_to_f16x8(((vw[0][c] >> 4) & 0x0F0F0F0Fu) | (vw[1][c] & 0xF0F0F0F0u), o01);
        e2m1x8_to_f16x8((vw[2][c] & 0x0F0F0F0Fu) | ((vw[3][c] << 4) & 0xF0F0F0F0u), e89);
        e2m1x8_to_f16x8(((vw[2][c] >> 4) & 0x0F0F0F0Fu) | (vw[3][c] & 0xF0F0F0F0u), o89);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t a[4] = {hmul2(e01[m], s01), hmul2(o01[m], s01), hmul2(e89[m], s89), hmul2(o89[m], s89)};
          mma_f16(o[4 * c + m], a, pb0, pb1);
        }
      }
    };
    auto process = [&](auto full) {
      constexpr bool kFull = decltype(full)::value;
      float x[kSub][4];
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        if (kFull || tokens(u) > 0) {
          scores(u, x[u]);
          if (!kFull) {
            const int nv = tokens(u);
            if (rt >= nv) x[u][0] = x[u][1] = -INFINITY;
            if (rt + 8 >= nv) x[u][2] = x[u][3] = -INFINITY;
          }
        } else {
          x[u][0] = x[u][1] = x[u][2] = x[u][3] = -INFINITY;
        }
      }
      float mx0 = fmaxf(x[0][0], x[0][2]), mx1 = fmaxf(x[0][1], x[0][3]);
#pragma unroll
      for (int u = 1; u < kSub; ++u) {
        mx0 = fmaxf(mx0, fmaxf(x[u][0], x[u][2]));
        mx1 = fmaxf(mx1, fmaxf(x[u][1], x[u][3]));
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
      }
      const float mn0 = fmaxf(m0, mx0 * lo_f32(sl2)), mn1 = fmaxf(m1, mx1 * hi_f32(sl2));
      const bool grew = mn0 > m0 || mn1 > m1;
      const float al0 = fast_exp2(m0 - mn0), al1 = fast_exp2(m1 - mn1);
      m0 = mn0;
      m1 = mn1;
      uint64_t l2 = pack_f32x2(l0 * al0, l1 * al1);
      const uint64_t nm2 = pack_f32x2(-mn0, -mn1);
      uint32_t pb[kSub][2];
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const uint64_t ya = fma_f32x2(pack_f32x2(x[u][0], x[u][1]), sl2, nm2);
        const uint64_t yb = fma_f32x2(pack_f32x2(x[u][2], x[u][3]), sl2, nm2);
        const float p0 = fast_exp2(lo_f32(ya)), p1 = fast_exp2(hi_f32(ya));
        const float p2 = fast_exp2(lo_f32(yb)), p3 = fast_exp2(hi_f32(yb));
        l2 = add_f32x2(l2, add_f32x2(pack_f32x2(p0, p1), pack_f32x2(p2, p3)));
        // P^T as the B operand: lane (g, t) needs head g, score rows {2t, 2t+1} and {2t+8, 2t+9}.
        pb[u][0] = movmatrix_trans(pack2<false>(p0, p1));
        pb[u][1] = movmatrix_trans(pack2<false>(p2, p3));
      }
      l0 = lo_f32(l2);
      l1 = hi_f32(l2);
      if (__any_sync(0xffffffffu, grew)) {   // the running max moved: rescale O
#pragma unroll
        for (int mt = 0; mt < C::kMTiles; ++mt) {
          o[mt][0] *= al0; o[mt][1] *= al1; o[mt][2] *= al0; o[mt][3] *= al1;
        }
      }
#pragma unroll
      for (int u = 0; u < kSub; ++u)
        if (kFull || tokens(u) > 0) values(u, tokens(u), pb[u][0], pb[u][1], full);
    };
    if (k == kSub && have == 0xFu && tl.len >= (tl.b + kSub) * kBS) process(std::true_type{});
    else if (have) process(std::false_type{});

    // Release the stage and refill it.  Every lane's shared loads of this stage have returned (their
    // values fed the MMAs above), so the copies cannot overtake them.
    __syncwarp();
    if (pdone < n) {
      advance(pc, 0);
      const int pk = step_tiles(pc, pdone);
      launch_step(tile_index(pc, pdone, pk), st);
      pdone += pk;
      pc.b += pk;                            // the segment's end is passed when the next step starts
    } else {
      valid &= ~(0xFu << (4 * st));
    }

    done += k;
    if (!ends && done < n) {
      tl.b += k;
      continue;
    }
    // ---- finish the piece [piece_b0, tl.b + k) of segment (s, h) -----------------------------
    float ls0 = l0, ls1 = l1;
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      ls0 += __shfl_xor_sync(0xffffffffu, ls0, off);
      ls1 += __shfl_xor_sync(0xffffffffu, ls1, off);
    }
    const float vs = p.v_scale ? p.v_scale[tl.h] : 1.f;
    const int64_t seg_t0 = int64_t(Hkv) * cum_nb[tl.s] + int64_t(tl.h) * tl.nb;
    // Where the piece's result goes, by the rules that paged_decode.cu and the merge share.
    const bool complete = piece_b0 == 0 && ends;
    const float f0 = complete ? (ls0 == 0.f ? 0.f : vs / ls0) : vs, f1 = complete ? (ls1 == 0.f ? 0.f : vs / ls1) : vs;
    const int64_t slot = 2 * int64_t(w) + (seg_t0 + piece_b0 == t_begin ? 0 : 1);
    // Thread (g, t) holds elements D/8 g .. + D/8 - 1 of heads 2t and 2t + 1: element 2 mt + r is
    // o[mt][2 r] (head 2t) and o[mt][2 r + 1].
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int head = 2 * tq + hh;
      if (head >= G) break;
      const float f = hh ? f1 : f0;
      if (complete) {
        const int64_t at = ((int64_t(tl.s) * Hkv + tl.h) * G + head) * D + D / 8 * gq;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = pack2<kQBF16>(o[4 * c + e][hh] * f, o[4 * c + e][2 + hh] * f);
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + 2 * (at + 8 * c)) = make_uint4(v[0], v[1], v[2], v[3]);
        }
      } else {
        float* po = p.po + (slot * G + head) * D + D / 8 * gq;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          reinterpret_cast<float4*>(po)[c] = make_float4(o[2 * c][hh] * f, o[2 * c][2 + hh] * f, o[2 * c + 1][hh] * f,
                                                         o[2 * c + 1][2 + hh] * f);
        if (gq == 0) p.ml[slot * G + head] = make_float2(hh ? m1 : m0, hh ? ls1 : ls0);
      }
    }
    if (done < n) advance(tl, k);
  }
}

template <int D, int NW>
size_t smem_bytes(int num_seqs) {
  return size_t(NW) * Fp4Cfg<D>::kStages * Fp4Cfg<D>::kStageBytes + 3 * sizeof(int) * (size_t(num_seqs) + 1);
}

template <bool kQBF16, int D, int NW>
pkv_status launch_cfg(DecodeParams prm, int grid, cudaStream_t stream) {
  auto kern = paged_decode_fp4_kernel<kQBF16, D, NW>;
  const size_t smem = smem_bytes<D, NW>(prm.num_seqs);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess)
    return PKV_ERR_CUDA;
  prm.num_workers = grid * NW;
  if (launch_pdl(kern, dim3(grid), dim3(NW * 32), smem, stream, prm) != cudaSuccess) return PKV_ERR_CUDA;
  return launch_merge(prm, kQBF16, D, true, stream);
}

// 12 worker warps when the per-sequence prefix arrays (12 bytes each) fit next to their stages (18 KB per
// warp): up to about 900 sequences; else 8 (about 7,040) or 4 (about 13,180; more are refused).
template <bool kQBF16, int D>
pkv_status launch(const DecodeParams& prm, int grid, cudaStream_t stream) {
  static thread_local int cached_dev = -1;
  static thread_local size_t lim = 0;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  if (dev != cached_dev) {                   // looked up once per device and thread
    lim = dynamic_smem_limit(paged_decode_fp4_kernel<kQBF16, D, kMaxWarps>);
    cached_dev = dev;
  }
  if (smem_bytes<D, kMaxWarps>(prm.num_seqs) <= lim) return launch_cfg<kQBF16, D, kMaxWarps>(prm, grid, stream);
  if (smem_bytes<D, 8>(prm.num_seqs) <= lim) return launch_cfg<kQBF16, D, 8>(prm, grid, stream);
  if (smem_bytes<D, 4>(prm.num_seqs) <= lim) return launch_cfg<kQBF16, D, 4>(prm, grid, stream);
  return PKV_ERR_UNSUPPORTED;
}

}  // namespace

pkv_status launch_decode_fp4(DecodeParams prm, bool q_bf16, int head_dim, int grid, cudaStream_t stream) {
  if (head_dim == 128)
    return q_bf16 ? launch<true, 128>(prm, grid, stream) : launch<false, 128>(prm, grid, stream);
  return q_bf16 ? launch<true, 64>(prm, grid, stream) : launch<false, 64>(prm, grid, stream);
}

}  // namespace pkv
