// Device-side building blocks shared by the libpkv kernels (sm_103a): mbarriers with
// bounded waits, TMA tile loads, warp-level tensor-core fragments, fp8 conversion.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "f32x2.cuh"
#include "pkv.h"

namespace pkv {

// Bounded waits give up after this many nanoseconds of %globaltimer and report
// PKV_DEVERR_TIMEOUT instead of hanging the GPU.
constexpr uint64_t kWaitLimitNs = 1000000000ull;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t global_timer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ void set_error(unsigned* err, unsigned bits) {
  if (err) atomicOr(err, bits);
}

// ---------------------------------------------------------------------------------------
// mbarrier
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Non-blocking check of the phase with the given parity.  try_wait may hold the thread for
// a while when the phase is not complete; a thread that polls several barriers in turn
// uses this instead, so that a barrier that is not ready does not delay one that is.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Waits for the phase with the given parity to complete; false after limit_ns.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns = kWaitLimitNs) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (global_timer_ns() - t0 > limit_ns) return false;
  }
}

// ---------------------------------------------------------------------------------------
// Programmatic dependent launch: a kernel launched with programmatic stream serialization
// may start while its predecessor runs; griddep_wait() blocks until the predecessor has
// completed and its memory is visible.  Both are no-ops for ordinary launches.
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void griddep_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------------------------------
// TMA (tensor memory accelerator) tile loads
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ uint64_t l2_policy_evict_first() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

__device__ __forceinline__ uint64_t l2_policy_evict_last() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// 2-D tiled load of the box at (x, y) into shared memory; completion is signalled on `bar`
// as transaction bytes.  x must be a multiple of 16 bytes / element size.
__device__ __forceinline__ void tma_load_2d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "l"(policy)
      : "memory");
}

// 3-D tiled load (x innermost).
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y,
                                            int z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

// The same box, multicast: it lands at smem_dst's offset in every CTA of the cluster named in
// cta_mask, and each of those CTAs' mbarrier at bar's offset receives the complete_tx.
__device__ __forceinline__ void tma_load_3d_mc(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y,
                                               int z, uint16_t cta_mask, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.multicast::cluster"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6, %7;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "h"(cta_mask), "l"(policy)
      : "memory");
}

// Untiled copy of `bytes` (a multiple of 16; both addresses on 16 bytes) into shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::
          "r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(pol)
      : "memory");
}

__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Byte offset of 16-byte chunk `chunk` (0..7) of row `row` inside a box of 128-byte rows
// written by TMA with 128-byte swizzling (chunk index XOR row % 8).
__device__ __forceinline__ uint32_t swz128(int row, int chunk) {
  return uint32_t(row) * 128u + (uint32_t(chunk ^ (row & 7)) << 4);
}

// ---------------------------------------------------------------------------------------
// Warp-level tensor-core fragments (m16n8k16, fp32 accumulate)
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                              uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// D = A * B + C, A 16x16 (row), B 16x8 (col), fp32 accumulators.
template <bool kBF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kBF16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// Transpose of an 8x8 matrix of 16-bit values held one row-pair per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two fp32 values to two e4m3 codes (round to nearest even, saturate to +-448); lo -> low byte.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// 16 f16/bf16 values (a: elements 0-7, b: 8-15) to 16 e4m3 codes of x / scale, in element
// order.  The division is correctly rounded, so every writer of the cache agrees bit for bit.
template <bool kBF16>
__device__ __forceinline__ uint4 quant16_e4m3(const uint4 a, const uint4 b, float scale) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float2 lo, hi;
    if constexpr (kBF16) {
      lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[2 * k]));
      hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[2 * k + 1]));
    } else {
      lo = __half22float2(*reinterpret_cast<const __half2*>(&w[2 * k]));
      hi = __half22float2(*reinterpret_cast<const __half2*>(&w[2 * k + 1]));
    }
    r[k] = f32x2_to_e4m3x2(__fdiv_rn(lo.x, scale), __fdiv_rn(lo.y, scale)) |
           (f32x2_to_e4m3x2(__fdiv_rn(hi.x, scale), __fdiv_rn(hi.y, scale)) << 16);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Two e4m3 codes (low byte -> low half) to two fp16 values; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_codes) {
  uint32_t out;
  const unsigned short in = static_cast<unsigned short>(two_codes & 0xFFFFu);
  asm volatile("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(out) : "h"(in));
  return out;
}

// Eight e2m1 codes, two per byte (low nibble first), to four pairs of fp16 values; exact.
__device__ __forceinline__ void e2m1x8_to_f16x8(uint32_t codes, uint32_t (&out)[4]) {
  asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
      "mov.b32 {c0, c1, c2, c3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, c0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, c1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, c3;\n\t}"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(codes));
}

// Eight fp32 values to eight e2m1 codes (round to nearest even, saturate to +-6), v[0] in the
// lowest nibble.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n\t"
      "mov.b32 %0, {c0, c1, c2, c3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

template <bool kBF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (kBF16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery, "Division by invariant integers
// using multiplication", 1994): s = ceil(log2 d), m = floor(2^32 (2^s - d) / d) + 1.
struct Divisor {
  uint32_t d, m, s;
  explicit Divisor(int by) : d(uint32_t(by)), m(0), s(0) {
    while ((uint64_t(1) << s) < d) ++s;
    m = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return (__umulhi(m, n) + n) >> s; }
};

// In both halves of m: the value of larger magnitude of m and w, NaN if either is; its sign means nothing.
template <bool kBF16>
__device__ __forceinline__ void max_magnitudes(uint32_t& m, uint32_t w) {
  if constexpr (kBF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w));
  else asm("max.NaN.xorsign.abs.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w));
}

// -a / b for both halves, given y close to 1 / b: an estimate of the quotient corrected by its exact
// residual, kSteps times.  With y = 1 / b correctly rounded the second step gives the correctly rounded
// quotient (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990:
// the first makes the estimate faithful), barring overflow and underflow.  Negated, because
// a + (-a / b) b keeps the sign of a zero and a - (a / b) b does not.
template <int kSteps>
__device__ __forceinline__ uint64_t minus_div_f32x2(uint64_t a, uint64_t b, uint64_t minus_y) {
  uint64_t q = mul_f32x2(a, minus_y);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) q = fma_f32x2(fma_f32x2(q, b, a), minus_y, q);
  return q;
}
// The same for one value, not negated (a >= 0, two steps).
__device__ __forceinline__ float div_by(float a, float b, float y) {
  float q = a * y;
  q = fmaf(fmaf(-q, b, a), y, q);
  return fmaf(fmaf(-q, b, a), y, q);
}

// What quant16_e2m1 needs of a head's scale.
struct HeadScale {
  float scale, y;         // scale, 1 / scale correctly rounded
  bool given, ordinary;   // there is one; within 2^-80 .. 2^100 in absolute value
  __device__ __forceinline__ HeadScale(const float* scales, int h) {
    given = scales != nullptr;
    scale = given ? __ldg(scales + h) : 1.f;
    y = __frcp_rn(scale);
    ordinary = fabsf(scale) > 0x1p-80f && fabsf(scale) < 0x1p100f;
  }
};

// 16 f16/bf16 values (a: elements 0-7, b: 8-15) to the 16 codes of a 4-bit cache (8 bytes, element
// order) and their e4m3 scale: u = x / head scale, s = max|u| / 6 in e4m3, code = u / s in e2m1, all
// quotients correctly rounded fp32 by definition.  Every writer of the cache takes this function.
//   max|u| is the quotient of max|x|, rounding being monotonic.
//   u / s needs no correct rounding, only the right side of every border between codes (0.25, 0.75,
// 1.25, 1.75, 2.5, 3.5, 5; a tie has to stay one).  With 1 / s to 1 ulp the estimate is within 3 ulp, and
// one correction leaves an error below half an ulp and 3 * 2^-22 ulp: on a tie u = s * border it gives the
// border itself; off it, u is an fp32 value next to s * border or further (an fp32 value too: s has 4
// bits), so the quotient is at least 0.53 ulp away (s's significand is at most 1.875).
//   Elements too small for an exact residual (below 2^-100) become code 0 with any rounding, as the head
// scale is above 2^-80 and s at least 2^-9; huge elements and other head scales take the division
// instruction.
template <bool kBF16>
__device__ __forceinline__ uint2 quant16_e2m1(const uint4 a, const uint4 b, const HeadScale& hs, uint32_t& scale_code) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t m = w[0];                                         // max|x| of the low and the high halves, NaN if any is
#pragma unroll
  for (int k = 1; k < 8; ++k) max_magnitudes<kBF16>(m, w[k]);
  const float2 mm = unpack2<kBF16>(m & 0x7fff7fffu);
  bool nan = mm.x != mm.x || mm.y != mm.y;
  float mx = fmaxf(mm.x, mm.y);
  uint64_t u[8];                                             // x, or -x / head scale
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 f = unpack2<kBF16>(w[k]);
    u[k] = pack_f32x2(f.x, f.y);
  }
  if (nan) {                                                 // the maximum of the others, for the scale's definition
    mx = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fmaxf(fabsf(lo_f32(u[k])), fabsf(hi_f32(u[k]))));
  }
  if (hs.given) {
    if (hs.ordinary && mx < 0x1p100f && div_by(mx, fabsf(hs.scale), fabsf(hs.y)) < 0x1p100f) {
      mx = mx < 0x1p-100f ? 0.f : div_by(mx, fabsf(hs.scale), fabsf(hs.y));
#pragma unroll
      for (int k = 0; k < 8; ++k)
        u[k] = minus_div_f32x2<2>(u[k], pack_f32x2(hs.scale, hs.scale), pack_f32x2(-hs.y, -hs.y));
    } else {
      mx = __fdiv_rn(mx, fabsf(hs.scale));
      nan |= mx != mx;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float lo = __fdiv_rn(lo_f32(u[k]), hs.scale), hi = __fdiv_rn(hi_f32(u[k]), hs.scale);
        nan |= lo != lo || hi != hi;
        u[k] = pack_f32x2(-lo, -hi);
      }
    }
  }
  const float want = mx < 0x1p100f ? div_by(mx, 6.f, 1.f / 6.f) : 448.f;
  scale_code = f32x2_to_e4m3x2(fmaxf(want, 0x1p-9f), 0.f) & 0xFFu;   // 2^-9: the smallest e4m3 value
  const float s = unpack2<false>(e4m3x2_to_f16x2(scale_code)).x;
  if (nan) scale_code = 0x7Fu;
  if (!(mx < 0x1p100f)) {                                    // past 6 s in any case; keeps the residuals finite
#pragma unroll
    for (int k = 0; k < 8; ++k)
      u[k] = pack_f32x2(fminf(fmaxf(lo_f32(u[k]), -0x1p100f), 0x1p100f), fminf(fmaxf(hi_f32(u[k]), -0x1p100f), 0x1p100f));
  }
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
  float q[16];                                               // -x / s, or x / head scale / s
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint64_t c = minus_div_f32x2<1>(u[k], pack_f32x2(s, s), pack_f32x2(-y, -y));
    q[2 * k] = lo_f32(c);
    q[2 * k + 1] = hi_f32(c);
  }
  const float lo[8] = {q[0], q[1], q[2], q[3], q[4], q[5], q[6], q[7]};
  const float hi[8] = {q[8], q[9], q[10], q[11], q[12], q[13], q[14], q[15]};
  const uint32_t flip = hs.given ? 0u : 0x88888888u;         // the codes' sign bits
  return make_uint2(f32x8_to_e2m1x8(lo) ^ flip, f32x8_to_e2m1x8(hi) ^ flip);
}

// The ordinary case of it without branches, so that two of them overlap: false (and no result) where
// some element is not finite or huge, or the head's scale is odd.
template <bool kBF16, bool kScaled>
__device__ __forceinline__ bool quant16_e2m1_ordinary(const uint4 a, const uint4 b, const HeadScale& hs, uint2& codes,
                                                      uint32_t& scale_code) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t m[2] = {w[0], w[1]};
#pragma unroll
  for (int k = 2; k < 8; ++k) max_magnitudes<kBF16>(m[k & 1], w[k]);
  max_magnitudes<kBF16>(m[0], m[1]);
  const float2 mm = unpack2<kBF16>(m[0] & 0x7fff7fffu);
  bool ok = mm.x < 0x1p100f && mm.y < 0x1p100f;              // also no NaN
  float mx = fmaxf(mm.x, mm.y);
  if constexpr (kScaled) {
    const float q = div_by(mx, fabsf(hs.scale), fabsf(hs.y));
    ok = ok && hs.ordinary && q < 0x1p100f;
    mx = mx < 0x1p-100f ? 0.f : q;
  }
  scale_code = f32x2_to_e4m3x2(fmaxf(div_by(mx, 6.f, 1.f / 6.f), 0x1p-9f), 0.f) & 0xFFu;
  const float s = unpack2<false>(e4m3x2_to_f16x2(scale_code)).x;
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
  uint32_t c[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float q[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = unpack2<kBF16>(w[4 * half + k]);
      uint64_t u = pack_f32x2(f.x, f.y);
      if constexpr (kScaled) u = minus_div_f32x2<2>(u, pack_f32x2(hs.scale, hs.scale), pack_f32x2(-hs.y, -hs.y));
      u = minus_div_f32x2<1>(u, pack_f32x2(s, s), pack_f32x2(-y, -y));
      q[2 * k] = lo_f32(u);
      q[2 * k + 1] = hi_f32(u);
    }
    c[half] = f32x8_to_e2m1x8(q) ^ (kScaled ? 0u : 0x88888888u);
  }
  codes = make_uint2(c[0], c[1]);
  return ok;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

template <bool kBF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kBF16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  } else {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
}

// Product of two pairs of fp16 values.
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace pkv

// ---------------------------------------------------------------------------------------
// tcgen05 (5th-generation tensor cores) and tensor memory (TMEM)
// ---------------------------------------------------------------------------------------
namespace pkv {

// Shared-memory matrix descriptor, 128-byte swizzle.  `lbo` / `sbo` are byte offsets:
// K-major: sbo = stride between 8-row groups (1024 for dense 128-byte rows), lbo unused (16);
// MN-major: lbo = stride between 64-element column blocks, sbo = stride between 8-row groups.
__device__ __forceinline__ uint64_t umma_sdesc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= uint64_t((saddr >> 4) & 0x3FFFu);
  d |= uint64_t((lbo >> 4) & 0x3FFFu) << 16;
  d |= uint64_t((sbo >> 4) & 0x3FFFu) << 32;
  d |= uint64_t(1) << 46;                 // descriptor version for tcgen05
  d |= uint64_t(2) << 61;                 // 128-byte swizzle
  return d;
}

// Instruction descriptor of kind::f16 with fp32 accumulation.
__device__ __forceinline__ constexpr uint32_t umma_idesc_f16(bool bf16, int M, int N, bool a_mn_major,
                                                            bool b_mn_major) {
  return (1u << 4)                                  // D: f32
         | (uint32_t(bf16) << 7) | (uint32_t(bf16) << 10)   // A, B: bf16 (1) or f16 (0)
         | (uint32_t(a_mn_major) << 15) | (uint32_t(b_mn_major) << 16)
         | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ void umma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives (once) on `bar` when every tcgen05 op issued so far by this thread has completed.
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// Arrive (once the prior tcgen05 operations are done) on the mbarrier at bar's offset in every
// CTA of the cluster named in cta_mask.
__device__ __forceinline__ void umma_commit_mc(uint64_t* bar, uint16_t cta_mask) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               ::"r"(smem_u32(bar)), "h"(cta_mask)
               : "memory");
}

__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Every thread of every CTA in the cluster: arrive (release), then wait (acquire).
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t* smem_dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_dst)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
      "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
      "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])),
      "r"(__float_as_uint(v[11])), "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])),
      "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15])), "r"(__float_as_uint(v[16])),
      "r"(__float_as_uint(v[17])), "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])),
      "r"(__float_as_uint(v[20])), "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])),
      "r"(__float_as_uint(v[23])), "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])),
      "r"(__float_as_uint(v[26])), "r"(__float_as_uint(v[27])), "r"(__float_as_uint(v[28])),
      "r"(__float_as_uint(v[29])), "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31]))
      : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Brings the 128-byte line holding `p` into this SM's L1.
__device__ __forceinline__ void prefetch_l1(const void* p) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}

// 16-byte global -> shared copy that bypasses L1 (sees data other SMs wrote and fenced).
__device__ __forceinline__ void cp_async16_cg(uint32_t smem_addr, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr), "l"(gmem) : "memory");
}
// Waits for all of this thread's cp.async copies.
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

}  // namespace pkv

namespace pkv {
// D (TMEM) [+]= A (TMEM, K-major, two 16-bit values per column) x B (shared-memory descriptor).
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 consecutive 32-bit columns of this thread's TMEM lane, from raw words.
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
}  // namespace pkv

namespace pkv {
// Brings the box at (x, y) of a tensor map into L2 (no shared memory, no completion signal).
__device__ __forceinline__ void tma_prefetch_l2_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}
}  // namespace pkv
