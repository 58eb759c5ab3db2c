// Tiles of 128 keys of a paged cache, and blocks of 128 query rows, as operands of the tensor cores: 16-bit
// rows in shared memory, [64-element half][128 rows] of 128 bytes each with the 128-byte swizzle.
//
// e4m3 and 4-bit rows are turned into fp16, which holds code * scale of their 16 exactly; the kv head's
// scale is applied to scores and outputs.  Their queries are then fp16 too: bf16 rows are multiplied by a
// power of two that brings their largest element to 2^14 .. 2^15, taken back with the scale of the scores.
#pragma once

#include "cache_row.cuh"
#include "pkv_host.h"

namespace pkv {

constexpr int kTile = 128;                    // keys of a tile, query rows of a block
constexpr int kHalfBytes = kTile * 128;

// The cache of a call, as its kernels see it.
struct PagedCache {
  const int32_t* tables;
  int max_blocks, num_blocks, num_kv_heads, block_size;
  int block_shift;                            // log2(block_size)
  unsigned* err;
};

// 128-byte swizzled place of 16-byte chunk c8 (of the row's D / 8) of row `row`.
__device__ __forceinline__ uint32_t operand_at(uint32_t base, int row, int c8) {
  return base + (c8 >> 3) * kHalfBytes + swz128(row, c8 & 7);
}

// 16 bytes, or zeros where `on` is not set; no branch.
__device__ __forceinline__ uint4 ld_stream(const void* p, bool on) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
      "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}\n"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"(int(on)));
  return v;
}
__device__ __forceinline__ uint32_t ld_16(const void* p, bool on) {
  uint16_t v;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.u16 %0, 0;\n\t@p ld.global.nc.u16 %0, [%1];\n\t}\n"
               : "=&h"(v)
               : "l"(p), "r"(int(on)));
  return v;
}

// A warp's window on a block table: lane i holds entry 32 w + i.
struct TableWindow {
  const int32_t* table;
  int entries;                                // entries that may be read
  int at;                                     // the window w held, -1: none
  int32_t cur, next;

  __device__ __forceinline__ void open(const int32_t* t, int n) {
    table = t;
    entries = n;
    at = -1;
  }
  __device__ __forceinline__ int32_t fetch(int w, int lane) const {
    const int i = 32 * w + lane;
    return i < entries ? __ldg(table + i) : -1;
  }
  // Makes window w the current one; the one after it is on its way.
  __device__ __forceinline__ void move(int w, int lane) {
    if (w == at) return;
    cur = at >= 0 && w == at + 1 ? next : fetch(w, lane);
    next = fetch(w + 1, lane);
    at = w;
  }
  __device__ __forceinline__ int32_t entry(int i) const { return __shfl_sync(0xffffffffu, cur, i & 31); }
};

// The stored rows of a tile on their way to shared memory: 16 bytes per thread and pass, 128 threads.
//   A warp's lanes are spread so that its loads cover whole rows and 8 lanes that store together hit 8 different
// 16-byte columns: 8 rows of one chunk, or for 128-byte rows 4 rows of chunks c and c + 4.
template <int KV, int D>
struct StoredTile {
  static constexpr bool kFp4 = KV == PKV_FP4_E2M1;
  static constexpr int kLanes = (kFp4 ? D / 2 : D) / 16;     // of a row
  static constexpr int kPasses = kLanes;                     // 128 threads, 128 / kLanes rows each
  static constexpr int kPassRows = kTile / kLanes;
  uint4 code[kPasses];
  uint32_t scale[kFp4 ? kPasses : 1];

  static __device__ __forceinline__ int sub(int lane) {
    if constexpr (kLanes == 8) return (lane >> 4) << 2 | ((lane >> 2) & 1) << 1 | ((lane >> 3) & 1);
    else if constexpr (kLanes == 4) return lane >> 3;
    else return (lane >> 3) & 1;
  }
  static __device__ __forceinline__ int row(int warp, int lane, int pass) {   // warp 0 .. 3
    const int r = kLanes == 8 ? lane & 3 : kLanes == 4 ? lane & 7 : (lane & 7) + 8 * (lane >> 4);
    return pass * kPassRows + warp * (kPassRows / 4) + r;
  }

  // Keys 128 tile .. of kv head h; keys from `end` on become zeros, as do those of blocks outside the pool.
  __device__ __forceinline__ void load(const uint8_t* cache, const PagedCache& pc, TableWindow& win, int h, int tile,
                                       int end, int warp, int lane) {
    const int per_window = pc.block_shift + 5 - 7;           // log2 of the tiles in a window
    win.move(tile >> per_window, lane);
    const int s = sub(lane), j0 = tile * kTile + row(warp, lane, 0);
    int blk[kPasses];
    bool missing = false;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) blk[p] = win.entry((j0 + p * kPassRows) >> pc.block_shift);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int j = j0 + p * kPassRows;
      const bool there = unsigned(blk[p]) < unsigned(pc.num_blocks), on = j < end && there;
      missing |= j < end && !there;
      const int64_t at = (int64_t(blk[p]) * pc.num_kv_heads + h) * pc.block_size + (j & (pc.block_size - 1));
      if constexpr (kFp4) {
        const uint8_t* t = cache + (at >> 4) * (9 * D);
        const int rr = int(at & 15);
        code[p] = ld_stream(t + rr * (D / 2) + 16 * s, on);
        scale[p] = ld_16(t + 8 * D + rr * (D / 16) + 2 * s, on);
      } else {
        code[p] = ld_stream(cache + at * D + 16 * s, on);
      }
    }
    if (missing) set_error(pc.err, PKV_DEVERR_BLOCK_ID);
  }

  // A row for each lane, of the 32 that its warp stores.
  static __device__ __forceinline__ int row_of_lane(int warp, int lane) {
    return lane / (kPassRows / 4) * kPassRows + warp * (kPassRows / 4) + lane % (kPassRows / 4);
  }

  // As fp16 to the operand at `base`.
  __device__ __forceinline__ void store(uint32_t base, int warp, int lane) const {
    const int s = sub(lane);
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int r = row(warp, lane, p);
      const uint32_t w[4] = {code[p].x, code[p].y, code[p].z, code[p].w};
      constexpr int kChunks = kFp4 ? 4 : 2;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint32_t o[4];
        if constexpr (kFp4) {
          const uint32_t sc = (scale[p] >> (c & 2 ? 8 : 0)) & 0xFFu, s2 = e4m3x2_to_f16x2(sc * 0x101u);
          e2m1x8_to_f16x8(w[c], o);
#pragma unroll
          for (int k = 0; k < 4; ++k) o[k] = hmul2(o[k], s2);
        } else {
          o[0] = e4m3x2_to_f16x2(w[2 * c]);
          o[1] = e4m3x2_to_f16x2(w[2 * c] >> 16);
          o[2] = e4m3x2_to_f16x2(w[2 * c + 1]);
          o[3] = e4m3x2_to_f16x2(w[2 * c + 1] >> 16);
        }
        sts128(operand_at(base, r, kChunks * s + c), o[0], o[1], o[2], o[3]);
      }
    }
  }
};

// A 16-bit tile by TMA, 16 rows at a time, issued by one lane: boxes of 64 elements by 16 rows of the pool's rows.
// Rows from `end` on (in whole 16s) and those of blocks outside the pool become zeros.  All lanes call it.
template <int D>
__device__ __forceinline__ void load_tile_16bit(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, const PagedCache& pc,
                                                TableWindow& win, int h, int tile, int end, int lane, uint64_t policy) {
  win.move(tile >> (pc.block_shift + 5 - 7), lane);
  // Lane i < 8 looks up the rows of group i.
  const int j = tile * kTile + 16 * (lane & 7);
  const int blk = win.entry(j >> pc.block_shift);
  const bool there = unsigned(blk) < unsigned(pc.num_blocks);
  if (j < end && !there && lane < 8) set_error(pc.err, PKV_DEVERR_BLOCK_ID);
  const int none = pc.num_blocks * pc.num_kv_heads * pc.block_size;           // a row outside: zeros
  const int y = j < end && there ? (blk * pc.num_kv_heads + h) * pc.block_size + (j & (pc.block_size - 1)) : none;
  if (lane == 0) mbar_arrive_expect_tx(bar, D / 64 * kHalfBytes);
  __syncwarp();
  if (lane < 8) {
#pragma unroll
    for (int d = 0; d < D / 64; ++d) tma_load_2d(dst + d * kHalfBytes + lane * 2048, map, bar, 64 * d, y, policy);
  }
}

// 16-bit values of a row that are infinite or NaN, set to zero in an operand's row; whether there were any.
template <bool kBF16, int D>
__device__ __forceinline__ bool make_row_finite(uint32_t base, int r) {
  uint32_t m = 0;                                            // the largest magnitudes; NaN if any is
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    const uint4 v = lds128(operand_at(base, r, c));
    max_magnitudes<kBF16>(m, v.x);
    max_magnitudes<kBF16>(m, v.y);
    max_magnitudes<kBF16>(m, v.z);
    max_magnitudes<kBF16>(m, v.w);
  }
  const float2 mm = unpack2<kBF16>(m);
  if (fabsf(mm.x) < INFINITY && fabsf(mm.y) < INFINITY) return false;
  for (int c = 0; c < D / 8; ++c) {
    const uint32_t at = operand_at(base, r, c);
    const uint4 v = lds128(at);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float2 f = unpack2<kBF16>(w[u]);
      if (!(fabsf(f.x) < INFINITY)) w[u] &= 0xffff0000u;
      if (!(fabsf(f.y) < INFINITY)) w[u] &= 0x0000ffffu;
    }
    sts128(at, w[0], w[1], w[2], w[3]);
  }
  return true;
}

// 2^-e as fp64, |e| < 1000.
__device__ __forceinline__ double exp2_int(int e) { return __hiloint2double((1023 + e) << 20, 0); }

// Flat rows f0 .. f0 + n - 1 (n <= 128) of a chunk whose first row is q0 and of kv head h, flat row f being
// row f / G of head h G + f mod G, as an operand at `base`, by kThreadsOf threads, 8 for a row.  Quantised
// caches (kToF16): as fp16, times the sign of the kv head's scale, and for bf16 times a power of two.
// put(r, c, e) gets, once for row r, the factor c from products to scores in units of log2 (scale_log2 *
// head_scale and that power; for 16-bit caches scale_log2) and e = extra(i), i being the row's number among
// [total_q][num_heads]; it is asked for together with the rows.  kAhead rows of a thread are on their way
// at a time, and ready() is called when the first of them are: it waits until the operand's place is free,
// and where it returns false nothing is written.  With copies > 1 (n <= 32) the rows also go to rows 32, 64
// .. on.
template <bool kBF16, bool kToF16, int D, int kThreadsOf, int kAhead, typename Ready, typename Extra, typename Put>
__device__ __forceinline__ bool load_queries(uint32_t base, const uint8_t* q, int64_t q0, int num_heads, int h,
                                             const Divisor& group, int f0, int n, int copies, float scale_log2, float head_scale, int tid,
                                             Ready ready, Extra extra, Put put) {
  constexpr int kRows = kThreadsOf / 8, kVec = D / 64;            // rows of a pass; 16-byte vectors per lane and row
  const int G = int(group.d), sub = tid & 7, r0 = tid >> 3;
  const int first = int(q0 * num_heads) + h * G;
  const uint32_t flip = kToF16 && head_scale < 0.f ? 0x80008000u : 0u;
  for (int b = r0; b < n + r0; b += kRows * kAhead) {        // (the same trip count for every thread)
    uint4 v[kAhead][kVec];
    float ex[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int r = b + u * kRows;
#pragma unroll
      for (int c = 0; c < kVec; ++c) v[u][c] = make_uint4(0, 0, 0, 0);
      if (r < n) {
        const int f = f0 + r, row = int(group.quotient(f));
        const int i = first + f + row * (num_heads - G);     // (below 2^31)
        const uint8_t* src = q + int64_t(i) * (2 * D);
        ex[u] = extra(i);
#pragma unroll
        for (int c = 0; c < kVec; ++c) v[u][c] = ld_stream(src + 16 * (sub + 8 * c), true);
      }
    }
    if (b == r0 && !ready()) return false;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int r = b + u * kRows;
      int shift = 0;
      float mul = 1.f;
      if constexpr (kToF16 && kBF16) {
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
          max_magnitudes<true>(m, v[u][c].x);
          max_magnitudes<true>(m, v[u][c].y);
          max_magnitudes<true>(m, v[u][c].z);
          max_magnitudes<true>(m, v[u][c].w);
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) max_magnitudes<true>(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float2 mm = unpack2<true>(m & 0x7fff7fffu);
        const float top = mm.x > mm.y ? mm.x : mm.y;
        const bool finite = mm.x < INFINITY && mm.y < INFINITY;
        shift = finite ? min(14 - (int(__float_as_uint(top) >> 23) - 127), 126) : 0;
        mul = __uint_as_float(uint32_t(127 + shift) << 23);  // shift is -113 .. 126
      }
      if (r < n) {
        if (sub == 0) {
          float c = scale_log2;
          if constexpr (kToF16) {
            // 0 * -inf would be NaN.  Products are below 2^35 here, so that with 1e-35 scores are as good as 0.
            c = float(double(scale_log2) * fabs(double(head_scale)) * exp2_int(-shift));
            c = c < 1e-35f ? 1e-35f : c;
          }
          put(r, c, ex[u]);
        }
#pragma unroll
        for (int c = 0; c < kVec; ++c) {
          uint32_t w[4] = {v[u][c].x, v[u][c].y, v[u][c].z, v[u][c].w};
          if constexpr (kToF16) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if constexpr (kBF16) {
                const float2 f = unpack2<true>(w[k]);
                w[k] = pack2<false>(f.x * mul, f.y * mul);
              }
              w[k] ^= flip;
            }
          }
          for (int k = 0; k < copies; ++k) sts128(operand_at(base, r + 32 * k, sub + 8 * c), w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
  return true;
}

}  // namespace pkv
