// Single elements of a paged cache of any type, for code where speed does not matter.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// Elements 2 c and 2 c + 1 of pool row `row` (of [num_blocks * num_kv_heads * block_size] rows), without the
// head's scale; exact.
__device__ __forceinline__ float2 cache_pair(const uint8_t* cache, pkv_dtype kv, int D, int64_t row, int c) {
  if (kv == PKV_FP4_E2M1) {
    const uint8_t* tile = cache + (row >> 4) * 9 * D;
    const int rr = int(row & 15);
    uint32_t half[4];
    e2m1x8_to_f16x8(tile[rr * (D / 2) + c], half);
    const float s = unpack2<false>(e4m3x2_to_f16x2(tile[8 * D + rr * (D / 16) + c / 8])).x;
    const float2 v = unpack2<false>(half[0]);
    return make_float2(v.x * s, v.y * s);
  }
  if (kv == PKV_FP8_E4M3)
    return unpack2<false>(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(cache + row * D + 2 * c)));
  const uint32_t w = *reinterpret_cast<const uint32_t*>(cache + (row * D + 2 * c) * 2);
  return kv == PKV_BF16 ? unpack2<true>(w) : unpack2<false>(w);
}

}  // namespace pkv
