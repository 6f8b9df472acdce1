// Eight consecutive elements of a row -> their packed form, shared by the packing
// kernel and the training forward's X-transform (which packs X as it reads it).
#pragma once

#include "common.cuh"
#include "mx.cuh"

namespace lcvq {
namespace mx {

// Eight consecutive elements of a lane as they lie in memory (bf16: four words).
template <bool kF32>
struct Eight {
  uint32_t w[kF32 ? 8 : 4];

  __device__ __forceinline__ void load(const char* at) {
#pragma unroll
    for (int i = 0; i < (kF32 ? 2 : 1); ++i) {
      const uint4 v = ld_global_v4(at + 16 * i);
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (kF32 ? 8 : 4); ++i) w[i] = 0;
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (kF32) return __uint_as_float(w[i]);
    else return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
  }
  // bits of the largest magnitude, as fp32 (integers order like magnitudes)
  __device__ __forceinline__ uint32_t max_bits() const {
    if constexpr (kF32) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
      return m;
    } else {
      uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
      for (int i = 1; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
      return max(m << 16, m & 0xFFFF0000u);
    }
  }
  // the top bytes (with the signs) of elements 4 g + 0, 2, 1, 3
  __device__ __forceinline__ uint32_t signs(int g) const {
    if constexpr (kF32)
      return __byte_perm(__byte_perm(w[4 * g], w[4 * g + 2], 0x0073), __byte_perm(w[4 * g + 1], w[4 * g + 3], 0x0073), 0x5410);
    else
      return __byte_perm(w[2 * g], w[2 * g + 1], 0x7351);
  }
};

// The packed form of eight elements: mx4 in .x, mx8 in .x and .y.
template <bool kMx4, bool kF32>
__device__ __forceinline__ uint2 pack8(const Eight<kF32>& x, uint32_t sb) {
  const float inv = scale_inverse(sb);
  uint2 o = make_uint2(0, 0);
  if (sb >= (kMx4 ? 253u : 249u)) {  // blocks that are not finite, and the highest binade
    const float top = element_top<kMx4>(sb);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = sb == 255u ? 0.f : fminf(fmaxf(x[i] * inv, -top), top);
    if constexpr (kMx4) {
      o.x = e2m1_x4(v[0], v[1], v[2], v[3]) | e2m1_x4(v[4], v[5], v[6], v[7]) << 16;
    } else {
#pragma unroll
      for (int b = 0; b < 8; ++b) {  // byte b of a group of four holds element 0, 2, 1, 3
        const int i = (b & 4) + ((b >> 1) & 1) + 2 * (b & 1);
        const uint32_t c = (mx8_bits(v[i], 1.f) & 0x7Fu) | (__float_as_uint(v[i]) >> 24 & 0x80u);
        (b < 4 ? o.x : o.y) |= c << (8 * (b & 3));
      }
    }
    return o;
  }
  if constexpr (kMx4) {
    o.x = e2m1_x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv) |
          e2m1_x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv) << 16;
  } else {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = mx8_bits(x[4 * g + i], inv);
      const uint32_t m = __byte_perm(__byte_perm(u[0], u[2], 0x0040), __byte_perm(u[1], u[3], 0x0040), 0x5410);
      (g ? o.y : o.x) = m | (x.signs(g) & 0x80808080u);
    }
  }
  return o;
}

}  // namespace mx
}  // namespace lcvq
