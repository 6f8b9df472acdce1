// The block-scaled formats (mx4, mx8): scales, element codes and the layout of
// the scale bytes, shared by every kernel that writes or reads them.
//
// A block is 32 consecutive elements of a row.  Its scale is s = 2^e with e the
// smallest integer >= -127 such that the largest |x| of the block is at most
// top * s (top = 6 for mx4, 127 for mx8), so no element is clipped and each is
// off by at most half a step of its own grid.  The scale byte is e + 127; 255
// marks a block that held a NaN or an infinity (its element codes are 0 and it
// stands for NaN).
//   mx4  e2m1: sign, two exponent bits, one mantissa bit: 0 0.5 1 1.5 2 3 4 6.
//        Byte i of a row: element 2 i in the low nibble, 2 i + 1 in the high.
//   mx8  sign bit and 7-bit magnitude (0 .. 127): the magnitude fits bf16's
//        mantissa as it stands (mx8_word_bf16); two's complement would not.  In each
//        group of four elements the bytes hold elements 0, 2, 1, 3: masking the
//        even bytes of a word then gives consecutive elements in one register.
// Scales of 128 rows x 128 columns are one 512-byte tile, byte
// 16 (r % 32) + 4 (r / 32 % 4) + (c / 32 % 4): the order in which the tensor core's
// scale copy reads them from shared memory (32 lanes x 16 bytes), so a tile
// moves there with one bulk copy.  Tiles lie row of tiles after row of tiles.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace lcvq {

namespace mx {

constexpr int kBlock = 32;
constexpr int kTileBytes = 512;

__host__ __device__ constexpr int64_t scale_tiles_k(int64_t cols) { return ceil_div(cols, 128); }
__host__ __device__ constexpr int64_t scale_bytes(int64_t rows, int64_t cols) {
  return ceil_div(rows, 128) * scale_tiles_k(cols) * kTileBytes;
}
// byte offset of the 4-byte word with the scales of row r, columns 128 kt .. 128 kt + 127
__host__ __device__ constexpr int64_t scale_word(int64_t r, int64_t kt, int64_t tiles_k) {
  return ((r >> 7) * tiles_k + kt) * kTileBytes + ((r & 31) << 4) + ((r >> 3) & 12);
}

// the scale tiles as a tensor of 512-byte rows, loaded two at a time (the two
// tiles of 256 columns; past the end, zeros)
inline bool make_scale_map(CUtensorMap* map, const uint8_t* scales, int64_t rows, int64_t cols) {
  return make_tensor_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, scales, kTileBytes / 4,
                            uint64_t(ceil_div(rows, 128) * scale_tiles_k(cols)), kTileBytes,
                            kTileBytes / 4, 2, false);
}

// 2^(b - 127); byte 255 is NaN
__device__ __forceinline__ float scale_value(uint32_t b) {
  const uint32_t bits = b == 255u ? 0x7FC00000u : (b == 0u ? 0x00400000u : b << 23);
  return __uint_as_float(bits);
}

// Scale byte of a block from the bits of its largest |x| (as unsigned integers
// the magnitudes order like their values, NaN above infinity above the rest).
template <bool kMx4>
__device__ __forceinline__ uint32_t scale_byte(uint32_t max_bits) {
  if (max_bits >= 0x7F800000u) return 255u;
  // max = m 2^E: 6 = 1.5 * 2^2, 127 = 1.984375 * 2^6
  constexpr uint32_t kEdge = kMx4 ? 0x00400000u : 0x007E0000u;
  constexpr int kDrop = kMx4 ? 2 : 6;
  const int b = static_cast<int>(max_bits >> 23) - kDrop + ((max_bits & 0x007FFFFFu) > kEdge ? 1 : 0);
  return static_cast<uint32_t>(b < 0 ? 0 : b);
}
// 1 / scale, exact (bytes 0 .. 253 occur for finite blocks); 0 for byte 255
__device__ __forceinline__ float scale_inverse(uint32_t b) {
  return b == 255u ? 0.f : __uint_as_float((254u - b) << 23);
}
// The largest element that keeps element * scale finite: the top of the grid,
// except in the highest binade, where rounding up could reach 2^128.
template <bool kMx4>
__device__ __forceinline__ float element_top(uint32_t b) {
  return kMx4 ? (b >= 253u ? 3.f : 6.f) : (b >= 249u ? 63.f : 127.f);
}

// four fp32 already divided by the scale -> four e2m1 nibbles (round to nearest
// even), the first in the lowest nibble
__device__ __forceinline__ uint32_t e2m1_x4(float x0, float x1, float x2, float x3) {
  uint32_t r;
  asm("{\n"
      ".reg .b8 b0, b1;\n"
      ".reg .b16 h0;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      "mov.b16 h0, {b0, b1};\n"
      "cvt.u32.u16 %0, h0;\n"
      "}\n"
      : "=r"(r)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return r;
}
// bits of 2^23 + |x| inv: its low byte is the magnitude |x| / s <= 127, rounded
// to nearest even by the one rounding of the fused multiply-add
__device__ __forceinline__ uint32_t mx8_bits(float x, float inv) {
  return __float_as_uint(fmaf(fabsf(x), inv, 8388608.f));
}

// value of the mx8 byte in bits 0 .. 7 of w, times the scale (exact)
__device__ __forceinline__ float mx8_value(uint32_t w, float s) {
  const float m = (__uint_as_float(0x4B000000u | (w & 0x7Fu)) - 8388608.f) * s;
  return __uint_as_float(__float_as_uint(m) ^ (w << 24 & 0x80000000u));
}

// two e2m1 nibbles (the low byte of w) -> their values (in units of the scale)
__device__ __forceinline__ float2 e2m1_values(uint32_t w) {
  uint32_t h;
  asm("{\n"
      ".reg .b8 b0, b1, b2, b3;\n"
      "mov.b32 {b0, b1, b2, b3}, %1;\n"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
      "}\n"
      : "=r"(h)
      : "r"(w));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four mx8 bytes (one word) -> elements 0, 1 and 2, 3 as bf16 pairs, times the
// scale (s2: the scale as a bf16 pair).  0x4300 | m is the bf16 128 + m, so
// subtracting 128 leaves m and m s is a bf16: both steps are exact.  (One fused
// (128 + m) s - 128 s would save an instruction, but 128 s overflows for the
// largest scales.)  The sign goes in last.
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void mx8_word_bf16(uint32_t w, uint32_t s2, uint32_t& p01, uint32_t& p23) {
  const uint32_t a = mul_bf16x2(sub_bf16x2((w & 0x007F007Fu) | 0x43004300u, 0x43004300u), s2);
  const uint32_t b = mul_bf16x2(sub_bf16x2(((w >> 8) & 0x007F007Fu) | 0x43004300u, 0x43004300u), s2);
  p01 = a ^ ((w << 8) & 0x80008000u);
  p23 = b ^ (w & 0x80008000u);
}
// the scale of byte b as a bf16 pair (exact: a power of two, or NaN)
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t b) {
  const uint32_t h = b == 255u ? 0x7FC0u : (b == 0u ? 0x0040u : b << 7);
  return h | (h << 16);
}

}  // namespace mx
}  // namespace lcvq
