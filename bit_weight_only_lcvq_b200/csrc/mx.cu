// Packing into the block-scaled formats and decoding them (see mx.cuh for the
// formats): element i of a block with largest magnitude max becomes
//     q_i = round(x_i / s),  s the smallest power of two with max <= top s,
// and stands for q_i s.  Division by s is exact, so the one rounding is that to
// the format's grid (to nearest, ties to even).
//
// Both kernels are bound by HBM: packing reads 2 or 4 B an element and writes
// 0.53 (mx4) or 1.03 (mx8), decoding the reverse.  A warp takes 256 consecutive
// columns of one row at a time, eight elements a lane, so a block is four
// neighbouring lanes and its maximum two shuffles.  A warp has four such
// pieces in flight where there is enough work to fill the GPU that way.
// Measured on 8192 x 14336 (bytes read and written over time): mx8 from bf16 56 us
// (6.4 TB/s), from fp32 83 (7.1); mx4 from bf16 51 (5.8), from fp32 76 (7.0);
// decoding to bf16 54 and 47, to fp32 91 and 83 (6.4 to 6.6).
#include "common.cuh"
#include "gemv_common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "mx_pack.cuh"
#include "pdl.cuh"

namespace lcvq {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPiece = 256;  // columns per warp piece, 8 per lane

// A warp packs kUnits pieces of one row: `segs` such segments make a row.
template <bool kMx4, bool kF32, int kUnits>
__global__ void __launch_bounds__(kThreads)
    mx_pack_kernel(const void* X, int64_t ld, int64_t rows, int64_t cols, int segs,
                   uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  // X may come from the kernel just before this one (see ld_global_v4)
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t seg = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t row = seg / segs;
  if (row >= rows) return;
  const int64_t c0 = (seg - row * segs) * (kUnits * kPiece) + 8 * lane;
  const int64_t tiles_k = mx::scale_tiles_k(cols);
  const int left = static_cast<int>(cols - c0), pad = static_cast<int>(tiles_k * 128 - c0);
  const char* src = static_cast<const char*>(X) + (row * ld + c0) * (kF32 ? 4 : 2);
  mx::Eight<kF32> x[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    if (u * kPiece < left) x[u].load(src + u * kPiece * (kF32 ? 4 : 2));
    else x[u].zero();
  }
  uint8_t* dst = q + (kMx4 ? row * (cols / 2) + c0 / 2 : row * cols + c0);
  uint8_t* sc = scales + mx::scale_word(row, c0 >> 7, tiles_k) + ((c0 >> 5) & 3);
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    uint32_t m = x[u].max_bits();
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t sb = mx::scale_byte<kMx4>(m);
    const bool in = u * kPiece < left;
    if (in) {
      const uint2 o = mx::pack8<kMx4, kF32>(x[u], sb);
      if constexpr (kMx4) *reinterpret_cast<uint32_t*>(dst + u * kPiece / 2) = o.x;
      else *reinterpret_cast<uint2*>(dst + u * kPiece) = o;
    }
    // every fourth lane has a block; the blocks of a tile past the last column are 0
    if ((lane & 3) == 0 && u * kPiece < pad) sc[u * (kPiece / 128) * mx::kTileBytes] = in ? sb : 0;
  }
}

// Decoding: a lane takes eight consecutive columns for bf16 and, for fp32, four in
// either half of the piece, so that a warp's 16-byte stores are 512 consecutive
// bytes (two stores to 32 bytes of a lane's own measured 121 us against 97 on
// mx4, 8192 x 14336).
template <bool kMx4, bool kF32, int kUnits>
__global__ void __launch_bounds__(kThreads)
    mx_decode_kernel(const uint8_t* q, const uint8_t* scales, int64_t rows, int64_t cols, int segs,
                     void* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kParts = kF32 ? 2 : 1;
  constexpr int kStep = kPiece / kParts;  // columns between a lane's parts
  const int lane = threadIdx.x & 31;
  const int64_t seg = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t row = seg / segs;
  if (row >= rows) return;
  const int64_t c0 = (seg - row * segs) * (kUnits * kPiece) + (kF32 ? 4 : 8) * lane;
  const int left = static_cast<int>(cols - c0);
  const uint8_t* src = q + (kMx4 ? row * (cols / 2) + c0 / 2 : row * cols + c0);
  const uint8_t* sc = scales + mx::scale_word(row, c0 >> 7, mx::scale_tiles_k(cols)) + ((c0 >> 5) & 3);
  char* dst = static_cast<char*>(out) + (row * cols + c0) * (kF32 ? 4 : 2);
  uint2 w[kUnits * kParts];
  uint32_t sb[kUnits * kParts];
#pragma unroll
  for (int u = 0; u < kUnits * kParts; ++u) {
    w[u] = make_uint2(0, 0);
    sb[u] = 0;
    if (u * kStep < left) {
      if constexpr (kF32) w[u].x = kMx4 ? ld_global_u16(src + u * kStep / 2) : ld_global_u32(src + u * kStep);
      else if constexpr (kMx4) w[u].x = ld_global_u32(src + u * kStep / 2);
      else w[u] = ld_global_v2(src + u * kStep);
      sb[u] = ld_global_u8(sc + u * (kStep / 128) * mx::kTileBytes);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnits * kParts; ++u) {
    if (u * kStep >= left) break;
    if constexpr (kF32) {
      const float s = mx::scale_value(sb[u]);
      float4 o;
      if constexpr (kMx4) {
        const float2 a = mx::e2m1_values(w[u].x), b = mx::e2m1_values(w[u].x >> 8);
        o = make_float4(a.x * s, a.y * s, b.x * s, b.y * s);
      } else {  // bytes 0, 1, 2, 3 hold elements 0, 2, 1, 3
        o = make_float4(mx::mx8_value(w[u].x, s), mx::mx8_value(w[u].x >> 16, s),
                        mx::mx8_value(w[u].x >> 8, s), mx::mx8_value(w[u].x >> 24, s));
      }
      *reinterpret_cast<float4*>(dst + u * kStep * 4) = o;
    } else {
      uint4 o;  // exact: products of at most seven significant bits with a power of two
      if constexpr (kMx4) {
        const float s = mx::scale_value(sb[u]);
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = mx::e2m1_values(w[u].x >> (8 * i));
          p[i] = pack_bf16x2(f.x * s, f.y * s);
        }
        o = make_uint4(p[0], p[1], p[2], p[3]);
      } else {
        const uint32_t s2 = mx::scale_bf16x2(sb[u]);
        mx::mx8_word_bf16(w[u].x, s2, o.x, o.y);
        mx::mx8_word_bf16(w[u].y, s2, o.z, o.w);
      }
      *reinterpret_cast<uint4*>(dst + u * kStep * 2) = o;
    }
  }
}

// Pieces of a row that a warp takes: four from one CTA per SM on (bf16 2048 x 4096 to
// mx4 5.3 us against 7.0 with one, 512 x 4096 2.3 against 2.7; 256 x 4096, below that,
// 1.9 with either), unless the last four would mostly lie beyond the row (mx8
// 4096 x 512: 3.4 with four, 2.6 with one).
constexpr int kUnits = 4;
int64_t segments(int64_t cols, int units) { return ceil_div(cols, int64_t(kPiece) * units); }
bool many_segments(int64_t rows, int64_t cols) {
  const int64_t segs = segments(cols, kUnits);
  return rows * segs >= int64_t(kNumSMsB200) * kWarps && 4 * cols >= 3 * segs * kUnits * kPiece;
}

}  // namespace

cudaError_t launch_mx_pack(const void* X, bool f32, int64_t rows, int64_t cols, int64_t ld, bool mx4,
                           uint8_t* q, uint8_t* scales, cudaStream_t s, int* launches) {
  const bool many = many_segments(rows, cols);
  const int64_t segs = segments(cols, many ? kUnits : 1), grid = ceil_div(rows * segs, kWarps);
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, kThreads, 0, s, X, ld, rows, cols, static_cast<int>(segs), q, scales);
  };
  ++*launches;
  if (mx4) {
    if (f32) return many ? go(mx_pack_kernel<true, true, kUnits>) : go(mx_pack_kernel<true, true, 1>);
    return many ? go(mx_pack_kernel<true, false, kUnits>) : go(mx_pack_kernel<true, false, 1>);
  }
  if (f32) return many ? go(mx_pack_kernel<false, true, kUnits>) : go(mx_pack_kernel<false, true, 1>);
  return many ? go(mx_pack_kernel<false, false, kUnits>) : go(mx_pack_kernel<false, false, 1>);
}

cudaError_t launch_mx_decode(const uint8_t* q, const uint8_t* scales, int64_t rows, int64_t cols,
                             bool mx4, void* out, bool f32, cudaStream_t s, int* launches) {
  const bool many = many_segments(rows, cols);
  const int64_t segs = segments(cols, many ? kUnits : 1), grid = ceil_div(rows * segs, kWarps);
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kern) {
    return launch_pdl(kern, grid, kThreads, 0, s, q, scales, rows, cols, static_cast<int>(segs), out);
  };
  ++*launches;
  if (mx4) {
    if (f32) return many ? go(mx_decode_kernel<true, true, kUnits>) : go(mx_decode_kernel<true, true, 1>);
    return many ? go(mx_decode_kernel<true, false, kUnits>) : go(mx_decode_kernel<true, false, 1>);
  }
  if (f32) return many ? go(mx_decode_kernel<false, true, kUnits>) : go(mx_decode_kernel<false, true, 1>);
  return many ? go(mx_decode_kernel<false, false, kUnits>) : go(mx_decode_kernel<false, false, 1>);
}

}  // namespace lcvq
