// Packing into the block-scaled formats and decoding them (see mx.cuh for the
// formats): element i of a block with largest magnitude max becomes
//     q_i = round(x_i / s),  s the smallest power of two with max <= top s,
// and stands for q_i s.  Division by s is exact, so the one rounding is that to
// the format's grid (to nearest, ties to even).
//
// Both kernels are bound by HBM: packing reads 2 or 4 B an element and writes
// 0.53 (mx4) or 1.03 (mx8), decoding the reverse.  A warp takes 256 consecutive
// columns of one row at a time, eight elements a lane, so a block is four
// neighbouring lanes and its maximum two shuffles; the four scale bytes of 128
// columns meet in one lane and leave as one word.  kUnits such pieces are in
// flight per warp where there is enough work to fill the GPU with four of them
// (kUnitsMin below).
#include "common.cuh"
#include "gemv_common.cuh"
#include "internal.h"
#include "mx.cuh"

namespace lcvq {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPiece = 256;  // columns per warp piece, 8 per lane

// the eight elements of a lane, as fp32
template <bool kF32>
__device__ __forceinline__ void load8(const void* X, int64_t off, float (&x)[8]) {
  if constexpr (kF32) {
    const uint4 a = ld_global_v4(static_cast<const float*>(X) + off);
    const uint4 b = ld_global_v4(static_cast<const float*>(X) + off + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  } else {
    const uint4 a = ld_global_v4(static_cast<const uint16_t*>(X) + off);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(w[i]);
      x[2 * i + 1] = bf16_hi(w[i]);
    }
  }
}

template <bool kMx4, bool kF32, int kUnits>
__global__ void __launch_bounds__(kThreads)
    mx_pack_kernel(const void* X, int64_t ld, int64_t cols, int64_t pieces_per_row, int64_t pieces,
                   uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  // X may come from the kernel just before this one (see ld_global_v4)
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t first = (int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kUnits;
  if (first >= pieces) return;
  int64_t row = first / pieces_per_row, pc = first % pieces_per_row;
  const int64_t tiles_k = mx::scale_tiles_k(cols);
  float x[kUnits][8];
  int64_t rows[kUnits], c0[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    rows[u] = first + u < pieces ? row : -1;
    c0[u] = pc * kPiece + 8 * lane;
    if (rows[u] >= 0 && c0[u] < cols) {
      load8<kF32>(X, row * ld + c0[u], x[u]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
    }
    if (++pc == pieces_per_row) { pc = 0; ++row; }
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    if (rows[u] < 0) break;
    const bool in = c0[u] < cols;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[u][i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t sb = mx::scale_byte<kMx4>(m);
    const float inv = mx::scale_inverse(sb), top = mx::element_top<kMx4>(sb);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = fminf(fmaxf(x[u][i] * inv, -top), top);
      if (sb == 255u) v[i] = 0.f;
    }
    if (in) {
      if constexpr (kMx4) {
        const uint32_t w = mx::e2m1_x4(v[0], v[1], v[2], v[3]) | mx::e2m1_x4(v[4], v[5], v[6], v[7]) << 16;
        *reinterpret_cast<uint32_t*>(q + rows[u] * (cols / 2) + c0[u] / 2) = w;
      } else {
        uint2 w;  // bytes 0, 1, 2, 3 hold elements 0, 2, 1, 3
        w.x = mx::mx8_code(v[0]) | mx::mx8_code(v[2]) << 8 | mx::mx8_code(v[1]) << 16 | mx::mx8_code(v[3]) << 24;
        w.y = mx::mx8_code(v[4]) | mx::mx8_code(v[6]) << 8 | mx::mx8_code(v[5]) << 16 | mx::mx8_code(v[7]) << 24;
        *reinterpret_cast<uint2*>(q + rows[u] * cols + c0[u]) = w;
      }
    }
    // the four blocks of 128 columns (lanes 0, 4, 8, 12 of each half warp)
    uint32_t word = in ? sb << (8 * ((lane >> 2) & 3)) : 0u;
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if ((lane & 15) == 0 && in)
      *reinterpret_cast<uint32_t*>(scales + mx::scale_word(rows[u], c0[u] >> 7, tiles_k)) = word;
  }
}

template <bool kMx4, bool kF32, int kUnits>
__global__ void __launch_bounds__(kThreads)
    mx_decode_kernel(const uint8_t* q, const uint8_t* scales, int64_t cols, int64_t pieces_per_row,
                     int64_t pieces, void* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t first = (int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kUnits;
  if (first >= pieces) return;
  int64_t row = first / pieces_per_row, pc = first % pieces_per_row;
  const int64_t tiles_k = mx::scale_tiles_k(cols);
  uint2 w[kUnits];
  uint32_t sb[kUnits];
  int64_t at[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int64_t c = pc * kPiece + 8 * lane;
    at[u] = first + u < pieces && c < cols ? row * cols + c : -1;
    w[u] = make_uint2(0, 0);
    sb[u] = 0;
    if (at[u] >= 0) {
      if constexpr (kMx4) w[u].x = ld_global_u32(q + at[u] / 2);
      else w[u] = ld_global_v2(q + at[u]);
      sb[u] = ld_global_u32(scales + mx::scale_word(row, c >> 7, tiles_k)) >> (8 * ((c >> 5) & 3)) & 255u;
    }
    if (++pc == pieces_per_row) { pc = 0; ++row; }
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    if (at[u] < 0) continue;
    const float s = mx::scale_value(sb[u]);
    float v[8];
    if constexpr (kMx4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = mx::e2m1_value(w[u].x >> (4 * i)) * s;
    } else {
      auto value = [&](uint32_t b) {
        const float m = static_cast<float>(b & 127u) * s;
        return (b & 128u) ? -m : m;
      };
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // element 4 g + 2 a + b is byte 4 g + a + 2 b
        const int byte = (i & 4) + ((i >> 1) & 1) + 2 * (i & 1);
        v[i] = value((byte < 4 ? w[u].x : w[u].y) >> (8 * (byte & 3)) & 255u);
      }
    }
    if constexpr (kF32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at[u]);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {  // exact: at most seven significant bits
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at[u]) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                     pack_bf16x2(v[6], v[7]));
    }
  }
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), int64_t grid, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...); e != cudaSuccess)
    return e;
  return cudaGetLastError();
}

// pieces from which a warp takes four at a time: two waves of eight resident
// CTAs per SM with four pieces a warp; below, one piece a warp spreads the work
// over more SMs
constexpr int64_t kUnitsMin = int64_t(kNumSMsB200) * 8 * kWarps * 4 * 2;

}  // namespace

cudaError_t launch_mx_pack(const void* X, bool f32, int64_t rows, int64_t cols, int64_t ld, bool mx4,
                           uint8_t* q, uint8_t* scales, cudaStream_t s, int* launches) {
  const int64_t ppr = ceil_div(cols, kPiece), pieces = rows * ppr;
  const bool many = pieces >= kUnitsMin;
  const int64_t grid = ceil_div(pieces, kWarps * (many ? 4 : 1));
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kern) { return launch_pdl(kern, grid, s, X, ld, cols, ppr, pieces, q, scales); };
  ++*launches;
  if (mx4) {
    if (f32) return many ? go(mx_pack_kernel<true, true, 4>) : go(mx_pack_kernel<true, true, 1>);
    return many ? go(mx_pack_kernel<true, false, 4>) : go(mx_pack_kernel<true, false, 1>);
  }
  if (f32) return many ? go(mx_pack_kernel<false, true, 4>) : go(mx_pack_kernel<false, true, 1>);
  return many ? go(mx_pack_kernel<false, false, 4>) : go(mx_pack_kernel<false, false, 1>);
}

cudaError_t launch_mx_decode(const uint8_t* q, const uint8_t* scales, int64_t rows, int64_t cols,
                             bool mx4, void* out, bool f32, cudaStream_t s, int* launches) {
  const int64_t ppr = ceil_div(cols, kPiece), pieces = rows * ppr;
  const bool many = pieces >= kUnitsMin;
  const int64_t grid = ceil_div(pieces, kWarps * (many ? 4 : 1));
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  auto go = [&](auto kern) { return launch_pdl(kern, grid, s, q, scales, cols, ppr, pieces, out); };
  ++*launches;
  if (mx4) {
    if (f32) return many ? go(mx_decode_kernel<true, true, 4>) : go(mx_decode_kernel<true, true, 1>);
    return many ? go(mx_decode_kernel<true, false, 4>) : go(mx_decode_kernel<true, false, 1>);
  }
  if (f32) return many ? go(mx_decode_kernel<false, true, 4>) : go(mx_decode_kernel<false, true, 1>);
  return many ? go(mx_decode_kernel<false, false, 4>) : go(mx_decode_kernel<false, false, 1>);
}

}  // namespace lcvq
