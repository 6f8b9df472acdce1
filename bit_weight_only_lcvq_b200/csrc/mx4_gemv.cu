// Product of two mx4 matrices for few tokens:
//     Y[m][n] = sum_b sx[m][b] sw[n][b] sum_{k in b} x[m][k] w[n][k]
// over the blocks b of 32 positions, x and w the e2m1 elements.
//
// Twice an e2m1 element is an integer in [-12, 12], so the inner sum of a block
// is an exact integer (|sum| <= 32 * 144), which one m16n8k32 integer MMA forms
// for 16 rows and 8 tokens: its k extent is one block.  The MMA starts from the
// bit pattern of 1.5 * 2^23, so its result read as a float is that constant plus
// the sum: a subtraction instead of an integer conversion (a quarter of the
// rate).  Each block's sum is then scaled and added in fp32.
//
// A word of eight nibbles becomes two registers of four signed bytes by byte
// permutes: a permute with a nibble as selector picks one of eight table bytes
// by its low three bits, and with the top bit set gives that byte's sign (zero
// in this table), so one permute yields the positive elements and one, with the
// top bits flipped, the negated ones.
//
// What bounds it: the packed weights' bytes (17/32 B a weight) when they stream
// from HBM, launch and load latency at the usual sizes, where all of a warp's
// loads are in flight at once.  A tile is 16 rows over the whole of K; its eight
// warps take the 128-position units u = w, w + 8, ... and are summed in warp
// order at the end.  The 16 rows are 32 q + 4 c + j (q, j < 4) of a 128-row
// scale tile: their scales are then 64 consecutive bytes.
#include "common.cuh"
#include "gemv_common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "sm100.cuh"

namespace lcvq {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;          // rows of a tile
constexpr int kUnitBytes = 64;     // packed bytes of 128 positions

template <int NT>
struct Ring {  // one stage of a warp's ring
  static constexpr int kTok = 8 * NT;
  static constexpr int kA = 0;                                // 16 rows x 64 B
  static constexpr int kX = kA + kRows * kUnitBytes;          // tokens x 64 B
  static constexpr int kSw = kX + kTok * kUnitBytes;          // 16 scale words
  static constexpr int kSx = kSw + kRows * 4;                 // tokens x 16 B
  static constexpr int kBytes = kSx + kTok * 16;
  static constexpr int kStages = NT <= 2 ? 4 : 3;
  static constexpr int kSmem = kWarps * kStages * kBytes;
};

// prmt with whole selector nibbles (the intrinsic drops the sign bit of each)
__device__ __forceinline__ uint32_t prmt(uint32_t lo, uint32_t hi, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;\n" : "=r"(r) : "r"(lo), "r"(hi), "r"(sel));
  return r;
}
// Eight e2m1 nibbles -> twice their values as signed bytes (nibbles 0-3, 4-7).
__device__ __forceinline__ void e2m1_s8(uint32_t w, uint32_t& lo, uint32_t& hi) {
  constexpr uint32_t kT0 = 0x03020100u, kT1 = 0x0C080604u;  // twice 0 .5 1 1.5, 2 3 4 6
  const uint32_t f = w ^ 0x88888888u;
  const uint32_t p0 = prmt(kT0, kT1, w), n0 = prmt(kT0, kT1, f);
  const uint32_t p1 = prmt(kT0, kT1, w >> 16), n1 = prmt(kT0, kT1, f >> 16);
  // bytes in 128 - 12 .. 128 + 12: no borrow between them
  lo = (p0 + 0x80808080u - n0) ^ 0x80808080u;
  hi = (p1 + 0x80808080u - n1) ^ 0x80808080u;
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
constexpr uint32_t kMagic = 0x4B400000u;  // 1.5 * 2^23
// D = A B + kMagic for one m16n8k32 tile of signed bytes
__device__ __forceinline__ void mma_s8_magic(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};\n"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(kMagic));
}
// scale of byte b of a word, without the NaN of 255 (handled per word)
__device__ __forceinline__ float scale_of(uint32_t word, int b) {
  const uint32_t bits = (b < 3 ? word << (23 - 8 * b) : word >> 1) & 0x7F800000u;
  return __uint_as_float(max(bits, 0x00400000u));
}
__device__ __forceinline__ bool has_nan(uint32_t word) { return __vcmpeq4(word, 0xFFFFFFFFu) != 0; }

template <int NT, bool kF32>
__global__ void __launch_bounds__(kThreads)
    mx4_gemv_kernel(const uint8_t* xq, const uint8_t* xs, int64_t M, const uint8_t* wq,
                    const uint8_t* ws, int64_t N, int64_t K, void* __restrict__ Y) {
  using R = Ring<NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t G = blockIdx.x >> 3;          // 128-row group
  const int ct = blockIdx.x & 7;              // tile within it
  const int64_t m0 = int64_t(blockIdx.y) * R::kTok;
  griddep_wait();  // the operands may come from the kernel just before this one
  griddep_launch_dependents();
  if (G * 128 + 4 * ct >= N) return;
  const int64_t row_bytes = K / 2, units = ceil_div(K, 128);
  const int quarter = static_cast<int>(m0 >> 5) & 3;
  const uint32_t ring = sm100::smem_u32(smem) + warp * R::kStages * R::kBytes;

  // this lane's copies of one unit
  const int r0 = lane >> 2, c0 = lane & 3;
  auto row_of = [&](int r) { return G * 128 + 32 * (r & 3) + 4 * ct + (r >> 2); };
  auto slot = [](int r, int c) { return r * kUnitBytes + ((c ^ ((r >> 1) & 3)) << 4); };
  auto load = [&](int stage, int64_t u) {
    const uint32_t st = ring + stage * R::kBytes;
    const int64_t off = u * kUnitBytes + 16 * c0;
    const bool in = off < row_bytes;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + 8 * i;
      const int64_t n = row_of(r);
      const bool ok = in && n < N;
      cp_async16_zfill(st + R::kA + slot(r, c0), ok ? wq + n * row_bytes + off : wq, ok);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int t = r0 + 8 * i;
      const bool ok = in && m0 + t < M;
      cp_async16_zfill(st + R::kX + slot(t, c0), ok ? xq + (m0 + t) * row_bytes + off : xq, ok);
    }
    if (lane < 4)
      cp_async16_zfill(st + R::kSw + 16 * lane, ws + (G * units + u) * mx::kTileBytes + 64 * ct + 16 * lane,
                       true);
    if (lane < R::kTok) {
      const int64_t m = m0 + lane;
      const bool ok = m < M;
      cp_async16_zfill(st + R::kSx + 16 * lane,
                       ok ? xs + ((m >> 7) * units + u) * mx::kTileBytes + ((m & 31) << 4) : xs, ok);
    }
  };

  const int g = lane >> 2, t = lane & 3;
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;

#pragma unroll
  for (int s = 0; s < R::kStages; ++s) {
    if (warp + kWarps * s < units) load(s, warp + kWarps * s);
    cp_async_commit();
  }
  int stage = 0;
  for (int64_t u = warp; u < units; u += kWarps) {
    cp_async_wait<R::kStages - 1>();
    __syncwarp();
    const uint32_t st = ring + stage * R::kBytes;
    uint32_t a[4][2];  // block b: the words of rows g and g + 8
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t v[4];
      ldmatrix4(st + R::kA + slot((lane & 7) + (lane & 8), 2 * h + (lane >> 4)), v);
      a[2 * h][0] = v[0]; a[2 * h][1] = v[1]; a[2 * h + 1][0] = v[2]; a[2 * h + 1][1] = v[3];
    }
    uint32_t x[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) ldmatrix4(st + R::kX + slot((lane & 7) + 8 * i, lane >> 3), x[i]);
    const uint32_t* sw = reinterpret_cast<const uint32_t*>(smem + (st - sm100::smem_u32(smem)) + R::kSw);
    const uint32_t* sx = reinterpret_cast<const uint32_t*>(smem + (st - sm100::smem_u32(smem)) + R::kSx);
    const uint32_t sw0 = sw[g], sw1 = sw[g + 8];
    uint32_t sx0[NT], sx1[NT];
    bool bad = has_nan(sw0) || has_nan(sw1);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      sx0[i] = sx[(8 * i + 2 * t) * 4 + quarter];
      sx1[i] = sx[(8 * i + 2 * t + 1) * 4 + quarter];
      bad = bad || has_nan(sx0[i]) || has_nan(sx1[i]);
    }
    __syncwarp();
    if (u + kWarps * R::kStages < units) load(stage, u + kWarps * R::kStages);
    cp_async_commit();
    if (++stage == R::kStages) stage = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t a0, a1, a2, a3;
      e2m1_s8(a[b][0], a0, a2);
      e2m1_s8(a[b][1], a1, a3);
      const float w0 = scale_of(sw0, b), w1 = scale_of(sw1, b);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        uint32_t b0, b1;
        e2m1_s8(x[i][b], b0, b1);
        int d[4];
        mma_s8_magic(d, a0, a1, a2, a3, b0, b1);
        const float x0 = scale_of(sx0[i], b), x1 = scale_of(sx1[i], b);
        acc[i][0] = fmaf((__int_as_float(d[0]) - 12582912.f) * w0, x0, acc[i][0]);
        acc[i][1] = fmaf((__int_as_float(d[1]) - 12582912.f) * w0, x1, acc[i][1]);
        acc[i][2] = fmaf((__int_as_float(d[2]) - 12582912.f) * w1, x0, acc[i][2]);
        acc[i][3] = fmaf((__int_as_float(d[3]) - 12582912.f) * w1, x1, acc[i][3]);
      }
    }
    if (bad) {  // a block that stands for NaN makes its row's or token's sums NaN
      const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (has_nan(sw0)) acc[i][0] = acc[i][1] = nan;
        if (has_nan(sw1)) acc[i][2] = acc[i][3] = nan;
        if (has_nan(sx0[i])) acc[i][0] = acc[i][2] = nan;
        if (has_nan(sx1[i])) acc[i][1] = acc[i][3] = nan;
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);  // [warp][row][token]
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    float* p = part + (warp * kRows + g) * R::kTok + 8 * i + 2 * t;
    p[0] = acc[i][0];
    p[1] = acc[i][1];
    p[8 * R::kTok] = acc[i][2];
    p[8 * R::kTok + 1] = acc[i][3];
  }
  __syncthreads();
  // thread (q, token): rows 32 q + 4 ct .. + 3, summed over the warps in order;
  // the elements were doubled on both sides
  const int tok = threadIdx.x >> 2, q = threadIdx.x & 3;
  const int64_t n = G * 128 + 32 * q + 4 * ct, m = m0 + tok;
  if (tok < R::kTok && m < M && n < N) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += part[(w * kRows + 4 * j + q) * R::kTok + tok];
      y[j] = 0.25f * s;
    }
    if constexpr (kF32)
      *reinterpret_cast<float4*>(static_cast<float*>(Y) + m * N + n) = make_float4(y[0], y[1], y[2], y[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(Y) + m * N + n) =
          make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
  }
}

template <int NT, bool kF32>
cudaError_t launch_nt(const uint8_t* xq, const uint8_t* xs, int64_t M, const uint8_t* wq,
                      const uint8_t* ws, int64_t N, int64_t K, void* Y, cudaStream_t s) {
  using R = Ring<NT>;
  static_assert(R::kSmem >= kWarps * kRows * R::kTok * 4, "the partial sums reuse the rings");
  auto kern = mx4_gemv_kernel<NT, kF32>;
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), R::kSmem);
      e != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(N, 128) * 8), static_cast<unsigned>(ceil_div(M, R::kTok)), 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = R::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, kern, xq, xs, M, wq, ws, N, K, Y); e != cudaSuccess)
    return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx4_gemv(const uint8_t* xq, const uint8_t* xs, int64_t M, const uint8_t* wq,
                            const uint8_t* ws, int64_t N, int64_t K, void* Y, bool f32,
                            cudaStream_t s, int* launches) {
  ++*launches;
  if (M <= 8)
    return f32 ? launch_nt<1, true>(xq, xs, M, wq, ws, N, K, Y, s)
               : launch_nt<1, false>(xq, xs, M, wq, ws, N, K, Y, s);
  if (M <= 16)
    return f32 ? launch_nt<2, true>(xq, xs, M, wq, ws, N, K, Y, s)
               : launch_nt<2, false>(xq, xs, M, wq, ws, N, K, Y, s);
  return f32 ? launch_nt<4, true>(xq, xs, M, wq, ws, N, K, Y, s)
             : launch_nt<4, false>(xq, xs, M, wq, ws, N, K, Y, s);
}

}  // namespace lcvq
