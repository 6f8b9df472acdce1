// CUDA-core paths: forward, dX and the dW epilogue for any M and either
// activation type (fp32 or bf16), with fp32 arithmetic throughout.  They carry
// the fp32 workloads (where tensor-core inputs would not meet an fp32
// tolerance) and every shape the tensor-core kernels do not take.
//
//   forward  Y[m][n]  = sum_k X[m][k] W~[n][k]            (decoupleQ eq. (1))
//   dX[m][k]          = sum_n dY[m][n] W~[n][k]            (gradient through the
//                                                           linear map, LC-QAT
//                                                           Methodology 1)
//   G[n][k]           = sum_m dY[m][n] X[m][k]   -> per d-vector epilogue:
//   dWp[n][gd+j]      = mask * sum_i A[i][j] G[n][gd+i]    (STE, Methodology 3)
//   dA[i][j] += G[n][gd+i] z[n][gd+j],  dB[i] += G[n][gd+i]  (per-tile partials)
//
// W~ tiles are decoded on chip from the packed codes (A z + B in fp32, a fixed
// FMA order) and never written to memory.
#include "common.cuh"
#include "gemv_common.cuh"
#include "internal.h"
#include "pdl.cuh"

namespace lcvq {

namespace {

constexpr int kT = 64;   // output tile edge
constexpr int kBK = 32;  // contraction chunk
constexpr int kThreads = 256;

template <bool kBf16>
__device__ __forceinline__ void load8(const void* base, int64_t idx, float (&v)[8]) {
  if constexpr (kBf16) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + idx);
    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x);
    v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z);
    v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + idx);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

template <bool kBf16>
__device__ __forceinline__ void store_out(void* base, int64_t idx, float v) {
  if constexpr (kBf16)
    static_cast<uint16_t*>(base)[idx] = f32_to_bf16(v);
  else
    static_cast<float*>(base)[idx] = v;
}

// decode 8 consecutive weights (whole d-vectors) of one row from 16 code bits
template <int D>
__device__ __forceinline__ void decode8(uint32_t bits16, const float* sA, const float* sB,
                                        float (&w)[8]) {
#pragma unroll
  for (int v = 0; v < 8 / D; ++v) {
    float z[D];
#pragma unroll
    for (int j = 0; j < D; ++j) z[j] = static_cast<float>((bits16 >> (2 * (v * D + j))) & 3u);
#pragma unroll
    for (int i = 0; i < D; ++i) {
      float acc = sB[i];
#pragma unroll
      for (int j = 0; j < D; ++j) acc = fmaf(sA[i * D + j], z[j], acc);
      w[v * D + i] = acc;
    }
  }
}

__device__ __forceinline__ uint32_t codes16(const uint8_t* packed, int64_t Kb, int64_t row,
                                            int64_t k) {
  return *reinterpret_cast<const uint16_t*>(packed + row * Kb + (k >> 2));
}

template <int D>
__device__ __forceinline__ void load_AB(const float* A, const float* B, float* sA, float* sB) {
  for (int i = threadIdx.x; i < D * D; i += blockDim.x) sA[i] = A[i];
  for (int i = threadIdx.x; i < D; i += blockDim.x) sB[i] = B[i];
}

// acc[i][j] += sum over one chunk of P[.][4 ty + i] Q[.][4 tx + j], in chunk order.
// The chunks are double buffered in shared memory (one barrier each) and the next
// one's global loads are issued before this one's products (dW and its reduction at
// 2000 x 1024 -> 1024: 155 us, waiting for each chunk's loads 222).
__device__ __forceinline__ void mac_step(const float (*P)[kT + 4], const float (*Q)[kT + 4], int ty,
                                         int tx, float (&acc)[4][4]) {
#pragma unroll 8
  for (int kk = 0; kk < kBK; ++kk) {
    const float4 p = *reinterpret_cast<const float4*>(&P[kk][ty * 4]);
    const float4 q = *reinterpret_cast<const float4*>(&Q[kk][tx * 4]);
    const float a[4] = {p.x, p.y, p.z, p.w}, b[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
  }
}

// ---------------------------------------------------------------- forward
template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads) simt_forward_kernel(
    const void* __restrict__ X, int64_t M, const uint8_t* __restrict__ packed, int64_t N,
    int64_t K, const float* __restrict__ A, const float* __restrict__ B, void* __restrict__ Y) {
  __shared__ float sA[D * D], sB[D];
  __shared__ __align__(16) float Xs[2][kBK][kT + 4], Ws[2][kBK][kT + 4];
  load_AB<D>(A, B, sA, sB);
  const int tid = threadIdx.x;
  const int64_t m0 = int64_t(blockIdx.y) * kT, n0 = int64_t(blockIdx.x) * kT;
  const int ty = tid / 16, tx = tid % 16;
  const int lrow = tid / 4, lk = (tid % 4) * 8;
  const int64_t Kb = K / 4;
  float acc[4][4] = {};
  float xv[8] = {};
  uint32_t bits = 0;
  auto load = [&](int64_t k0) {  // this thread's part of the next step
    if (m0 + lrow < M) load8<kBf16>(X, (m0 + lrow) * K + k0 + lk, xv);
    if (n0 + lrow < N) bits = codes16(packed, Kb, n0 + lrow, k0 + lk);
  };
  load(0);
  __syncthreads();
  int b = 0;
  for (int64_t k0 = 0; k0 < K; k0 += kBK, b ^= 1) {
    float wv[8] = {};
    if (n0 + lrow < N) decode8<D>(bits, sA, sB, wv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      Xs[b][lk + i][lrow] = xv[i];
      Ws[b][lk + i][lrow] = wv[i];
    }
    __syncthreads();
    if (k0 + kBK < K) load(k0 + kBK);
    mac_step(Xs[b], Ws[b], ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < M && n < N) store_out<kBf16>(Y, m * N + n, acc[i][j]);
    }
}

// ---------------------------------------------------------------- dX
template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads) simt_dx_kernel(
    const void* __restrict__ dY, int64_t M, const uint8_t* __restrict__ packed, int64_t N,
    int64_t K, const float* __restrict__ A, const float* __restrict__ B, void* __restrict__ dX) {
  __shared__ float sA[D * D], sB[D];
  __shared__ __align__(16) float Ds[2][kBK][kT + 4];  // [n][m]
  __shared__ __align__(16) float Ws[2][kBK][kT + 4];  // [n][k]
  load_AB<D>(A, B, sA, sB);
  const int tid = threadIdx.x;
  const int64_t m0 = int64_t(blockIdx.y) * kT, k0 = int64_t(blockIdx.x) * kT;
  const int ty = tid / 16, tx = tid % 16;
  const int64_t Kb = K / 4;
  float acc[4][4] = {};
  const int lm = tid / 4, lnd = (tid % 4) * 8;  // dY tile: 64 m x 32 n
  const int lnw = tid / 8, lk = (tid % 8) * 8;  // W~ tile: 32 n x 64 k
  float v[8];
  uint32_t bits;
  bool w_in;
  auto load = [&](int64_t nb) {  // this thread's part of the next step
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (m0 + lm < M && nb + lnd < N) load8<kBf16>(dY, (m0 + lm) * N + nb + lnd, v);
    w_in = nb + lnw < N;
    bits = w_in ? codes16(packed, Kb, nb + lnw, k0 + lk) : 0u;
  };
  load(0);
  __syncthreads();
  int b = 0;
  for (int64_t nb = 0; nb < N; nb += kBK, b ^= 1) {
    float w[8] = {};
    if (w_in) decode8<D>(bits, sA, sB, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      Ds[b][lnd + i][lm] = v[i];
      Ws[b][lnw][lk + i] = w[i];
    }
    __syncthreads();
    if (nb + kBK < N) load(nb + kBK);
    mac_step(Ds[b], Ws[b], ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, k = k0 + tx * 4 + j;
      if (m < M) store_out<kBf16>(dX, m * K + k, acc[i][j]);
    }
}

// ---------------------------------------------------------------- smaller tiles
// The forward and dX (fp32 activations) in tiles of kTile x kTile outputs, kTile / 16
// squared per thread, the next 64 contraction steps loaded while this one's products
// run.  Every output is the same sequence of fused multiply-adds as in the 64 x 64
// kernels, so it has the same bits whatever the tile.  16: a row's 64 steps are read
// by 16 lanes.  32: a thread reads whole sectors of one row and a warp's lanes take
// different rows, so that the transposed stores hit different banks (in the 64 x 64
// kernels they meet four at a time).
constexpr int kDeep = 64;  // contraction steps per chunk

template <int D, int kTile, bool kForward>  // kForward: C = X W~^T over k; else C = dY W~ over n
__global__ void __launch_bounds__(kThreads) simt_tile_kernel(
    const float* __restrict__ X, int64_t M, const uint8_t* __restrict__ packed, int64_t N, int64_t K,
    const float* __restrict__ A, const float* __restrict__ B, float* __restrict__ C) {
  constexpr int kR = kTile / 16;     // outputs per thread and dimension
  constexpr int kPitch = kTile == 16 ? 17 : 36;
  constexpr int kX = kTile * kDeep / kThreads;  // activations staged per thread: 4 or 8
  static_assert(kTile == 16 || kTile == 32, "tiles");
  __shared__ float sA[D * D], sB[D];
  __shared__ __align__(16) float Xs[2][kDeep][kPitch], Ws[2][kDeep][kPitch];
  load_AB<D>(A, B, sA, sB);
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const int64_t m0 = int64_t(blockIdx.y) * kTile, c0 = int64_t(blockIdx.x) * kTile;
  const int64_t depth = kForward ? K : N, cols = kForward ? N : K, Kb = K / 4;
  const int xr = kTile == 16 ? tid / 16 : tid % kTile;
  const int xc = kTile == 16 ? tid % 16 * 4 : tid / kTile * kX;
  // eight weights: forward kTile rows x 64 k, dX 64 rows x kTile k
  const int wr = !kForward ? tid / (kTile / 8) : (kTile == 16 ? tid / 8 : tid % kTile);
  const int wc = !kForward ? tid % (kTile / 8) * 8 : (kTile == 16 ? tid % 8 * 8 : tid / kTile * 8);
  const bool has_w = tid < kTile * 8;
  float xv[kX];
  uint32_t bits = 0;
  bool w_in = false;
  auto load = [&](int64_t d0) {
#pragma unroll
    for (int q = 0; q < kX; q += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (m0 + xr < M && d0 + xc + q < depth)
        v = *reinterpret_cast<const float4*>(X + (m0 + xr) * depth + d0 + xc + q);
      xv[q] = v.x; xv[q + 1] = v.y; xv[q + 2] = v.z; xv[q + 3] = v.w;
    }
    const int64_t n = kForward ? c0 + wr : d0 + wr, k = kForward ? d0 + wc : c0 + wc;
    w_in = has_w && n < N && k < K;
    bits = w_in ? codes16(packed, Kb, n, k) : 0u;
  };
  auto store = [&](int b) {
#pragma unroll
    for (int i = 0; i < kX; ++i) Xs[b][xc + i][xr] = xv[i];
    if (has_w) {
      float w[8] = {};
      if (w_in) decode8<D>(bits, sA, sB, w);
      if constexpr (kForward) {
#pragma unroll
        for (int i = 0; i < 8; ++i) Ws[b][wc + i][wr] = w[i];
      } else if constexpr (kTile == 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) Ws[b][wr][wc + i] = w[i];
      } else {
        float4* o = reinterpret_cast<float4*>(&Ws[b][wr][wc]);
        o[0] = make_float4(w[0], w[1], w[2], w[3]);
        o[1] = make_float4(w[4], w[5], w[6], w[7]);
      }
    }
  };
  float acc[kR][kR] = {};
  load(0);
  __syncthreads();  // A, B
  int b = 0;
  for (int64_t d0 = 0; d0 < depth; d0 += kDeep, b ^= 1) {
    store(b);
    __syncthreads();
    if (d0 + kDeep < depth) load(d0 + kDeep);
#pragma unroll
    for (int kk = 0; kk < kDeep; ++kk) {
      float a[kR], w[kR];
      if constexpr (kR == 2) {
        const float2 p = *reinterpret_cast<const float2*>(&Xs[b][kk][2 * ty]);
        const float2 q = *reinterpret_cast<const float2*>(&Ws[b][kk][2 * tx]);
        a[0] = p.x; a[1] = p.y; w[0] = q.x; w[1] = q.y;
      } else {
        a[0] = Xs[b][kk][ty];
        w[0] = Ws[b][kk][tx];
      }
#pragma unroll
      for (int i = 0; i < kR; ++i)
#pragma unroll
        for (int j = 0; j < kR; ++j) acc[i][j] = fmaf(a[i], w[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int j = 0; j < kR; ++j) {
      const int64_t m = m0 + ty * kR + i, c = c0 + tx * kR + j;
      if (m < M && c < cols) C[m * cols + c] = acc[i][j];
    }
}

template <int kTile, bool kForward>
cudaError_t launch_tile(const float* x, int64_t M, const uint8_t* packed, int64_t N, int64_t K, int d,
                        const float* A, const float* B, float* c, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(kForward ? N : K, kTile)),
                  static_cast<unsigned>(ceil_div(M, kTile)));
  switch (d) {
    case 1: simt_tile_kernel<1, kTile, kForward><<<grid, kThreads, 0, s>>>(x, M, packed, N, K, A, B, c); break;
    case 2: simt_tile_kernel<2, kTile, kForward><<<grid, kThreads, 0, s>>>(x, M, packed, N, K, A, B, c); break;
    case 4: simt_tile_kernel<4, kTile, kForward><<<grid, kThreads, 0, s>>>(x, M, packed, N, K, A, B, c); break;
    default: simt_tile_kernel<8, kTile, kForward><<<grid, kThreads, 0, s>>>(x, M, packed, N, K, A, B, c); break;
  }
  return cudaGetLastError();
}

// The tile: the largest that still gives the SMs one or two CTAs each.  Measured
// (16, 32, 64): 16 x 512 -> 512 7.8, 12.9, 24 us; 128 x 512 -> 1024 23, 14.5, 25;
// 100 x 1024 -> 1024 44, 28, 47; 512 x 512 -> 512 39, 25, 25; 512 x 1024 -> 1024 148, 92, 47.
int tile_of(int64_t M, int64_t cols) {
  if (ceil_div(M, 16) * ceil_div(cols, 16) <= kNumSMsB200) return 16;
  if (ceil_div(M, 32) * ceil_div(cols, 32) <= 2 * kNumSMsB200) return 32;
  return 64;
}

// ---------------------------------------------------------------- dW epilogue
template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads) simt_dw_kernel(
    const void* __restrict__ X, const void* __restrict__ dY, int64_t M,
    const uint8_t* __restrict__ packed, const uint8_t* __restrict__ mask, int64_t N, int64_t K,
    const float* __restrict__ A, float* __restrict__ dWp, float* __restrict__ partials) {
  constexpr int NP = D * D + D;
  __shared__ float sA[D * D];
  __shared__ __align__(16) float buf[2][2][kBK][kT + 4];  // dY tiles [m][n], X tiles [m][k]; then G
  __shared__ float red[kThreads / 32][NP];
  for (int i = threadIdx.x; i < D * D; i += blockDim.x) sA[i] = A[i];
  const int tid = threadIdx.x;
  const int64_t n0 = int64_t(blockIdx.y) * kT, k0 = int64_t(blockIdx.x) * kT;
  const int ty = tid / 16, tx = tid % 16;
  const int64_t Kb = K / 4;
  float acc[4][4] = {};
  const int lm = tid / 8, lc = (tid % 8) * 8;
  float dv[8], xv[8];
  auto load = [&](int64_t mb) {  // this thread's part of the next step
#pragma unroll
    for (int i = 0; i < 8; ++i) dv[i] = xv[i] = 0.f;
    if (mb + lm < M && n0 + lc < N) load8<kBf16>(dY, (mb + lm) * N + n0 + lc, dv);
    if (mb + lm < M) load8<kBf16>(X, (mb + lm) * K + k0 + lc, xv);
  };
  load(0);
  int b = 0;
  for (int64_t mb = 0; mb < M; mb += kBK, b ^= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      buf[0][b][lm][lc + i] = dv[i];
      buf[1][b][lm][lc + i] = xv[i];
    }
    __syncthreads();
    if (mb + kBK < M) load(mb + kBK);
    mac_step(buf[0][b], buf[1][b], ty, tx, acc);
  }
  __syncthreads();
  // G tile -> shared memory, reusing the operand buffers (64 x 65 <= 4 x 32 x 68 floats)
  float* Gs = &buf[0][0][0][0];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) Gs[(ty * 4 + i) * (kT + 1) + tx * 4 + j] = acc[i][j];
  __syncthreads();

  float pa[D * D], pb[D];
#pragma unroll
  for (int i = 0; i < D * D; ++i) pa[i] = 0.f;
#pragma unroll
  for (int i = 0; i < D; ++i) pb[i] = 0.f;
  constexpr int VPR = kT / D;  // vectors per tile row
  for (int v = tid; v < kT * VPR; v += kThreads) {
    const int lr = v / VPR, gv = v % VPR;
    const int64_t n = n0 + lr;
    if (n >= N) continue;
    const int64_t kv = k0 + int64_t(gv) * D;
    float G[D];
#pragma unroll
    for (int i = 0; i < D; ++i) G[i] = Gs[lr * (kT + 1) + gv * D + i];
    float z[D];
    uint32_t mbits = 0;
#pragma unroll
    for (int j = 0; j < D; ++j) {
      const int64_t k = kv + j;
      z[j] = static_cast<float>((packed[n * Kb + (k >> 2)] >> (2 * (k & 3))) & 3u);
      if (mask != nullptr) mbits |= ((mask[n * (K / 8) + (k >> 3)] >> (k & 7)) & 1u) << j;
    }
#pragma unroll
    for (int i = 0; i < D; ++i) {
      pb[i] += G[i];
#pragma unroll
      for (int j = 0; j < D; ++j) pa[i * D + j] = fmaf(G[i], z[j], pa[i * D + j]);
    }
    if (dWp != nullptr) {
#pragma unroll
      for (int j = 0; j < D; ++j) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < D; ++i) s = fmaf(sA[i * D + j], G[i], s);
        dWp[n * K + kv + j] = ((mbits >> j) & 1u) ? s : 0.f;
      }
    }
  }
  // fixed-order block reduction of the D*D + D partials
  const int warp = tid >> 5, lane = tid & 31;
#pragma unroll
  for (int e = 0; e < NP; ++e) {
    float x = e < D * D ? pa[e] : pb[e - D * D];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_down_sync(0xffffffffu, x, off);
    if (lane == 0) red[warp][e] = x;
  }
  __syncthreads();
  if (tid < NP) {
    float s = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) s += red[w][tid];
    const int64_t tile = int64_t(blockIdx.y) * gridDim.x + blockIdx.x;
    partials[tile * NP + tid] = s;
  }
}

// one CTA per output element; fp64, fixed order
__global__ void __launch_bounds__(256) reduce_partials_kernel(const float* partials,
                                                              int64_t num_parts, int np, int dd,
                                                              float* __restrict__ dA,
                                                              float* __restrict__ dB) {
  __shared__ double red[256];
  const int e = blockIdx.x;
  double s = 0.0;
  griddep_wait();  // the partials come from the kernel just before this one (see ld_global_f32)
  griddep_launch_dependents();
  for (int64_t p = threadIdx.x; p < num_parts; p += 256) s += ld_global_f32(partials + p * np + e);
  red[threadIdx.x] = s;
  __syncthreads();
  for (int off = 128; off > 0; off >>= 1) {
    if (threadIdx.x < off) red[threadIdx.x] += red[threadIdx.x + off];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    if (e < dd) dA[e] = static_cast<float>(red[0]);
    else dB[e - dd] = static_cast<float>(red[0]);
  }
}

}  // namespace

#define LCVQ_DISPATCH_D(d, BF, KERNEL, GRID, ...)                                    \
  do {                                                                               \
    switch (d) {                                                                     \
      case 1: if (BF) KERNEL<1, true><<<GRID, kThreads, 0, s>>>(__VA_ARGS__);        \
              else KERNEL<1, false><<<GRID, kThreads, 0, s>>>(__VA_ARGS__); break;   \
      case 2: if (BF) KERNEL<2, true><<<GRID, kThreads, 0, s>>>(__VA_ARGS__);        \
              else KERNEL<2, false><<<GRID, kThreads, 0, s>>>(__VA_ARGS__); break;   \
      case 4: if (BF) KERNEL<4, true><<<GRID, kThreads, 0, s>>>(__VA_ARGS__);        \
              else KERNEL<4, false><<<GRID, kThreads, 0, s>>>(__VA_ARGS__); break;   \
      default: if (BF) KERNEL<8, true><<<GRID, kThreads, 0, s>>>(__VA_ARGS__);       \
              else KERNEL<8, false><<<GRID, kThreads, 0, s>>>(__VA_ARGS__); break;   \
    }                                                                                \
  } while (0)

cudaError_t launch_simt_forward(const void* X, bool bf16, int64_t M, const uint8_t* packed,
                                int64_t d_out, int64_t d_in, int d, const float* A,
                                const float* B, void* Y, cudaStream_t s, int* launches) {
  if (const int tile = bf16 ? 64 : tile_of(M, d_out); tile < 64) {
    ++*launches;
    const float* x = static_cast<const float*>(X);
    float* y = static_cast<float*>(Y);
    return tile == 16 ? launch_tile<16, true>(x, M, packed, d_out, d_in, d, A, B, y, s)
                      : launch_tile<32, true>(x, M, packed, d_out, d_in, d, A, B, y, s);
  }
  const dim3 grid(static_cast<unsigned>(ceil_div(d_out, kT)), static_cast<unsigned>(ceil_div(M, kT)));
  LCVQ_DISPATCH_D(d, bf16, simt_forward_kernel, grid, X, M, packed, d_out, d_in, A, B, Y);
  ++*launches;
  return cudaGetLastError();
}

cudaError_t launch_simt_backward_dx(const void* dY, bool bf16, int64_t M, const uint8_t* packed,
                                    int64_t d_out, int64_t d_in, int d, const float* A,
                                    const float* B, void* dX, cudaStream_t s, int* launches) {
  if (const int tile = bf16 ? 64 : tile_of(M, d_in); tile < 64) {
    ++*launches;
    const float* y = static_cast<const float*>(dY);
    float* x = static_cast<float*>(dX);
    return tile == 16 ? launch_tile<16, false>(y, M, packed, d_out, d_in, d, A, B, x, s)
                      : launch_tile<32, false>(y, M, packed, d_out, d_in, d, A, B, x, s);
  }
  const dim3 grid(static_cast<unsigned>(d_in / kT), static_cast<unsigned>(ceil_div(M, kT)));
  LCVQ_DISPATCH_D(d, bf16, simt_dx_kernel, grid, dY, M, packed, d_out, d_in, A, B, dX);
  ++*launches;
  return cudaGetLastError();
}

int64_t simt_dw_num_tiles(int64_t d_out, int64_t d_in) { return ceil_div(d_out, kT) * (d_in / kT); }

cudaError_t launch_simt_backward_dw(const void* X, const void* dY, bool bf16, int64_t M,
                                    const uint8_t* packed, const uint8_t* mask_bits,
                                    int64_t d_out, int64_t d_in, int d, const float* A,
                                    float* dWp, float* partials, cudaStream_t s, int* launches) {
  const dim3 grid(static_cast<unsigned>(d_in / kT), static_cast<unsigned>(ceil_div(d_out, kT)));
  LCVQ_DISPATCH_D(d, bf16, simt_dw_kernel, grid, X, dY, M, packed, mask_bits, d_out, d_in, A,
                  dWp, partials);
  ++*launches;
  return cudaGetLastError();
}

cudaError_t launch_reduce_partials(const float* partials, int64_t num_parts, int d, float* dA,
                                   float* dB, cudaStream_t s, int* launches) {
  const int np = d * d + d;
  ++*launches;
  return launch_pdl(reduce_partials_kernel, np, 256, 0, s, partials, num_parts, np, d * d, dA, dB);
}

}  // namespace lcvq
