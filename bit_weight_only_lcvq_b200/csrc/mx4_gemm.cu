// Product of two mx4 matrices for many tokens, on the block-scaled tensor-core
// MMA of sm_100a (tcgen05.mma kind::mxf4): Y = X W^T with the packed nibbles and
// scale bytes as they lie in memory.  Nothing is decoded: TMA brings 256
// positions of 128 tokens and 192 weight rows (128 bytes a row, SW128) and bulk
// copies their 512-byte scale tiles into a stage; the MMA thread copies the scale
// tiles from shared memory to TMEM and issues four MMAs of 64 positions.
//
//   warp 0      producer (TMA and bulk copies)
//   warp 1      TMEM allocation, scale copies, MMA issue
//   warps 2-5   epilogue: TMEM -> registers -> Y
//
// What bounds it: the tensor cores (an MMA of 128 x 192 x 64 takes 96 cycles at
// the nominal rate; operand reads from shared memory are 106 of its 128 bytes
// a cycle).  Why 192 columns: two accumulators of 192 columns, so that a tile's
// epilogue overlaps the next tile's MMAs, leave 128 columns of TMEM, and the
// scales of a stage take 24 of them, one slot per stage of the ring (a slot is
// rewritten only after the MMAs of its stage have completed, as the stage
// itself).  Two accumulators of 256 would leave no room for scales.
//
// A 192-row tile of weights starts at row 0 or 64 of a 128-row scale tile and
// ends within the next one: both are copied, and an odd tile's scales start two
// columns (64 rows) in.
#include "common.cuh"
#include "gemv_common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "sm100.cuh"

namespace lcvq {

using namespace sm100;

namespace {

constexpr int BM = 128;
constexpr int BN = 192;
constexpr int BK = 256;            // positions per stage: 128 bytes a row
constexpr int STAGES = 5;
constexpr int A_BYTES = BM * 128;
constexpr int B_BYTES = BN * 128;
constexpr int SF_BYTES = 6 * mx::kTileBytes;  // A: 2 tiles (k); B: 2 (rows) x 2 (k)
constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SF_BYTES;
static_assert(STAGE_BYTES % 1024 == 0, "swizzled tiles start on 1024-byte boundaries");
constexpr int SF_COLS = 24;        // TMEM columns of a stage's scales: A 2 x 4, B 2 x 8
constexpr int kTmemCols = 512;
static_assert(2 * BN + STAGES * SF_COLS <= kTmemCols, "accumulators and scales fit TMEM");
constexpr int kThreads = 32 * 6;
constexpr size_t kSmemBytes = 1024 + size_t(STAGES) * STAGE_BYTES + 256;

struct Params {
  int64_t M, N, K;
  const uint8_t* xs;
  const uint8_t* ws;
  void* Y;
  unsigned int* err;
};

__device__ __forceinline__ void fail(const Params& p, volatile int* abort_flag, unsigned site) {
  record_error(p.err, LCVQ_ERR_DEVICE_TIMEOUT, site);
  *abort_flag = 1;
}

template <bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + size_t(STAGES) * STAGE_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t m_tiles = ceil_div(p.M, BM), n_tiles = ceil_div(p.N, BN);
  const int64_t tiles = m_tiles * n_tiles;
  const int64_t kblocks = ceil_div(p.K, BK);
  const int64_t tiles_k = mx::scale_tiles_k(p.K);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);  // one arrive per epilogue warp
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  griddep_wait();  // the operands may come from the kernel just before this one
  griddep_launch_dependents();
  const long long lim = wait_limit(p.err);
  auto warp_abort = [&]() { return __shfl_sync(0xffffffffu, *abort_flag, 0) != 0; };
  // bands of 16 token tiles: the CTAs that run together share both operands in L2
  auto coords = [&](int64_t tile, int64_t& mt, int64_t& nt) {
    const int64_t per_band = 16 * n_tiles, b = tile / per_band, r = tile % per_band;
    const int64_t rows = (b + 1) * 16 <= m_tiles ? 16 : m_tiles - b * 16;
    mt = b * 16 + r % rows;
    nt = r / rows;
  };

  if (warp == 0) {
    if (lane == 0) {
      const int64_t w_tiles = ceil_div(p.N, 128);
      int s = 0;
      uint32_t ph = 0;
      int64_t issued = 0;
      for (int64_t tile = blockIdx.x; tile < tiles && !*abort_flag; tile += gridDim.x) {
        int64_t mt, nt;
        coords(tile, mt, nt);
        // the second scale tile of weight rows may lie beyond the last: any tile
        // stands in for it (its rows of D are not stored)
        const int64_t w0 = nt * BN >> 7, w1 = w0 + 1 < w_tiles ? w0 + 1 : w0;
        for (int64_t kb = 0; kb < kblocks; ++kb) {
          if (!mbar_wait(&empty[s], ph ^ 1, lim)) { fail(p, abort_flag, 31); break; }
          if (*abort_flag) break;
          ++issued;
          mbar_arrive_expect_tx(&full[s], STAGE_BYTES);
          uint8_t* st = smem + size_t(s) * STAGE_BYTES;
          tma_load_2d(&tmA, &full[s], st, static_cast<int>(kb) * 128, static_cast<int>(mt) * BM);
          tma_load_2d(&tmB, &full[s], st + A_BYTES, static_cast<int>(kb) * 128, static_cast<int>(nt) * BN);
          const uint32_t sf = smem_u32(st) + A_BYTES + B_BYTES;
          const int64_t k0 = 2 * kb, k1 = k0 + 1 < tiles_k ? k0 + 1 : k0;  // the last may not exist: unused
          bulk_load(sf, p.xs + (mt * tiles_k + k0) * mx::kTileBytes, mx::kTileBytes, &full[s]);
          bulk_load(sf + 512, p.xs + (mt * tiles_k + k1) * mx::kTileBytes, mx::kTileBytes, &full[s]);
          bulk_load(sf + 1024, p.ws + (w0 * tiles_k + k0) * mx::kTileBytes, mx::kTileBytes, &full[s]);
          bulk_load(sf + 1536, p.ws + (w1 * tiles_k + k0) * mx::kTileBytes, mx::kTileBytes, &full[s]);
          bulk_load(sf + 2048, p.ws + (w0 * tiles_k + k1) * mx::kTileBytes, mx::kTileBytes, &full[s]);
          bulk_load(sf + 2560, p.ws + (w1 * tiles_k + k1) * mx::kTileBytes, mx::kTileBytes, &full[s]);
          if (++s == STAGES) { s = 0; ph ^= 1; }
        }
      }
      if (*abort_flag) {  // no copy may land in shared memory after the CTA exits
        for (int64_t n = issued - 1; n >= 0 && n >= issued - STAGES; --n)
          mbar_wait(&full[n % STAGES], static_cast<uint32_t>((n / STAGES) & 1), kDefaultWaitLimit);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      int64_t local = 0;
      bool issued = false;
      for (int64_t tile = blockIdx.x; tile < tiles && !*abort_flag; tile += gridDim.x, ++local) {
        int64_t mt, nt;
        coords(tile, mt, nt);
        const int buf = static_cast<int>(local & 1);
        const uint32_t use = static_cast<uint32_t>(local >> 1);
        if (!mbar_wait(&tempty[buf], (use & 1) ^ 1, lim)) { fail(p, abort_flag, 32); break; }
        tc_fence_after();
        const uint32_t dt = tmem + buf * BN;
        const uint32_t b_off = nt & 1 ? 2 : 0;  // an odd tile starts 64 rows into its scale tile
        bool ok = true;
        for (int64_t kb = 0; kb < kblocks; ++kb) {
          if (!mbar_wait(&full[s], ph, lim)) { fail(p, abort_flag, 33); ok = false; break; }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem + size_t(s) * STAGE_BYTES);
          const uint32_t b0 = a0 + A_BYTES, sf = b0 + B_BYTES;
          const uint32_t ta = tmem + 2 * BN + s * SF_COLS, tb = ta + 8;
#pragma unroll
          for (int i = 0; i < 2; ++i) tmem_copy_scales(ta + 4 * i, sdesc_scales(sf + 512 * i));
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_copy_scales(tb + 4 * i, sdesc_scales(sf + 1024 + 512 * i));
          const int64_t left = p.K - kb * BK;
#pragma unroll
          for (int k = 0; k < BK / 64; ++k) {
            if (k * 64 < left)  // K is a multiple of 64
              mma_mxf4(dt, sdesc_sw128(a0 + k * 32, 16, 1024), sdesc_sw128(b0 + k * 32, 16, 1024),
                       idesc_mxf4(BM, BN, k & 1), ta + 4 * (k >> 1), tb + 8 * (k >> 1) + b_off,
                       (kb | k) != 0 ? 1u : 0u);
          }
          issued = true;
          mma_commit(&empty[s]);
          if (++s == STAGES) { s = 0; ph ^= 1; }
        }
        if (!ok) break;
        mma_commit(&tfull[buf]);
      }
      if (issued) {  // no MMA may still run when TMEM is released
        mma_commit(drain);
        if (!mbar_wait(drain, 0, kDefaultWaitLimit)) fail(p, abort_flag, 34);
      }
    }
  } else {
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    int64_t local = 0;
    for (int64_t tile = blockIdx.x; tile < tiles && !warp_abort(); tile += gridDim.x, ++local) {
      int64_t mt, nt;
      coords(tile, mt, nt);
      const int buf = static_cast<int>(local & 1);
      const uint32_t use = static_cast<uint32_t>(local >> 1);
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[buf], use & 1, lim))) {  // one outcome per warp
        fail(p, abort_flag, 35);
        break;
      }
      tc_fence_after();
      const int64_t m = mt * BM + row;
      const uint32_t tbase = tmem + buf * BN + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        uint32_t r[32];
        tmem_ld32(tbase + c * 32, r);
        tmem_ld_wait();
        const int64_t n0 = nt * BN + c * 32;
        if (m >= p.M) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // N is a multiple of 8
          if (n0 + 8 * q >= p.N) break;
          if constexpr (kF32) {
            float4* y = reinterpret_cast<float4*>(static_cast<float*>(p.Y) + m * p.N + n0 + 8 * q);
            y[0] = make_float4(__uint_as_float(r[8 * q]), __uint_as_float(r[8 * q + 1]),
                               __uint_as_float(r[8 * q + 2]), __uint_as_float(r[8 * q + 3]));
            y[1] = make_float4(__uint_as_float(r[8 * q + 4]), __uint_as_float(r[8 * q + 5]),
                               __uint_as_float(r[8 * q + 6]), __uint_as_float(r[8 * q + 7]));
          } else {
            uint4 v;
            v.x = pack_bf16x2(__uint_as_float(r[8 * q]), __uint_as_float(r[8 * q + 1]));
            v.y = pack_bf16x2(__uint_as_float(r[8 * q + 2]), __uint_as_float(r[8 * q + 3]));
            v.z = pack_bf16x2(__uint_as_float(r[8 * q + 4]), __uint_as_float(r[8 * q + 5]));
            v.w = pack_bf16x2(__uint_as_float(r[8 * q + 6]), __uint_as_float(r[8 * q + 7]));
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.Y) + m * p.N + n0 + 8 * q) = v;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[buf]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_mx4_gemm(const uint8_t* xq, const uint8_t* xs, int64_t M, const uint8_t* wq,
                            const uint8_t* ws, int64_t N, int64_t K, void* Y, bool f32,
                            unsigned int* err, cudaStream_t s, int* launches) {
  CUtensorMap ta, tb;
  if (!make_tensor_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, K / 2, M, K / 2, 128, BM, true) ||
      !make_tensor_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, wq, K / 2, N, K / 2, 128, BN, true))
    return cudaErrorInvalidValue;
  auto kern = f32 ? mx4_gemm_kernel<true> : mx4_gemm_kernel<false>;
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), kSmemBytes);
      e != cudaSuccess)
    return e;
  const int64_t tiles = ceil_div(M, BM) * ceil_div(N, BN);
  const Params p{M, N, K, xs, ws, Y, err};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles < tc_max_grid() ? tiles : tc_max_grid()), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ++*launches;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, kern, ta, tb, p); e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace lcvq
