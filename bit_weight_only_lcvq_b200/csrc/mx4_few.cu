// Product of two mx4 matrices for few tokens, on the block-scaled tensor-core
// MMA of sm_100a (tcgen05.mma kind::mxf4): Y = X W^T for M <= 128.
//
// The weights are the MMA's 128-row operand and the tokens its columns (8, 16,
// 32, 64 or 128 of them), so the packed weights go from memory to the tensor
// cores undecoded, whatever M is: an MMA of 64 positions reads 4 KB of them.
// What bounds it: the weights' bytes (17/32 B each) when they come from HBM, and
// at the usual sizes the chain of latencies launch - load - MMA - join. So K is
// split over a cluster of up to 8 CTAs, all of whose loads are in flight at once
// where the ring holds them; each CTA pushes its fp32 partial sums of 128 / S
// rows to the CTA of the cluster that owns those rows (distributed shared
// memory), and after one cluster barrier the owner adds them in CTA order and
// writes Y: one launch, no scratch in memory, the same bits every time.
// Measured (graph replay): 1 x 4096 -> 4096 5.3 us, 16 x 4096 -> 11008 6.5 us,
// 1 x 14336 -> 14336 19.1 us (5.7 TB/s of packed weights).  Decoding to bytes for the
// integer MMA of a warp instead took 9.8, 20.5 and 63 us, bound by its instructions.
//
//   warp 0      producer (TMA boxes of W, X and their scale tiles)
//   warp 1      TMEM allocation, scale copies, MMA issue
//   warps 2-5   TMEM -> registers -> the owners' shared memory
#include <type_traits>

#include "common.cuh"
#include "gemv_common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "sm100.cuh"

namespace lcvq {

using namespace sm100;

namespace {

constexpr int kRows = 128;       // weight rows per tile
constexpr int BK = 256;          // positions per stage: 128 bytes a row
constexpr int kThreads = 32 * 6;
constexpr int SF_COLS = 16;      // TMEM columns of a stage's scales: 2 x (4 + 4)

// The stages that two CTAs of an SM have room for.  The partial sums reuse them.
template <int NT>
struct Cfg {
  static constexpr int kStages = NT <= 16 ? 5 : (NT <= 64 ? 4 : 3);
  static constexpr int kW = kRows * 128;
  static constexpr int kX = NT * 128;
  static constexpr int kStage = kW + kX + 4 * mx::kTileBytes;  // scales: W k0, k1, X k0, k1
  static constexpr size_t kSmem = 1024 + size_t(kStages) * kStage + 256;
  static_assert(NT * kRows * 4 <= kStages * kStage, "the partial sums fit the stages");
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
  static constexpr int kCols = NT + kStages * SF_COLS <= 128 ? 128 : 256;  // TMEM
  static_assert(kStage % 1024 == 0 && NT + kStages * SF_COLS <= kCols, "layout");
};

struct Params {
  int64_t M, N, K;
  void* Y;
  unsigned int* err;
};

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(addr), "f"(v) : "memory");
}

template <int NT, bool kF32>
__global__ void __launch_bounds__(kThreads)
    mx4_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const __grid_constant__ CUtensorMap tmSw, const __grid_constant__ CUtensorMap tmSx,
                   const Params p, const int splits) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* red = reinterpret_cast<float*>(smem);  // [split][token][128 / S rows], once the stages are spent
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + size_t(C::kStages) * C::kStage);
  uint64_t* empty = full + C::kStages;
  uint64_t* done = empty + C::kStages;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = static_cast<int>(blockIdx.x) % splits;  // rank in the cluster
  const int64_t tile = blockIdx.x / splits;
  const int64_t tiles_k = mx::scale_tiles_k(p.K);
  const int64_t all = ceil_div(p.K, BK);
  // this CTA's k blocks: split, split + splits, ...
  const int64_t kblocks = (all - split + splits - 1) / splits;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::kCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tmW);
    tma_prefetch_map(&tmX);
    tma_prefetch_map(&tmSw);
    tma_prefetch_map(&tmSx);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  griddep_wait();  // the operands may come from the kernel just before this one
  griddep_launch_dependents();
  const long long lim = wait_limit(p.err);
  auto fail = [&](unsigned site) {
    record_error(p.err, LCVQ_ERR_DEVICE_TIMEOUT, site);
    *abort_flag = 1;
  };

  if (warp == 0) {
    int s = 0;
    uint32_t ph = 0;
    int64_t issued = 0;
    // two scale tiles per block (the second, past the last column, is not used)
    const int sw0 = static_cast<int>(tile * tiles_k);
    for (int64_t i = 0; i < kblocks; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ph ^ 1, lim))) { fail(41); break; }
      if (__shfl_sync(0xffffffffu, *abort_flag, 0) != 0) break;
      const int kb = static_cast<int>(split + i * splits);
      uint8_t* st = smem + size_t(s) * C::kStage;
      if (elect_one()) {
        mbar_arrive_expect_tx(&full[s], C::kStage);
        tma_load_2d(&tmW, &full[s], st, kb * 128, static_cast<int>(tile) * kRows);
        tma_load_2d(&tmX, &full[s], st + C::kW, kb * 128, 0);
        tma_load_2d(&tmSw, &full[s], st + C::kW + C::kX, 0, sw0 + 2 * kb);
        tma_load_2d(&tmSx, &full[s], st + C::kW + C::kX + 1024, 0, 2 * kb);
      }
      __syncwarp();
      ++issued;
      if (++s == C::kStages) { s = 0; ph ^= 1; }
    }
    // no copy may land in shared memory that is used again below or after the CTA
    // has left (the MMAs have waited for every copy, unless a wait gave up)
    for (int64_t n = issued - 1; n >= 0 && n >= issued - C::kStages; --n)
      mbar_wait(&full[n % C::kStages], static_cast<uint32_t>((n / C::kStages) & 1), kDrainLimit);
  } else if (warp == 1) {
    constexpr uint32_t idesc0 = idesc_mxf4(kRows, NT, 0), idesc1 = idesc_mxf4(kRows, NT, 1);
    const uint64_t desc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t sdesc0 = sdesc_scales(smem_u32(smem) + C::kW + C::kX);
    int s = 0;
    uint32_t ph = 0;
    bool issued = false;
    for (int64_t i = 0; i < kblocks; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], ph, lim))) { fail(42); break; }
      tc_fence_after();
      const uint32_t off = static_cast<uint32_t>(s * C::kStage) >> 4;
      const uint64_t ad = desc0 + off, bd = ad + (C::kW >> 4), sd = sdesc0 + off;
      const uint32_t ta = tmem + NT + s * SF_COLS, tb = ta + 8;
      const int64_t rest = p.K - (split + i * splits) * BK;
      const int left = rest < BK ? static_cast<int>(rest) : BK;
      if (elect_one()) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tmem_copy_scales(ta + 4 * h, sd + 32 * h);
          tmem_copy_scales(tb + 4 * h, sd + 64 + 32 * h);
        }
#pragma unroll
        for (int k = 0; k < BK / 64; ++k)
          if (k * 64 < left)  // K is a multiple of 64
            mma_mxf4(tmem, ad + 2 * k, bd + 2 * k, k & 1 ? idesc1 : idesc0, ta + 4 * (k >> 1),
                     tb + 4 * (k >> 1), (i | k) != 0 ? 1u : 0u);
        mma_commit(&empty[s]);
      }
      __syncwarp();
      issued = true;
      if (++s == C::kStages) { s = 0; ph ^= 1; }
    }
    if (issued) {
      if (elect_one()) mma_commit(done);
      __syncwarp();
      // the default limit: running MMAs finish in microseconds, and TMEM may be
      // released only after them
      if (!mbar_wait(done, 0, kDefaultWaitLimit)) fail(43);
    }
  }
  __syncwarp();  // warps 0 and 1 are whole again
  const int per = kRows / splits;  // rows that each CTA of the cluster owns
  __syncthreads();                 // the MMAs have completed
  tc_fence_after();
  // every CTA of the cluster is past its copies and MMAs: its stages may be
  // overwritten (after a wait that gave up, too: the producer waits for its copies)
  cluster_sync();
  if (warp >= 2) {
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t dst = mapa_shared(smem_u32(red + (split * NT) * per + row % per),
                                     static_cast<uint32_t>(row / per));
#pragma unroll 1
    for (int c = 0; c < NT && c < p.M; c += 8) {
      uint32_t r[8];
      tmem_ld8(base + c, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 8; ++j) st_cluster_f32(dst + (c + j) * per * 4, __uint_as_float(r[j]));
    }
    tc_fence_before();
  }
  cluster_sync();  // all partial sums have arrived
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols);
  }
  // rows of this CTA, four at a time (N is a multiple of 8, so four rows lie
  // inside it or outside together), summed over the splits in order
  const int quads = per / 4;
  for (int e = threadIdx.x; e < quads * static_cast<int>(p.M); e += kThreads) {
    const int m = e / quads, q = e % quads;
    const int64_t n = tile * kRows + split * per + 4 * q;
    if (n >= p.N) continue;
    float4 s = reinterpret_cast<const float4*>(red + m * per)[q];
    for (int w = 1; w < splits; ++w) {
      const float4 v = reinterpret_cast<const float4*>(red + (w * NT + m) * per)[q];
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    if constexpr (kF32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.Y) + m * p.N + n) = s;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.Y) + m * p.N + n) =
          make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

template <int NT, bool kF32>
cudaError_t launch_nt(const CUtensorMap (&t)[4], const Params& p, cudaStream_t s) {
  using C = Cfg<NT>;
  auto kern = mx4_few_kernel<NT, kF32>;
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), C::kSmem);
      e != cudaSuccess)
    return e;
  const int64_t tiles = ceil_div(p.N, kRows), kb = ceil_div(p.K, BK);
  const int64_t room = 2 * kNumSMsB200;  // two CTAs per SM
  int splits = 1;
  while (splits < 8 && 2 * splits <= kb && tiles * 2 * splits <= room) splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaError_t e = cudaLaunchKernelEx(&cfg, kern, t[0], t[1], t[2], t[3], p, splits); e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx4_few(const uint8_t* xq, const uint8_t* xs, int64_t M, const uint8_t* wq,
                           const uint8_t* ws, int64_t N, int64_t K, void* Y, bool f32,
                           unsigned int* err, cudaStream_t s, int* launches) {
  const int nt = M <= 8 ? 8 : (M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : 128)));
  CUtensorMap t[4];
  if (!make_tensor_map_2d(&t[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, wq, K / 2, N, K / 2, 128, kRows, true) ||
      !make_tensor_map_2d(&t[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, K / 2, M, K / 2, 128, nt, true) ||
      !mx::make_scale_map(&t[2], ws, N, K) || !mx::make_scale_map(&t[3], xs, M, K))
    return cudaErrorInvalidValue;
  const Params p{M, N, K, Y, err};
  ++*launches;
  auto go = [&](auto n) {
    constexpr int NT = decltype(n)::value;
    return f32 ? launch_nt<NT, true>(t, p, s) : launch_nt<NT, false>(t, p, s);
  };
  switch (nt) {
    case 8: return go(std::integral_constant<int, 8>{});
    case 16: return go(std::integral_constant<int, 16>{});
    case 32: return go(std::integral_constant<int, 32>{});
    case 64: return go(std::integral_constant<int, 64>{});
    default: return go(std::integral_constant<int, 128>{});
  }
}

}  // namespace lcvq
