// Product of two mx4 matrices for many tokens, on the block-scaled tensor-core
// MMA of sm_100a (tcgen05.mma kind::mxf4): Y = X W^T with the packed nibbles and
// scale bytes as they lie in memory; nothing is decoded.  A CTA pair (cta_group::2)
// computes 256 tokens x 192 weight rows: each CTA loads 128 tokens and 96 weight
// rows of 256 positions (128 bytes a row, SW128) and the scale tiles of its tokens
// and of all 192 weight rows; the even CTA copies the scales of both from shared
// memory to TMEM and issues the MMAs of 64 positions for both.
//
//   warp 0      producer (TMA, both CTAs; all bytes count on the even CTA's barrier)
//   warp 1      TMEM allocation; in the even CTA MMA issue
//   warp 2      in the even CTA scale copies to TMEM
//   warps 3-6   epilogue: TMEM -> registers -> Y
//
// What bounds it: the tensor cores and the shared memory that feeds them.  On one
// CTA a tile of 128 x 192 reads 10 KB for each MMA of 96 cycles (nominal), close
// to the 128 bytes a cycle that shared memory gives before TMA's writes; the pair
// reads 7 KB.  Why 192 columns: two accumulators of 192, so that a tile's epilogue
// overlaps the next tile's MMAs, leave 128 columns of TMEM for scales, 24 for
// each 256 positions; two accumulators of 256 would leave none.  The scales have
// five slots and the ring six stages: before a slot is rewritten its MMAs, five
// blocks back, have completed (the same barrier that frees their stage).
//
// Measured: 2048 x 4096 -> 11008 42 us (4.4 PFLOP/s), 8192 x 14336 -> 4096 185 us (5.2);
// without its operand copies the second would take 172.  Single CTAs took 75 and 338,
// pairs whose one lane issued everything 91 and 425 (see elect_one).
//
// A 192-row tile of weights starts at row 0 or 64 of a 128-row scale tile and
// ends within the next one: both are copied, and an odd tile's scales start two
// columns (64 rows) in.
#include "common.cuh"
#include "gemv_common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "pdl.cuh"
#include "sm100.cuh"

namespace lcvq {

using namespace sm100;

namespace {

constexpr int BM = 128;            // tokens per CTA, 256 per pair
constexpr int BN = 192;            // weight rows per pair, 96 loaded by each CTA
constexpr int BK = 256;            // positions per stage: 128 bytes a row
constexpr int STAGES = 6;
constexpr int A_BYTES = BM * 128;
constexpr int B_BYTES = BN / 2 * 128;
constexpr int SF_BYTES = 6 * mx::kTileBytes;  // A: 2 tiles (k); B: 2 (rows) x 2 (k)
constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SF_BYTES;
static_assert(STAGE_BYTES % 1024 == 0, "swizzled tiles start on 1024-byte boundaries");
constexpr int SF_COLS = 24;        // TMEM columns of a block's scales: A 2 x 4, B 2 x 8
constexpr int SF_SLOTS = 5;
constexpr int kTmemCols = 512;
static_assert(2 * BN + SF_SLOTS * SF_COLS <= kTmemCols, "accumulators and scales fit TMEM");
static_assert(SF_SLOTS <= STAGES, "a slot's MMAs free a stage that has not been filled again");
constexpr int kThreads = 32 * 7;
// epilogue: two buffers of 32 rows x 128 bytes per warp
constexpr int OUT_BYTES = 32 * 128;
constexpr size_t kSmemBytes = 1024 + size_t(STAGES) * STAGE_BYTES + 8 * OUT_BYTES + 256;

struct Params {
  int64_t M, N, K;
  unsigned int* err;
};

__device__ __forceinline__ void fail(const Params& p, volatile int* abort_flag, unsigned site) {
  record_error(p.err, LCVQ_ERR_DEVICE_TIMEOUT, site);
  *abort_flag = 1;
}

template <bool kF32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSa, const __grid_constant__ CUtensorMap tmSb,
                    const __grid_constant__ CUtensorMap tmY, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out = smem + size_t(STAGES) * STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(out + 8 * OUT_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* sfull = empty + STAGES;  // even CTA: the stage's scales are in TMEM
  uint64_t* tfull = sfull + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* sdrain = drain + 1;
  // stages whose copies each CTA has issued, and whether the peer gave up a wait
  volatile int64_t* issued_here = reinterpret_cast<volatile int64_t*>(sdrain + 1);
  volatile int64_t* peer = issued_here + 1;  // its stages; negative (~stages): it gave up
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sdrain + 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int64_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int64_t m_tiles = ceil_div(p.M, 2 * BM), n_tiles = ceil_div(p.N, BN);
  const int64_t tiles = m_tiles * n_tiles;
  const int64_t kblocks = ceil_div(p.K, BK);
  const int64_t tiles_k = mx::scale_tiles_k(p.K);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sfull[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 8);  // even CTA: one arrive per epilogue warp of both
    }
    mbar_init(drain, 1);
    mbar_init(sdrain, 1);
    *issued_here = 0;
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, kTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
    tma_prefetch_map(&tmSa);
    tma_prefetch_map(&tmSb);
    tma_prefetch_map(&tmY);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers of both CTAs initialised before any cross-CTA use
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  griddep_wait();  // the operands may come from the kernel just before this one
  griddep_launch_dependents();
  const long long lim = wait_limit(p.err);
  auto warp_abort = [&]() { return __shfl_sync(0xffffffffu, *abort_flag, 0) != 0; };
  // bands of 8 token tiles: the CTAs that run together share both operands in L2
  auto coords = [&](int64_t tile, int64_t& mt, int64_t& nt) {
    const int64_t per_band = 8 * n_tiles, b = tile / per_band, r = tile % per_band;
    const int64_t rows = (b + 1) * 8 <= m_tiles ? 8 : m_tiles - b * 8;
    mt = b * 8 + r % rows;
    nt = r / rows;
  };

  if (warp == 0) {
    // the even CTA's full barriers and this CTA's stages as shared addresses: the
    // operands of the copies stay uniform over the warp (see elect_one)
    const uint32_t bar0 = mapa_shared(smem_u32(full), 0), st0 = smem_u32(smem);
    int s = 0;
    uint32_t ph = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int64_t tile = pair; tile < tiles && ok; tile += npairs) {
      int64_t mt, nt;
      coords(tile, mt, nt);
      const int row_a = static_cast<int>(mt * 2 * BM + rank * BM);
      const int row_b = static_cast<int>(nt * BN + rank * (BN / 2));
      // two scale tiles per block (the second, past the last column, is not used;
      // tiles past the last row scale rows of D that are not stored)
      const int64_t w0 = nt * BN >> 7;  // first scale tile of the weight rows
      int sa = static_cast<int>((mt * 2 + rank) * tiles_k), sb = static_cast<int>(w0 * tiles_k);
      const int sb_next = static_cast<int>(tiles_k);
      for (int kb = 0; kb < static_cast<int>(kblocks); ++kb, sa += 2, sb += 2) {
        const bool free_stage = mbar_wait(&empty[s], ph ^ 1, lim);
        if (!__all_sync(0xffffffffu, free_stage)) { fail(p, abort_flag, 31); ok = false; break; }
        if (warp_abort()) { ok = false; break; }
        const uint32_t bar = bar0 + 8 * s, st = st0 + s * STAGE_BYTES, sf = st + A_BYTES + B_BYTES;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * STAGE_BYTES);
          tma_load_2d_pair(&tmA, bar, st, kb * 128, row_a);
          tma_load_2d_pair(&tmB, bar, st + A_BYTES, kb * 128, row_b);
          tma_load_2d_pair(&tmSa, bar, sf, 0, sa);
          tma_load_2d_pair(&tmSb, bar, sf + 1024, 0, sb);
          tma_load_2d_pair(&tmSb, bar, sf + 2048, 0, sb + sb_next);
        }
        __syncwarp();
        ++issued;
        if (++s == STAGES) { s = 0; ph ^= 1; }
      }
    }
    if (lane == 0) *issued_here = issued;
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint32_t idesc0 = idesc_mxf4(2 * BM, BN, 0), idesc1 = idesc_mxf4(2 * BM, BN, 1);
      const uint64_t desc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
      const int last = static_cast<int>(p.K - (kblocks - 1) * BK);  // positions of the last block
      int s = 0, slot = 0;
      uint32_t ph = 0;
      int64_t local = 0;
      bool issued = false, ok = true;
      for (int64_t tile = pair; tile < tiles && ok && !warp_abort(); tile += npairs, ++local) {
        int64_t mt, nt;
        coords(tile, mt, nt);
        const int buf = static_cast<int>(local & 1);
        const uint32_t use = static_cast<uint32_t>(local >> 1);
        // the odd CTA's epilogue arrives from the other SM: acquire at cluster scope
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(&tempty[buf], (use & 1) ^ 1, lim))) {
          fail(p, abort_flag, 32);
          break;
        }
        tc_fence_after();
        const uint32_t dt = tmem + buf * BN;
        const uint32_t b_off = nt & 1 ? 2 : 0;  // an odd tile starts 64 rows into its scale tile
        for (int64_t kb = 0; kb < kblocks; ++kb) {
          // the operands, and their scales in TMEM
          if (!__all_sync(0xffffffffu, mbar_wait(&full[s], ph, lim) && mbar_wait(&sfull[s], ph, lim))) {
            fail(p, abort_flag, 33);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = desc0 + (static_cast<uint32_t>(s * STAGE_BYTES) >> 4), bd = ad + (A_BYTES >> 4);
          const uint32_t ta = tmem + 2 * BN + slot * SF_COLS, tb = ta + 8 + b_off;
          const int left = kb + 1 < kblocks ? BK : last;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < BK / 64; ++k)
              if (k * 64 < left)  // K is a multiple of 64
                mma_mxf4_pair(dt, ad + 2 * k, bd + 2 * k, k & 1 ? idesc1 : idesc0, ta + 4 * (k >> 1),
                              tb + 8 * (k >> 1), (kb | k) != 0 ? 1u : 0u);
            mma_commit_pair(&empty[s]);
          }
          __syncwarp();
          issued = true;
          if (++s == STAGES) { s = 0; ph ^= 1; }
          if (++slot == SF_SLOTS) slot = 0;
        }
        if (!ok) break;
        if (elect_one()) mma_commit_pair(&tfull[buf]);
        __syncwarp();
      }
      if (issued) {  // no MMA may still run when TMEM is released
        if (elect_one()) mma_commit_pair_here(drain);
        __syncwarp();
        if (!mbar_wait(drain, 0, kDefaultWaitLimit)) fail(p, abort_flag, 34);
      }
    }
  } else if (warp == 2) {
    if (rank == 0) {
      const uint64_t desc0 = sdesc_scales(smem_u32(smem) + A_BYTES + B_BYTES);
      int s = 0, slot = 0, old = 0;     // old: the stage of the block SF_SLOTS back
      uint32_t ph = 0, old_ph = 0;
      int filled = 0;
      bool ok = true, issued = false;
      for (int64_t tile = pair; tile < tiles && ok && !warp_abort(); tile += npairs) {
        for (int64_t kb = 0; kb < kblocks; ++kb) {
          // the stage has landed, and the MMAs that read this slot have completed
          bool ready = mbar_wait(&full[s], ph, lim);
          if (filled == SF_SLOTS) ready = ready && mbar_wait(&empty[old], old_ph, lim);
          if (!__all_sync(0xffffffffu, ready)) {
            fail(p, abort_flag, 36);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t sd = desc0 + (static_cast<uint32_t>(s * STAGE_BYTES) >> 4);
          const uint32_t ta = tmem + 2 * BN + slot * SF_COLS, tb = ta + 8;
          if (elect_one()) {
            // A: k half h to columns 4 h; B: rows tile w, k half h to columns 8 h + 4 w
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              tmem_copy_scales_pair(ta + 4 * h, sd + 32 * h);
              tmem_copy_scales_pair(tb + 8 * h, sd + 64 + 32 * h);
              tmem_copy_scales_pair(tb + 8 * h + 4, sd + 128 + 32 * h);
            }
            mma_commit_pair_here(&sfull[s]);
          }
          __syncwarp();
          issued = true;
          if (++s == STAGES) { s = 0; ph ^= 1; }
          if (++slot == SF_SLOTS) slot = 0;
          if (filled == SF_SLOTS) {
            if (++old == STAGES) { old = 0; old_ph ^= 1; }
          } else {
            ++filled;
          }
        }
      }
      if (issued) {  // no copy may still run when TMEM is released
        if (elect_one()) mma_commit_pair_here(sdrain);
        __syncwarp();
        if (!mbar_wait(sdrain, 0, kDefaultWaitLimit)) fail(p, abort_flag, 37);
      }
    }
  } else {
    // A warp's 32 rows leave in tiles of 128 bytes a row: written to shared memory
    // in the SW128 order (a row per lane, chunks permuted: no bank conflicts) and
    // stored by TMA, which clips what lies outside Y.  (Stored from registers, 16
    // bytes a lane in 32 different rows, Y set the pace:
    // 53 us against 47 at 2048 x 4096 -> 11008.)
    constexpr int kCols = kF32 ? 32 : 64;
    const int quarter = warp & 3;
    const uint32_t buf0 = smem_u32(out) + quarter * 2 * OUT_BYTES;
    int64_t local = 0;
    int ob = 0;
    for (int64_t tile = pair; tile < tiles && !warp_abort(); tile += npairs, ++local) {
      int64_t mt, nt;
      coords(tile, mt, nt);
      const int buf = static_cast<int>(local & 1);
      const uint32_t use = static_cast<uint32_t>(local >> 1);
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[buf], use & 1, lim))) {  // one outcome per warp
        fail(p, abort_flag, 35);
        break;
      }
      tc_fence_after();
      const int64_t m = mt * 2 * BM + int64_t(rank) * BM + quarter * 32;
      const uint32_t tbase = tmem + buf * BN + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < BN / kCols; ++c) {
        uint32_t r[kCols];
#pragma unroll
        for (int h = 0; h < kCols / 32; ++h)
          tmem_ld32(tbase + c * kCols + 32 * h, reinterpret_cast<uint32_t(&)[32]>(r[32 * h]));
        tmem_ld_wait();
        if (c == BN / kCols - 1) {  // the accumulator is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[buf]), 0));
        }
        if (lane == 0) bulk_wait_read<1>();  // the store before last has left this buffer
        __syncwarp();
        const uint32_t line = buf0 + ob * OUT_BYTES + lane * 128;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint4 v;
          if constexpr (kF32)
            v = make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
          else
            v = make_uint4(pack_bf16x2(__uint_as_float(r[8 * q]), __uint_as_float(r[8 * q + 1])),
                           pack_bf16x2(__uint_as_float(r[8 * q + 2]), __uint_as_float(r[8 * q + 3])),
                           pack_bf16x2(__uint_as_float(r[8 * q + 4]), __uint_as_float(r[8 * q + 5])),
                           pack_bf16x2(__uint_as_float(r[8 * q + 6]), __uint_as_float(r[8 * q + 7])));
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(line + ((q ^ (lane & 7)) << 4)),
                       "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                       : "memory");
        }
        fence_async_smem();
        __syncwarp();
        const int64_t n = nt * BN + c * kCols;
        if (lane == 0) {
          if (m < p.M && n < p.N)
            tma_store_2d(&tmY, buf0 + ob * OUT_BYTES, static_cast<int>(n), static_cast<int>(m));
          bulk_commit();
        }
        ob ^= 1;
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int64_t n = *issued_here;
    st_cluster_u64(mapa_shared(smem_u32(const_cast<int64_t*>(peer)), rank ^ 1),
                   static_cast<uint64_t>(*abort_flag ? ~n : n));
  }
  __syncwarp();
  cluster_sync();  // neither CTA leaves while its peer may still use its shared memory
  if (*abort_flag || *peer < 0) {
    // A wait gave up in one of the CTAs: no copy may land in shared memory after
    // either has left.  The even CTA's barriers count the bytes of both: the bytes
    // of stages that only one of them issued are made up for, and what was issued
    // is waited for.
    if (rank == 0 && threadIdx.x == 0) {
      const int64_t a = *issued_here, b = *peer < 0 ? ~*peer : *peer;
      for (int64_t n = b; n < a; ++n) mbar_complete_tx(&full[n % STAGES], STAGE_BYTES);
      for (int64_t n = a; n < b; ++n) mbar_arrive_expect_tx(&full[n % STAGES], STAGE_BYTES);
      const int64_t most = a > b ? a : b;
      for (int64_t n = most - 1; n >= 0 && n >= most - STAGES; --n)
        mbar_wait(&full[n % STAGES], static_cast<uint32_t>((n / STAGES) & 1), kDrainLimit);
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_mx4_gemm(const uint8_t* xq, const uint8_t* xs, int64_t M, const uint8_t* wq,
                            const uint8_t* ws, int64_t N, int64_t K, void* Y, bool f32,
                            unsigned int* err, cudaStream_t s, int* launches) {
  CUtensorMap ta, tb, sa, sb, ty;
  if (!make_tensor_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, K / 2, M, K / 2, 128, BM, true) ||
      !make_tensor_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, wq, K / 2, N, K / 2, 128, BN / 2, true) ||
      !mx::make_scale_map(&sa, xs, M, K) || !mx::make_scale_map(&sb, ws, N, K) ||
      !make_tensor_map_2d(&ty, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, Y, N, M,
                          N * (f32 ? 4 : 2), f32 ? 32 : 64, 32, true))
    return cudaErrorInvalidValue;
  auto kern = f32 ? mx4_gemm_kernel<true> : mx4_gemm_kernel<false>;
  if (cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kern), kSmemBytes);
      e != cudaSuccess)
    return e;
  const int64_t tiles = ceil_div(M, 2 * BM) * ceil_div(N, BN);
  const int64_t pairs = tiles < tc_max_grid() / 2 ? tiles : tc_max_grid() / 2;
  const Params p{M, N, K, err};
  ++*launches;
  return launch_pdl(kern, 2 * pairs, kThreads, kSmemBytes, s, ta, tb, sa, sb, ty, p);
}

}  // namespace lcvq
