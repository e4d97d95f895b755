// fp8_gemm.cu -- the product of two e4m3 operands with a scale per block of 128:
//
//   y[t, n] = sum_b sa[t, b] sw[n / 128, b] sum_{k in block b} a[t, k] w[n, k]
//
// a [T, K] (an activation: one scale per row and 128 columns), w [N, K] (a weight: one scale
// per 128 x 128 tile), both K-major.  The products of one block are summed by the tensor core
// in fp32 (tcgen05.mma kind::f8f6f4); because the scales change from block to block, each
// block's sums go to their own TMEM buffer, and the epilogue warps add them, scaled, into fp32
// registers while the tensor core works on the next block.  The only rounding to fewer bits is
// the output's.
//
// Two kernels.
// gemm_fp8_pair_kernel, for many outputs: a pair of CTAs shares a 256 x BN tile
// (tcgen05.mma.cta_group::2), so that a block of 128 columns costs each SM (128 + BN / 2) x 128
// bytes of operands for 128 x BN outputs.  What bounds it is the epilogue: every block is read
// back from TMEM and added in fp32 registers, and a block takes 740 cycles at BN = 256 against
// 512 of the tensor core's (510 at BN = 128); alone, without products or copies, the epilogue
// takes 700.  At 13112 x 12352 x 4096 a call takes 0.68 ms (1.9 PFLOP/s, at the power limit); a
// library product with one scale for everything takes 0.47-0.55 ms there.  The first version,
// tiles of 128 x 128 of single CTAs whose products one lane issued, took 1.14 ms.
// gemm_fp8_few_kernel, for few tokens: the weight's rows take the tensor core's M side, and a
// cluster splits K, so that a small product uses many SMs (8 x 6176 x 2048: 6.4 us).
#include <cuda_bf16.h>

#include <algorithm>

#include "fp8_ptx.cuh"
#include "layer_ops.h"
#include "tr_internal.h"

namespace tr {
namespace {

constexpr int BM = 128;
constexpr int BK = 128;              // one scale block; 128 bytes, one swizzle row

// 2D tensor map, 128-byte swizzle, of elements of `esz` bytes: boxes of 128 bytes x `box_rows`.
// What a load's box holds past the matrix reads as 0 (the last block of a K that is not a
// multiple of 128; rows past the end), and a store leaves it out.
bool make_tmap_2d(CUtensorMap *tm, const void *base, int esz, uint64_t inner, uint64_t rows,
                  uint64_t row_stride, uint32_t box_rows, std::string *err) {
  typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                             const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                             const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<Encode>(p);
  }();
  if (!fn) {
    if (err) *err = "cuTensorMapEncodeTiled is not available from the driver";
    return false;
  }
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {row_stride};   // bytes
  cuuint32_t box[2] = {(cuuint32_t)(128 / esz), box_rows};
  const CUtensorMapDataType type = esz == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : esz == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(tm, type, 2, const_cast<void *>(base), dims, strides,
                        box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    if (err) *err = "cuTensorMapEncodeTiled failed (" + std::to_string((int)r) + ")";
    return false;
  }
  return true;
}

// One thread's n consecutive outputs of row `row` from column c; 16-byte stores where the row
// allows them.
template <int NC>
__device__ __forceinline__ void store_row(const GemmFp8Launch &p, int row, int c, const float (&v)[NC]) {
  if (row >= p.T || c >= p.N) return;
  const int64_t off = (int64_t)row * p.y_stride + c;
  const bool whole = c + NC <= p.N;
  if (p.y_bf16) {
    __nv_bfloat16 *y = reinterpret_cast<__nv_bfloat16 *>(p.y) + off;
    if (whole && (reinterpret_cast<uintptr_t>(y) & 15) == 0) {
#pragma unroll
      for (int i = 0; i < NC; i += 8)
        *reinterpret_cast<uint4 *>(y + i) =
            make_uint4(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]),
                       pack_bf16x2(v[i + 4], v[i + 5]), pack_bf16x2(v[i + 6], v[i + 7]));
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (c + i < p.N) y[i] = __float2bfloat16_rn(v[i]);
    }
  } else {
    float *y = reinterpret_cast<float *>(p.y) + off;
    if (whole && (reinterpret_cast<uintptr_t>(y) & 15) == 0) {
#pragma unroll
      for (int i = 0; i < NC; i += 4)
        *reinterpret_cast<float4 *>(y + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (c + i < p.N) y[i] = v[i];
    }
  }
}

// On the abort path (a wait that ran out): the last `issued` loads of a ring may still be
// writing to shared memory; wait for them, each wait bounded.
__device__ __forceinline__ void drain_loads(const uint64_t *full, int stages, unsigned issued) {
  const unsigned from = issued > (unsigned)stages ? issued - (unsigned)stages : 0u;
  for (unsigned j = from; j < issued; ++j)
    mbar_wait_drain(smem_u32(&full[j % (unsigned)stages]), (j / (unsigned)stages) & 1u);
}

// ------------------------------------------------------------------ many outputs: CTA pairs

// The scales of kScaleSet blocks of K, for the epilogue: lane = row, so rows are an odd number
// of words apart.  Two warps of their own load them: read by the epilogue itself from global
// memory, 32 rows of them a load, they were what bound it.
constexpr int kScaleSet = 16;
struct Scales {
  float sa[BM][kScaleSet + 1];
  float sw[2][kScaleSet];          // per 128 columns of the tile
};

constexpr int kLaunchRegs = 168, kCopyRegs = 56, kEpiRegs = 224;   // per thread (see below)
static_assert(128 * kCopyRegs + 256 * kEpiRegs <= 384 * kLaunchRegs, "registers of the launch");

template <int BN>
struct PairCfg {
  static constexpr int EPI_WARPS = 8;                          // 32 rows x NC columns each
  static constexpr int NC = BN / 2;
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr uint32_t A_BYTES = BM * BK;                 // this CTA's 128 rows
  static constexpr uint32_t B_BYTES = (BN / 2) * BK;           // this CTA's BN / 2 rows
  static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN == 256 ? 5 : 6;
  static constexpr int BUFS = 512 / BN;                        // TMEM buffers, one block's sums each
  static constexpr uint32_t OUT_BYTES = 4096u * EPI_WARPS;     // 32 rows x 128 bytes per warp
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + OUT_BYTES + 2 * sizeof(Scales) + 256;
};

// Tiles run down bands of 8 rows of tiles, so that the tiles in flight at one time (74 pairs)
// share about 8 rows' and 9 columns' operands: at 13112 x 12352 x 4096 that is 18 MB where
// whole columns of tiles would need all of a (54 MB) with every column.
struct Tile {
  int m, n;
};
__device__ __forceinline__ Tile tile_at(int t, int m_tiles, int n_tiles) {
  constexpr int kBand = 8;
  const int band = t / (kBand * n_tiles), r = t - band * kBand * n_tiles;
  const int rows = m_tiles - band * kBand < kBand ? m_tiles - band * kBand : kBand;
  return {band * kBand + r % rows, r / rows};
}

struct PairCtl {
  uint64_t sfull[2];
  uint64_t sempty[2];
  uint64_t full[8];
  uint64_t empty[8];
  uint64_t tfull[4];
  uint64_t tempty[4];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

template <int BN>
__global__ void __launch_bounds__(PairCfg<BN>::THREADS, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmY, const __grid_constant__ GemmFp8Launch p,
                         bool tma_out, unsigned *err_word) {
  using C = PairCfg<BN>;
  constexpr int NC = C::NC;   // columns a thread sums
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *smem_out = smem + C::STAGES * C::STAGE_BYTES;
  Scales *scales = reinterpret_cast<Scales *>(smem_out + C::OUT_BYTES);
  PairCtl *ctl = reinterpret_cast<PairCtl *>(scales + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int m_tiles = (p.T + 2 * BM - 1) / (2 * BM);
  const int n_tiles = (p.N + BN - 1) / BN;
  const int n_total = m_tiles * n_tiles;
  const int kblocks = (p.K + BK - 1) / BK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);    // the leader's: its expect-tx arrival
      mbar_init(smem_u32(&ctl->empty[s]), 1);   // the leader's commit, in both CTAs
    }
    for (int b = 0; b < C::BUFS; ++b) {
      mbar_init(smem_u32(&ctl->tfull[b]), 1);                   // the leader's commit
      mbar_init(smem_u32(&ctl->tempty[b]), 2 * C::EPI_WARPS);   // both CTAs' epilogue warps
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&ctl->sfull[b]), 2);                   // the two warps that load scales
      mbar_init(smem_u32(&ctl->sempty[b]), C::EPI_WARPS);
    }
    mbar_init(smem_u32(&ctl->drain), 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (tma_out) tma_prefetch_desc(&tmY);
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(&ctl->tmem_base), 512);
  // both CTAs' barriers are initialised before either CTA's loads or arrivals reach them
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const AbortFlag ab{&ctl->abort, err_word, ERRBIT_GEMM_TIMEOUT};
  pdl_trigger();
  pdl_wait();

  // Registers: 384 threads are launched with 168 each (the most that fit); the four warps that
  // copy and issue give up 112 each, the epilogue's eight take 56 more for their NC sums.
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 0;
      unsigned issued = 0;
      bool ok = true;
      for (int t = pair; t < n_total && ok; t += n_pairs) {
        const Tile at = tile_at(t, m_tiles, n_tiles);
        const int row_a = at.m * 2 * BM + (int)rank * BM;
        const int row_b = at.n * BN + (int)rank * (BN / 2);
        for (int kb = 0; kb < kblocks; ++kb, ++issued) {
          if (!(ok = mbar_wait(smem_u32(&ctl->empty[stage]), ph ^ 1u, ab))) break;
          const uint32_t sa = smem_u32(smem + stage * C::STAGE_BYTES);
          const uint32_t fb = cluster_map(smem_u32(&ctl->full[stage]), 0);
          if (leader) mbar_arrive_expect_tx(smem_u32(&ctl->full[stage]), 2u * C::STAGE_BYTES);
          tma_load_2d_pair(sa, &tmA, kb * BK, row_a, fb);
          tma_load_2d_pair(sa + C::A_BYTES, &tmB, kb * BK, row_b, fb);
          if (++stage == C::STAGES) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
      // (the pair's loads all signal the leader, and its peer leaves only after it)
      if (!ok && leader) drain_loads(ctl->full, C::STAGES, issued);
    }
  } else if (warp == 1) {
    if (leader) {
      constexpr uint32_t idesc = idesc_e4m3(2 * BM, BN);
      int stage = 0;
      uint32_t ph = 0, phases = 0;
      bool ok = true;
      for (int t = pair; t < n_total && ok; t += n_pairs) {
        for (int kb = 0; kb < kblocks; ++kb) {
          const int buf = kb % C::BUFS;
          if (!(ok = mbar_wait(smem_u32(&ctl->full[stage]), ph, ab) &&
                     mbar_wait(smem_u32(&ctl->tempty[buf]), (phases >> buf & 1u) ^ 1u, ab)))
            break;
          phases ^= 1u << buf;
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * C::STAGE_BYTES);
          const uint64_t ad = sw128_desc(sa, 16, 1024);
          const uint64_t bd = sw128_desc(sa + C::A_BYTES, 16, 1024);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)   // 32 bytes of K: 2 units of 16
              tc_mma_fp8_pair(tmem + (uint32_t)(buf * BN), ad + 2u * kk, bd + 2u * kk, idesc, kk ? 1u : 0u);
            tc_commit_pair(smem_u32(&ctl->empty[stage]));
            tc_commit_pair(smem_u32(&ctl->tfull[buf]));
          }
          __syncwarp();
          if (++stage == C::STAGES) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) {
        if (elect_one()) tc_commit_pair(smem_u32(&ctl->drain));
        __syncwarp();
        mbar_wait_drain(smem_u32(&ctl->drain), 0);
      }
    }
  } else if (warp < 4) {
    int b = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int t = pair; t < n_total && ok; t += n_pairs) {
      const Tile at = tile_at(t, m_tiles, n_tiles);
      const int row0 = at.m * 2 * BM + (int)rank * BM + (warp - 2) * 64;
      const int nb0 = at.n * (BN / kScaleBlock);
      const int n_blocks = (p.N + kScaleBlock - 1) / kScaleBlock;
      for (int kb = 0; kb < kblocks; kb += kScaleSet) {
        if (!(ok = mbar_wait(smem_u32(&ctl->sempty[b]), ph ^ 1u, ab))) break;
        const int k = lane % kScaleSet;
#pragma unroll 8
        for (int i = lane / kScaleSet; i < 64; i += 32 / kScaleSet)
          scales[b].sa[(warp - 2) * 64 + i][k] =
              row0 + i < p.T && kb + k < kblocks ? __ldg(p.sa + (int64_t)(row0 + i) * kblocks + kb + k) : 0.f;
        if (warp == 2) {
          const int g = lane / kScaleSet;
          scales[b].sw[g][k] = nb0 + g < n_blocks && kb + k < kblocks
                                   ? __ldg(p.sw + (int64_t)(nb0 + g) * kblocks + kb + k) : 0.f;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->sfull[b]));
        b ^= 1;
        ph ^= b == 0 ? 1u : 0u;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int q4 = warp & 3;             // TMEM lanes this warp may read: 32 q4 .. 32 q4 + 31
    const int group = (warp - 4) >> 2;   // its NC columns of the tile
    uint8_t *out = smem_out + (warp - 4) * 4096;
    const float *my_sa = scales->sa[q4 * 32 + lane], *my_sw = scales->sw[group * NC / kScaleBlock];
    const uint32_t tempty0 = cluster_map(smem_u32(&ctl->tempty[0]), 0);
    const uint32_t tbase = tmem + ((uint32_t)(q4 * 32) << 16) + (uint32_t)(group * NC);
    int sb = 0;
    uint32_t phases = 0, sph = 0;
    bool ok = true;
    for (int t = pair; t < n_total && ok; t += n_pairs) {
      const Tile at = tile_at(t, m_tiles, n_tiles);
      const int row0 = at.m * 2 * BM + (int)rank * BM + q4 * 32;
      const int row = row0 + lane;
      const int c0 = at.n * BN + group * NC;
      uint64_t sum[NC / 2];   // two columns each
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) sum[i] = 0;
      // Block kb uses TMEM buffer kb % BUFS, so that the buffer is a constant of the unrolled
      // loop; `phases` holds one bit per buffer.
      auto step = [&](int b, const float *sa, const float *sw) {
        const float s = *sa * *sw;
        ok = mbar_wait(smem_u32(&ctl->tfull[b]), phases >> b & 1u, ab) && ok;
        phases ^= 1u << b;
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < NC / 16; ++j) {
          float v[16];
          tmem_ld(tbase + (uint32_t)(b * BN + 16 * j), v);
          tc_wait_ld(v);
          if (j + 1 == NC / 16) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + (uint32_t)(b * sizeof(uint64_t)));
          }
#pragma unroll
          for (int i = 0; i < 16; i += 2)
            sum[8 * j + i / 2] = fma_f32x2(pair_f32(v[i], v[i + 1]), pair_f32(s, s), sum[8 * j + i / 2]);
        }
      };
      // (a wait that gives up does not leave these loops: with an exit in them the sums would be
      // copied, register by register, in every round)
#pragma unroll 1
      for (int set = 0; set < kblocks; set += kScaleSet) {
        ok = mbar_wait(smem_u32(&ctl->sfull[sb]), sph, ab) && ok;
        constexpr int kSet = sizeof(Scales) / sizeof(float);
        const float *sa = my_sa + sb * kSet, *sw = my_sw + sb * kSet;
        const int n = kblocks - set < kScaleSet ? kblocks - set : kScaleSet;
#pragma unroll 1
        for (int k = 0; k < n; k += C::BUFS) {
#pragma unroll
          for (int b = 0; b < C::BUFS; ++b)
            if (b == 0 || k + b < n) step(b, sa + k + b, sw + k + b);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->sempty[sb]));
        sb ^= 1;
        sph ^= sb == 0 ? 1u : 0u;
      }
      if (!ok) break;
      float acc[NC];
#pragma unroll
      for (int i = 0; i < NC; i += 2) split_f32(sum[i / 2], acc[i], acc[i + 1]);
      if (!tma_out) {
        store_row(p, row, c0, acc);
      } else if (row0 < p.T && c0 < p.N) {
        // through shared memory, 128 bytes of each row at a time: a row of y per lane would
        // write 16-byte pieces of 32 rows with every store
        const uint32_t so = smem_u32(out);
        if (p.y_bf16) {
#pragma unroll
          for (int h = 0; h < NC; h += 64) {
            if (c0 + h >= p.N) break;
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 64; i += 8)
              st_shared_v4(so + sw128_offset((uint32_t)lane, 2u * i),
                           pack_bf16x2(acc[h + i], acc[h + i + 1]), pack_bf16x2(acc[h + i + 2], acc[h + i + 3]),
                           pack_bf16x2(acc[h + i + 4], acc[h + i + 5]), pack_bf16x2(acc[h + i + 6], acc[h + i + 7]));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmY, so, c0 + h, row0);
              bulk_commit();
            }
          }
        } else {
#pragma unroll
          for (int h = 0; h < NC; h += 32) {
            if (c0 + h >= p.N) break;
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              st_shared_v4(so + sw128_offset((uint32_t)lane, 4u * i), __float_as_uint(acc[h + i]),
                           __float_as_uint(acc[h + i + 1]), __float_as_uint(acc[h + i + 2]),
                           __float_as_uint(acc[h + i + 3]));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmY, so, c0 + h, row0);
              bulk_commit();
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait<0>();
  }

  // no CTA leaves while its peer may still signal its barriers or read its operands
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ few tokens: K split

constexpr int kFewThreads = 192;
constexpr int kScaleChunk = 32;     // k-blocks whose scales are staged at a time

template <int NT>
struct FewCfg {
  static constexpr uint32_t W_BYTES = BM * BK;
  static constexpr uint32_t A_BYTES = NT * BK;
  static constexpr uint32_t STAGE_BYTES = W_BYTES + A_BYTES;
  static constexpr int STAGES = 7;
  static constexpr int BUFS = 4;
  static constexpr uint32_t TMEM_COLS = BUFS * NT;
  static constexpr uint32_t PART_BYTES = NT * BM * 4;   // every rank's sums of this rank's tokens
  static constexpr uint32_t SC_BYTES = kScaleChunk * NT * 4;
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + PART_BYTES + SC_BYTES + 256;
};

struct FewCtl {
  uint64_t full[8];
  uint64_t empty[8];
  uint64_t tfull[4];
  uint64_t tempty[4];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

template <int NT>
__global__ void __launch_bounds__(kFewThreads, 1)
    gemm_fp8_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ GemmFp8Launch p, unsigned *err_word) {
  using C = FewCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  float *part = reinterpret_cast<float *>(smem + C::STAGES * C::STAGE_BYTES);
  float *sc = part + C::PART_BYTES / 4;
  FewCtl *ctl = reinterpret_cast<FewCtl *>(sc + C::SC_BYTES / 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = (int)cluster_size(), r = (int)cluster_rank();
  const int kblocks = (p.K + BK - 1) / BK;
  const int kb0 = (int)((int64_t)kblocks * r / S), kb1 = (int)((int64_t)kblocks * (r + 1) / S);
  const int n_tiles = (p.N + BM - 1) / BM;
  const int tile = (int)(blockIdx.x / (unsigned)S);
  const int tn = tile % n_tiles, t0 = tile / n_tiles * NT;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int b = 0; b < C::BUFS; ++b) {
      mbar_init(smem_u32(&ctl->tfull[b]), 1);
      mbar_init(smem_u32(&ctl->tempty[b]), 4);
    }
    mbar_init(smem_u32(&ctl->drain), 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmA);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl->tmem_base), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // every CTA of the cluster has started before any writes to it (waited for below)
  if (S > 1) cluster_arrive();
  const uint32_t tmem = ctl->tmem_base;
  const AbortFlag ab{&ctl->abort, err_word, ERRBIT_GEMM_TIMEOUT};
  pdl_trigger();
  pdl_wait();

  float acc[NT];
  const int n = tn * BM + (warp & 3) * 32 + lane;   // the weight row whose sums this thread holds
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 0;
      unsigned issued = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb, ++issued) {
        if (!(ok = mbar_wait(smem_u32(&ctl->empty[stage]), ph ^ 1u, ab))) break;
        const uint32_t sw = smem_u32(smem + stage * C::STAGE_BYTES);
        const uint32_t fb = smem_u32(&ctl->full[stage]);
        mbar_arrive_expect_tx(fb, C::STAGE_BYTES);
        tma_load_2d(sw, &tmW, kb * BK, tn * BM, fb);
        tma_load_2d(sw + C::W_BYTES, &tmA, kb * BK, t0, fb);
        if (++stage == C::STAGES) {
          stage = 0;
          ph ^= 1u;
        }
      }
      if (!ok) drain_loads(ctl->full, C::STAGES, issued);
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_e4m3(BM, NT);
    int stage = 0, buf = 0;
    uint32_t ph = 0, bph = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!(ok = mbar_wait(smem_u32(&ctl->tempty[buf]), bph ^ 1u, ab) &&
                 mbar_wait(smem_u32(&ctl->full[stage]), ph, ab)))
        break;
      tc_fence_after();
      const uint32_t sw = smem_u32(smem + stage * C::STAGE_BYTES);
      const uint64_t wd = sw128_desc(sw, 16, 1024);
      const uint64_t ad = sw128_desc(sw + C::W_BYTES, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)
          tc_mma_fp8(tmem + (uint32_t)(buf * NT), wd + 2u * kk, ad + 2u * kk, idesc, kk ? 1u : 0u);
        tc_commit(smem_u32(&ctl->empty[stage]));
        tc_commit(smem_u32(&ctl->tfull[buf]));
      }
      __syncwarp();
      if (++stage == C::STAGES) {
        stage = 0;
        ph ^= 1u;
      }
      if (++buf == C::BUFS) {
        buf = 0;
        bph ^= 1u;
      }
    }
    if (!ok) {
      if (elect_one()) tc_commit(smem_u32(&ctl->drain));
      __syncwarp();
      mbar_wait_drain(smem_u32(&ctl->drain), 0);
    }
  } else {
    const uint32_t tbase = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    int buf = 0;
    uint32_t bph = 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = 0.f;
#pragma unroll 1
    for (int kb = kb0; kb < kb1; ++kb) {
      const int at = (kb - kb0) % kScaleChunk;
      if (at == 0) {
        // the next blocks' scale products, one per token
        bar_sync_n(1, 128);
        const int t = ((int)threadIdx.x - 64) % NT, n_b = kb1 - kb < kScaleChunk ? kb1 - kb : kScaleChunk;
        const float *sa = p.sa + (int64_t)(t0 + t) * kblocks + kb, *sw = p.sw + (int64_t)tn * kblocks + kb;
        const bool in = t0 + t < p.T;
#pragma unroll 4
        for (int b = ((int)threadIdx.x - 64) / NT; b < n_b; b += 128 / NT)
          sc[b * NT + t] = in ? __ldg(sa + b) * __ldg(sw + b) : 0.f;
        bar_sync_n(1, 128);
      }
      const bool ok = mbar_wait(smem_u32(&ctl->tfull[buf]), bph, ab);
      tc_fence_after();
      // (after an abort the loop goes on, so that all warps meet at the barriers above)
      if (ok) {
#pragma unroll
        for (int j = 0; j < NT; j += 16) {
          float v[16];
          tmem_ld(tbase + (uint32_t)(buf * NT + j), v);
          tc_wait_ld(v);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[j + i] = fmaf(v[i], sc[at * NT + j + i], acc[j + i]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->tempty[buf]));
      if (++buf == C::BUFS) {
        buf = 0;
        bph ^= 1u;
      }
    }
  }

  auto put = [&](int t, float v) {
    if (n >= p.N) return;
    const int64_t at = (int64_t)t * p.y_stride + n;
    if (p.y_bf16) reinterpret_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(v);
    else reinterpret_cast<float *>(p.y)[at] = v;
  };
  const int nl = (warp & 3) * 32 + lane;
  __syncwarp();
  if (S == 1) {
    if (warp >= 2) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (t0 + i < p.T) put(t0 + i, acc[i]);
    }
  } else {
    // rank q adds, in the order of K, the S partial sums of tokens q per .. (q + 1) per - 1
    const int lg = 31 - __clz(NT / S), per = 1 << lg;   // S is a power of two
    cluster_wait();
    if (warp >= 2) {
      const uint32_t mine = smem_u32(part) + (uint32_t)((r * per * BM + nl) * 4);
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (t0 + i < p.T)
          st_cluster(cluster_map(mine + (uint32_t)((i & (per - 1)) * BM * 4), (uint32_t)(i >> lg)), acc[i]);
    }
    __syncwarp();
    cluster_sync_all();
    if (warp >= 2) {
      for (int i = 0; i < per && t0 + r * per + i < p.T; ++i) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < S) v += part[(k * per + i) * BM + nl];
        put(t0 + r * per + i, v);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

cudaError_t launch_clusters(const void *kern, unsigned grid, unsigned threads, size_t smem, unsigned cluster,
                            cudaStream_t s, bool pdl, void **args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, kern, args);
}

template <int BN>
cudaError_t launch_pair(const GemmFp8Launch &p, unsigned *err_word, cudaStream_t s, bool pdl, std::string *err) {
  using C = PairCfg<BN>;
  CUtensorMap ta, tb, ty;
  if (!make_tmap_2d(&ta, p.a, 1, (uint64_t)p.K, (uint64_t)p.T, (uint64_t)p.a_stride, BM, err) ||
      !make_tmap_2d(&tb, p.w, 1, (uint64_t)p.K, (uint64_t)p.N, (uint64_t)p.w_stride, BN / 2, err))
    return cudaErrorInvalidValue;
  // tiled stores where y's rows are 16-byte aligned
  const int esz = p.y_bf16 ? 2 : 4;
  bool tma_out = (reinterpret_cast<uintptr_t>(p.y) & 15) == 0 && (p.y_stride * esz) % 16 == 0;
  if (tma_out) {
    if (!make_tmap_2d(&ty, p.y, esz, (uint64_t)p.N, (uint64_t)p.T, (uint64_t)p.y_stride * esz, 32, err))
      return cudaErrorInvalidValue;
  } else {
    ty = ta;
  }
  const void *kern = reinterpret_cast<const void *>(gemm_fp8_pair_kernel<BN>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  // the epilogue takes registers that the copying warps give up, out of what the launch got: a
  // build that launches with fewer would wait for them for good
  static const int regs = [&] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess ? a.numRegs : 0;
  }();
  if (regs < kLaunchRegs) {
    if (err) *err = "gemm_fp8_pair_kernel was built with " + std::to_string(regs) + " registers";
    return cudaErrorInvalidValue;
  }
  const int64_t tiles = (int64_t)((p.T + 2 * BM - 1) / (2 * BM)) * ((p.N + BN - 1) / BN);
  const int64_t pairs = std::min<int64_t>(tiles, std::max(1, device_sm_count() / 2));
  GemmFp8Launch q = p;
  void *args[] = {&ta, &tb, &ty, &q, &tma_out, &err_word};
  return launch_clusters(kern, (unsigned)(2 * pairs), C::THREADS, C::SMEM, 2, s, pdl, args);
}

// CTAs that split K: as long as the clusters still fit the GPU at once and each keeps two blocks.
int few_split(int64_t tiles, int kblocks) {
  int S = 1;
  while (S < 8 && tiles * S * 2 <= device_sm_count() && kblocks >= 4 * S) S *= 2;
  return S;
}

template <int NT>
cudaError_t launch_few(const GemmFp8Launch &p, unsigned *err_word, cudaStream_t s, bool pdl, std::string *err) {
  using C = FewCfg<NT>;
  CUtensorMap tw, ta;
  if (!make_tmap_2d(&tw, p.w, 1, (uint64_t)p.K, (uint64_t)p.N, (uint64_t)p.w_stride, BM, err) ||
      !make_tmap_2d(&ta, p.a, 1, (uint64_t)p.K, (uint64_t)p.T, (uint64_t)p.a_stride, NT, err))
    return cudaErrorInvalidValue;
  const void *kern = reinterpret_cast<const void *>(gemm_fp8_few_kernel<NT>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)((p.T + NT - 1) / NT) * ((p.N + BM - 1) / BM);
  const int S = few_split(tiles, (p.K + BK - 1) / BK);
  GemmFp8Launch q = p;
  void *args[] = {&tw, &ta, &q, &err_word};
  return launch_clusters(kern, (unsigned)(tiles * S), kFewThreads, C::SMEM, (unsigned)S, s, pdl, args);
}

}  // namespace

cudaError_t launch_gemm_fp8(const GemmFp8Launch &p, unsigned *err_word, cudaStream_t s, bool pdl,
                            std::string *err) {
  if (p.T <= 0 || p.N <= 0) return cudaSuccess;
  // The cycles that a call takes, by rounds of tiles and blocks of K: 350 + 9 NT for a block of
  // the few-token kernel (measured 500 at 16 tokens, 950 at 64), 510 and 740 for one of the pair
  // kernel's, and 1500 more for what a pair or a split tile does once.
  const int sms = device_sm_count(), pairs = std::max(1, sms / 2), kblocks = (p.K + BK - 1) / BK;
  auto rounds = [](int64_t tiles, int64_t at_once) { return (tiles + at_once - 1) / at_once; };
  const int nt = p.T <= 16 ? 16 : p.T <= 32 ? 32 : 64;
  const int64_t few_tiles = (int64_t)((p.T + nt - 1) / nt) * ((p.N + BM - 1) / BM);
  const int S = few_split(few_tiles, kblocks);
  const int64_t few = rounds(few_tiles * S, sms) * ((kblocks + S - 1) / S) * (350 + 9 * nt) + (S > 1 ? 1500 : 0);
  const int64_t m = (p.T + 2 * BM - 1) / (2 * BM);
  const int64_t p128 = rounds(m * ((p.N + 127) / 128), pairs) * kblocks * 510 + 1500;
  const int64_t p256 = rounds(m * ((p.N + 255) / 256), pairs) * kblocks * 740 + 1500;
  if (few <= std::min(p128, p256))
    return nt == 16   ? launch_few<16>(p, err_word, s, pdl, err)
           : nt == 32 ? launch_few<32>(p, err_word, s, pdl, err)
                      : launch_few<64>(p, err_word, s, pdl, err);
  return p128 <= p256 ? launch_pair<128>(p, err_word, s, pdl, err) : launch_pair<256>(p, err_word, s, pdl, err);
}

}  // namespace tr
