// fp8_gemm.cu -- the product of two e4m3 operands with a scale per block of 128:
//
//   y[t, n] = sum_b sa[t, b] sw[n / 128, b] sum_{k in block b} a[t, k] w[n, k]
//
// a [T, K] (an activation: one scale per row and 128 columns), w [N, K] (a weight: one scale
// per 128 x 128 tile), both K-major.  The products of one block are summed by the tensor core
// in fp32 (tcgen05.mma kind::f8f6f4); because the scales change from block to block, each
// block's 128 x BN sums go to their own TMEM buffer, and the epilogue warps add them, scaled,
// into fp32 registers while the tensor core works on the next block.  The only rounding to
// fewer bits is the output's.
#include <cuda_bf16.h>

#include "fp8_ptx.cuh"
#include "layer_ops.h"
#include "tr_internal.h"

namespace tr {
namespace {

constexpr int BM = 128;
constexpr int BK = 128;              // one scale block; 128 bytes, one swizzle row
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;

// 2D byte tensor map, 128-byte swizzle: boxes of 128 bytes x `box_rows`, bytes past the matrix
// read as 0 (the last block of a K that is not a multiple of 128; rows past the end)
bool make_tmap_bytes_2d(CUtensorMap *tm, const void *base, uint64_t inner, uint64_t rows,
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
  cuuint64_t strides[1] = {row_stride};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides,
                        box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    if (err) *err = "cuTensorMapEncodeTiled failed (" + std::to_string((int)r) + ")";
    return false;
  }
  return true;
}

template <int BN>
struct Cfg {
  static constexpr uint32_t A_BYTES = BM * BK;
  static constexpr uint32_t B_BYTES = BN * BK;
  static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = 6;
  static constexpr int BUFS = 512 / BN;      // TMEM buffers, one block's sums each
  static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + 256;
};

struct Ctl {
  uint64_t full[8];
  uint64_t empty[8];
  uint64_t tfull[4];
  uint64_t tempty[4];
  uint32_t tmem_base;
  int abort;
};

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

template <int BN>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ GemmFp8Launch p, unsigned *err_word) {
  using C = Cfg<BN>;
  constexpr int NC = BN / 2;   // columns a thread sums: half of the tile's (see the epilogue)
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  Ctl *ctl = reinterpret_cast<Ctl *>(smem + C::STAGES * C::STAGE_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m_tiles = (p.T + BM - 1) / BM;
  const int n_tiles = (p.N + BN - 1) / BN;
  const int n_total = m_tiles * n_tiles;
  const int kblocks = (p.K + BK - 1) / BK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int b = 0; b < C::BUFS; ++b) {
      mbar_init(smem_u32(&ctl->tfull[b]), 1);
      mbar_init(smem_u32(&ctl->tempty[b]), kEpiWarps);
    }
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const AbortFlag ab{&ctl->abort, err_word, ERRBIT_GEMM_TIMEOUT};
  pdl_trigger();
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 0;
      for (int t = blockIdx.x; t < n_total; t += gridDim.x) {
        const int tm = t % m_tiles, tn = t / m_tiles;
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!mbar_wait(smem_u32(&ctl->empty[stage]), ph ^ 1u, ab)) goto producer_done;
          const uint32_t sa = smem_u32(smem + stage * C::STAGE_BYTES);
          const uint32_t fb = smem_u32(&ctl->full[stage]);
          mbar_arrive_expect_tx(fb, C::STAGE_BYTES);
          tma_load_2d(sa, &tmA, kb * BK, tm * BM, fb);
          tma_load_2d(sa + C::A_BYTES, &tmB, kb * BK, tn * BN, fb);
          if (++stage == C::STAGES) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
    producer_done:;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3(BM, BN);
      int stage = 0, buf = 0;
      uint32_t ph = 0, bph = 0;
      for (int t = blockIdx.x; t < n_total; t += gridDim.x) {
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!mbar_wait(smem_u32(&ctl->tempty[buf]), bph ^ 1u, ab)) goto mma_done;
          if (!mbar_wait(smem_u32(&ctl->full[stage]), ph, ab)) goto mma_done;
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * C::STAGE_BYTES);
          const uint64_t ad = sw128_desc(sa, 16, 1024);
          const uint64_t bd = sw128_desc(sa + C::A_BYTES, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)   // 32 bytes of K: 2 units of 16
            tc_mma_fp8(tmem + (uint32_t)(buf * BN), ad + 2u * kk, bd + 2u * kk, idesc, kk ? 1u : 0u);
          tc_commit(smem_u32(&ctl->empty[stage]));
          tc_commit(smem_u32(&ctl->tfull[buf]));
          if (++stage == C::STAGES) {
            stage = 0;
            ph ^= 1u;
          }
          if (++buf == C::BUFS) {
            buf = 0;
            bph ^= 1u;
          }
        }
      }
    mma_done:;
    }
  } else {
    const int q4 = warp & 3;             // TMEM lanes this warp may read: 32 q4 .. 32 q4 + 31
    const int half = (warp - 2) >> 2;    // which half of the tile's columns
    int buf = 0;
    uint32_t bph = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < n_total && ok; t += gridDim.x) {
      const int tm = t % m_tiles, tn = t / m_tiles;
      const int row = tm * BM + q4 * 32 + lane;
      const int c0 = tn * BN + half * NC;
      // past the end of y the sums are 0 (the operands read as 0): any scale does
      const float *sa = p.sa + (int64_t)(row < p.T ? row : 0) * kblocks;
      const float *sw = p.sw + (int64_t)(c0 < p.N ? c0 / kScaleBlock : 0) * kblocks;
      float acc[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) acc[i] = 0.f;
#pragma unroll 1
      for (int kb = 0; kb < kblocks; ++kb) {
        const float s = __ldg(sa + kb) * __ldg(sw + kb);
        if (!mbar_wait(smem_u32(&ctl->tfull[buf]), bph, ab)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tb = tmem + ((uint32_t)(q4 * 32) << 16) + (uint32_t)(buf * BN + half * NC);
#pragma unroll
        for (int j = 0; j < NC / 32; ++j) {
          float v[32];
          tmem_ld32(tb + 32 * j, v);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[32 * j + i] = fmaf(v[i], s, acc[32 * j + i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->tempty[buf]));
        if (++buf == C::BUFS) {
          buf = 0;
          bph ^= 1u;
        }
      }
      if (ok) {
#pragma unroll
        for (int j = 0; j < NC / 32; ++j) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = acc[32 * j + i];
          store_row<32>(p, row, c0 + 32 * j, v);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_gemm_fp8(const GemmFp8Launch &p, unsigned *err_word, cudaStream_t s, bool pdl,
                            std::string *err) {
  if (p.T <= 0 || p.N <= 0) return cudaSuccess;
  using C = Cfg<128>;
  CUtensorMap ta, tb;
  if (!make_tmap_bytes_2d(&ta, p.a, (uint64_t)p.K, (uint64_t)p.T, (uint64_t)p.a_stride, BM, err) ||
      !make_tmap_bytes_2d(&tb, p.w, (uint64_t)p.K, (uint64_t)p.N, (uint64_t)p.w_stride, 128, err))
    return cudaErrorInvalidValue;
  auto kern = gemm_fp8_kernel<128>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)((p.T + BM - 1) / BM) * ((p.N + 127) / 128);
  const int grid = (int)(tiles < device_sm_count() ? tiles : device_sm_count());
  return launch_kernel(kern, dim3((unsigned)grid), dim3(kThreads), C::SMEM, s, pdl, ta, tb, p, err_word);
}

}  // namespace tr
