// fp8_quant.cu -- the e4m3 operands of the 8-bit projections: RMSNorm (with the residual's
// addition) written as e4m3 with scales, and the plain quantisation of a matrix.
//
//   r = x + residual,  n = r / sqrt(mean r^2 + eps) * gain          (fp32; or n = x)
//   per block of 128 columns (and block_rows rows):
//     s = max(max|n| / 448, 2^-126),  q = e4m3(n * (1 / s))         (round to nearest even)
//
// 448 is e4m3's largest value; the floor of 2^-126 keeps 1 / s finite for an all-zero block
// (its q is 0 with any scale).  A NaN in a block makes the block's scale and values NaN; an
// infinity makes the scale infinite, so the block reads back as NaN.  The division and the
// reciprocal are IEEE, one per block; the products round once.  r is kept in fp32 (the
// residual output rounds it on its own), and the e4m3 rounding is the only other one.
// HBM-bound: each input is read once into registers and each output written once (13112 x 4096
// with an fp32 residual: 92 us, 13112 x 5632 bf16 by rows: 35 us, both 98-99% of the measured
// copy rate; 6176 x 2048 by tiles: 7 us; a few rows: the launch, 1.5-3 us).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "fp8_ptx.cuh"
#include "layer_ops.h"
#include "tr_internal.h"

namespace tr {
namespace {

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 8 elements as loaded
template <bool BF16> struct Raw8;
template <> struct Raw8<true> {
  uint4 u;
  __device__ __forceinline__ void load(const void *p, int64_t off) {
    u = *reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(p) + off);
  }
  __device__ __forceinline__ void to_f32(float (&f)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <> struct Raw8<false> {
  float4 a, b;
  __device__ __forceinline__ void load(const void *p, int64_t off) {
    const float4 *q = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + off);
    a = q[0];
    b = q[1];
  }
  __device__ __forceinline__ void to_f32(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};
template <bool BF16>
__device__ __forceinline__ void load8(const void *p, int64_t off, float (&f)[8]) {
  Raw8<BF16> r;
  r.load(p, off);
  r.to_f32(f);
}

template <bool BF16>
__device__ __forceinline__ void store8(void *p, int64_t off, const float (&f)[8]) {
  if (BF16) {
    *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(p) + off) =
        make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
  } else {
    float4 *q = reinterpret_cast<float4 *>(reinterpret_cast<float *>(p) + off);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// The largest magnitude of 8 elements as the bits of an fp32: magnitudes order like their bits
// as unsigned integers, with a NaN above infinity, so that the largest is NaN if any is.
__device__ __forceinline__ uint32_t abs_max8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ uint32_t abs_max8(const Raw8<true> &r) {   // two at a time
  const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(w[i] & 0x7fff7fffu));
  return max(m & 0xffff0000u, m << 16);
}
__device__ __forceinline__ uint32_t abs_max8(const Raw8<false> &r) {
  float f[8];
  r.to_f32(f);
  return abs_max8(f);
}
// Over the 16 lanes that share a scale block.
__device__ __forceinline__ uint32_t max_of_16(uint32_t m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// The scale of a block whose largest magnitude is m.
__device__ __forceinline__ float scale_of(uint32_t m) {
  return max_nan(__fdiv_rn(__uint_as_float(m), 448.f), 1.17549435e-38f);
}

__device__ __forceinline__ void store_q8(uint8_t *dst, const float (&f)[8], float inv) {
  uint32_t w[2];
  const uint64_t ii = pair_f32(inv, inv);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float a, b, c, d;
    split_f32(mul_f32x2(pair_f32(f[4 * h], f[4 * h + 1]), ii), a, b);
    split_f32(mul_f32x2(pair_f32(f[4 * h + 2], f[4 * h + 3]), ii), c, d);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    w[h] = lo | (hi << 16);
  }
  *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
}

constexpr int kNV = 4;   // 8-element vectors a lane holds of its row

// WPR warps with NV vectors a lane share a row (WPR * NV * 256 columns): vector v of the row is
// lane v % 32 of warp (v / 32) % WPR, so 16 neighbouring lanes hold a scale block and each
// warp's accesses are contiguous.  A few vectors per lane and several warps per row, rather than a warp per
// row with the whole row in its registers, so that a few rows use many warps too.
// A vector's division is done by one lane in NV, as in quantize_rows_kernel (one in four there).
template <bool XBF, bool RES, bool RBF, int WPR, int NV>
__global__ void __launch_bounds__(WPR < 8 ? 256 : WPR * 32)
    rmsnorm_fp8_kernel(NormFp8Launch p) {
  constexpr int kRows = WPR < 8 ? 8 / WPR : 1;   // rows of a block
  __shared__ float part[kRows][WPR];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = warp % WPR, slot = warp / WPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + slot;
  const bool live = row < p.rows;
  pdl_trigger();
  pdl_wait();
  float f[NV][8];
  float ss = 0.f;
  auto first = [&](int j) { return (j * WPR + wr) * 256; };   // a vector's first column in the warp
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = first(j) + lane * 8;
    const bool in = live && c < p.D;
    if (in) load8<XBF>(p.x, row * p.x_stride + c, f[j]);
    else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[j][i] = 0.f;
    }
    if (RES && in) {
      float r[8];
      load8<RBF>(p.res, row * p.res_stride + c, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[j][i] += r[i];
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = first(j) + lane * 8;
    if (RES && p.res_out && live && c < p.D)
      store8<RBF>(p.res_out, row * p.res_out_stride + c, f[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(f[j][i], f[j][i], ss);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (WPR > 1) {
    if (lane == 0) part[slot][wr] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) ss += part[slot][w];
  }
  const float rms = rsqrtf(ss / (float)p.D + p.eps);
  const int kb = (p.D + kScaleBlock - 1) / kScaleBlock;
  uint32_t mine = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = first(j) + lane * 8;
    const bool in = live && c < p.D;
    float g[8];
    if (p.gain && in) load8<false>(p.gain, c, g);
    else {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = 1.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[j][i] = f[j][i] * rms * g[i];
    const uint32_t m = max_of_16(abs_max8(f[j]));
    if ((lane & 15) % NV == j) mine = m;
  }
  const float my_scale = scale_of(mine), my_inv = __frcp_rn(my_scale);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = first(j) + lane * 8;
    const float s = __shfl_sync(0xffffffffu, my_scale, (lane & 16) + j);
    const float inv = __shfl_sync(0xffffffffu, my_inv, (lane & 16) + j);
    if (live && c < p.D) {
      store_q8(p.q + row * p.D + c, f[j], inv);
      if ((lane & 15) == 0) p.scale[row * kb + c / kScaleBlock] = s;
    }
  }
}

// One scale per row and 128 columns: a warp takes kNV vectors per lane, 1024 columns, of a row;
// 16 neighbouring lanes hold a scale block.  The division and the reciprocal of a vector's block
// are done by one lane in four and handed round: done by each lane for each of its vectors, they
// were most of the kernel's instructions, and with a 64-bit division per vector for its place
// they bound it (13112 x 5632 bf16: 71 us).
template <bool XBF>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantFp8Launch p) {
  const int lane = threadIdx.x & 31;
  const unsigned per = (unsigned)(p.cols + kNV * 256 - 1) / (kNV * 256);   // warps per row
  const unsigned rb = blockIdx.x / per;
  const int64_t row = (int64_t)rb * 8 + (threadIdx.x >> 5);
  const int c0 = (int)(blockIdx.x - rb * per) * kNV * 256 + lane * 8;
  const int kb = (p.cols + kScaleBlock - 1) / kScaleBlock;
  pdl_trigger();
  pdl_wait();
  if (row >= p.rows) return;
  Raw8<XBF> raw[kNV];
#pragma unroll
  for (int j = 0; j < kNV; ++j) {
    raw[j] = Raw8<XBF>{};
    if (c0 + 256 * j < p.cols) raw[j].load(p.x, row * p.x_stride + c0 + 256 * j);
  }
  uint32_t mine = 0;
#pragma unroll
  for (int j = 0; j < kNV; ++j) {
    const uint32_t m = max_of_16(abs_max8(raw[j]));
    if (lane % kNV == j) mine = m;
  }
  const float my_scale = scale_of(mine), my_inv = __frcp_rn(my_scale);
#pragma unroll
  for (int j = 0; j < kNV; ++j) {
    const float s = __shfl_sync(0xffffffffu, my_scale, (lane & 16) + j);
    const float inv = __shfl_sync(0xffffffffu, my_inv, (lane & 16) + j);
    const int c = c0 + 256 * j;
    if (c < p.cols) {
      float f[8];
      raw[j].to_f32(f);
      store_q8(p.q + row * p.cols + c, f, inv);
      if ((lane & 15) == 0) p.scale[row * kb + c / kScaleBlock] = s;
    }
  }
}

// One scale per 128 x 128 tile: a block holds the tile in registers as it was loaded, 8 rows per
// thread (16 lanes across the columns, 16 row groups).
template <bool XBF>
__global__ void __launch_bounds__(256) quantize_tile_kernel(QuantFp8Launch p) {
  __shared__ uint32_t part[8];
  const int kb = (p.cols + kScaleBlock - 1) / kScaleBlock;
  const int64_t rb = blockIdx.x / kb;
  const int cb = (int)(blockIdx.x - rb * kb);
  const int c = cb * kScaleBlock + (threadIdx.x & 15) * 8;
  const int64_t r0 = rb * kScaleBlock + (threadIdx.x >> 4);
  pdl_trigger();
  pdl_wait();
  Raw8<XBF> raw[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    raw[j] = Raw8<XBF>{};
    if (r0 + 16 * j < p.rows && c < p.cols) raw[j].load(p.x, (r0 + 16 * j) * p.x_stride + c);
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, abs_max8(raw[j]));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max(m, part[w]);
  const float s = scale_of(m);
  const float inv = __frcp_rn(s);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float f[8];
    raw[j].to_f32(f);
    if (r0 + 16 * j < p.rows && c < p.cols) store_q8(p.q + (r0 + 16 * j) * p.cols + c, f, inv);
  }
  if (threadIdx.x == 0) p.scale[rb * kb + cb] = s;
}

template <bool XBF, bool RES, bool RBF, int WPR>
cudaError_t launch_norm_wpr(const NormFp8Launch &p, int nv, cudaStream_t s, bool pdl) {
  constexpr int rows = WPR < 8 ? 8 / WPR : 1;
  const dim3 grid((unsigned)((p.rows + rows - 1) / rows)), block(WPR < 8 ? 256 : WPR * 32);
  if constexpr (WPR == 1) {
    if (nv == 1) return launch_kernel(rmsnorm_fp8_kernel<XBF, RES, RBF, 1, 1>, grid, block, 0, s, pdl, p);
    if (nv == 2) return launch_kernel(rmsnorm_fp8_kernel<XBF, RES, RBF, 1, 2>, grid, block, 0, s, pdl, p);
  }
  return nv <= 3 ? launch_kernel(rmsnorm_fp8_kernel<XBF, RES, RBF, WPR, 3>, grid, block, 0, s, pdl, p)
                 : launch_kernel(rmsnorm_fp8_kernel<XBF, RES, RBF, WPR, 4>, grid, block, 0, s, pdl, p);
}

template <bool XBF, bool RES, bool RBF>
cudaError_t launch_norm(const NormFp8Launch &p, cudaStream_t s, bool pdl) {
  // the fewest warps that hold the row with four vectors a lane, and the fewest vectors then
  // (13000 x 1040 bf16: 16 us, 19 with four vectors for every width; 13000 x 320: 8 and 10)
  const int units = (p.D + 255) / 256;
  int wpr = 1;
  while (wpr * 4 < units) wpr *= 2;
  const int nv = (units + wpr - 1) / wpr;
  switch (wpr) {
    case 1: return launch_norm_wpr<XBF, RES, RBF, 1>(p, nv, s, pdl);
    case 2: return launch_norm_wpr<XBF, RES, RBF, 2>(p, nv, s, pdl);
    case 4: return launch_norm_wpr<XBF, RES, RBF, 4>(p, nv, s, pdl);
    case 8: return launch_norm_wpr<XBF, RES, RBF, 8>(p, nv, s, pdl);
    case 16: return launch_norm_wpr<XBF, RES, RBF, 16>(p, nv, s, pdl);
    default: return launch_norm_wpr<XBF, RES, RBF, 32>(p, nv, s, pdl);
  }
}

}  // namespace

cudaError_t launch_rmsnorm_fp8(const NormFp8Launch &p, cudaStream_t s, bool pdl) {
  if (p.rows <= 0) return cudaSuccess;
  if (!p.res)
    return p.x_bf16 ? launch_norm<true, false, false>(p, s, pdl)
                    : launch_norm<false, false, false>(p, s, pdl);
  if (p.res_bf16)
    return p.x_bf16 ? launch_norm<true, true, true>(p, s, pdl)
                    : launch_norm<false, true, true>(p, s, pdl);
  return p.x_bf16 ? launch_norm<true, true, false>(p, s, pdl)
                  : launch_norm<false, true, false>(p, s, pdl);
}

cudaError_t launch_quantize_fp8(const QuantFp8Launch &p, cudaStream_t s, bool pdl) {
  if (p.rows <= 0) return cudaSuccess;
  if (p.block_rows == kScaleBlock) {
    const int64_t tiles = ((p.rows + kScaleBlock - 1) / kScaleBlock) *
                          ((p.cols + kScaleBlock - 1) / kScaleBlock);
    return p.x_bf16 ? launch_kernel(quantize_tile_kernel<true>, dim3((unsigned)tiles), dim3(256), 0, s, pdl, p)
                    : launch_kernel(quantize_tile_kernel<false>, dim3((unsigned)tiles), dim3(256), 0, s, pdl, p);
  }
  const int64_t blocks = (p.rows + 7) / 8 * ((p.cols + kNV * 256 - 1) / (kNV * 256));
  return p.x_bf16 ? launch_kernel(quantize_rows_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, s, pdl, p)
                  : launch_kernel(quantize_rows_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, s, pdl, p);
}

}  // namespace tr
