// mxquant.cu -- rows into MXFP8 (E4M3 codes, one E8M0 scale per 32 or 64
// elements), the operand form of mxfp8_scaled_mm and of the grouped products,
// with the residual add and the RMSNorm in front, or neither:
//
//   s    = bf16(x + residual)                       written back on request
//   y    = (s * rstd) * gamma                       FP32, rstd of s's row
//   X    = floor(log2 max|y|) - 8 per block, at least -127
//   code = E4M3(y * 2^-X), scale byte X + 127
//
// the codes of rmsnorm_linear_mxfp8 to the bit: the sum of squares is the
// rounding of the exact sum (exactsum.cuh), every other step one correctly
// rounded FP32 operation.  A block with an infinity or NaN gets scale byte 255
// (and codes 0).
//
// One CTA a row, the row in registers (NV 16-byte vectors a thread), so x and
// the residual are read once: 7 bytes of traffic an element with a residual
// and its sum.  Bound by HBM: 16384 x 4096 in 70 to 71 us, 6.6 TB/s; 8192 x 4096 38.4 us,
// 6.1 TB/s, with two vectors a thread 42, one 52, eight 48, with a persistent CTA
// that loads the next row while it works on one 47 and more.  Rows as they are: 8192 x
// 4096 16.5 us, 6.1 TB/s; short rows are bound by the start of their CTAs, one a
// nanosecond: 65536 x 768 66.8 us, 2.3 TB/s.
#include <cuda_fp8.h>

#include "bf16x8.cuh"
#include "exactsum.cuh"
#include "internal.h"
#include "ptx_more.cuh"

namespace rnl {
namespace {

struct QuantArgs {
  const uint4* x;
  const uint4* residual;  // may be null
  uint4* x_sum;           // may be null, x or residual
  const uint4* gamma;     // may be null
  int nvec;               // K / 8
  float inv_d, eps;
  uint2* codes;
  uint8_t* scale;
};

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}

// NORM 0: no norm; 1: rsqrt form; 2: sqrt + divide form.  blockDim.x is a
// multiple of 32 with NV * blockDim.x >= nvec.
template <int NORM, int NV, int BLK>
__global__ void __launch_bounds__(1024) quant_kernel(QuantArgs p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * p.nvec;
  uint4 u[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    u[i] = v < p.nvec ? p.x[at + v] : make_uint4(0u, 0u, 0u, 0u);
  }
  if (p.residual != nullptr) {
    constexpr int kAhead = NV < 4 ? NV : 4;  // the residual's vectors in flight (64 registers a thread)
#pragma unroll
    for (int i0 = 0; i0 < NV; i0 += kAhead) {
      uint4 r[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int v = threadIdx.x + (i0 + i) * blockDim.x;
        r[i] = v < p.nvec ? p.residual[at + v] : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int v = threadIdx.x + (i0 + i) * blockDim.x;
        u[i0 + i] = add_bf16x8(u[i0 + i], r[i]);
        if (p.x_sum != nullptr && v < p.nvec) p.x_sum[at + v] = u[i0 + i];
      }
    }
  }
  float rstd = 1.0f;
  if constexpr (NORM != 0) {
    constexpr int kMode = NORM - 1;
    uint64_t hs[4] = {0, 0, 0, 0}, ls[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < NV; ++i) ffx2_add_squares8<kMode>(u[i], p.inv_d, hs, ls);
    float hi, lo;
    ffx2_warp_hilo(hs, ls, hi, lo);
    if (blockDim.x > 32) {
      __shared__ float2 part[32];
      if (lane == 0) part[warp] = make_float2(hi, lo);
      __syncthreads();
      const float2 q = lane < (blockDim.x >> 5) ? part[lane] : make_float2(0.f, 0.f);
      hi = q.x;
      lo = q.y;
      ff_warp_merge(hi, lo);
    }
    rstd = rstd_of_sum<kMode>(ff_round(hi, lo), p.inv_d, p.eps);
  }
  constexpr int kGroup = BLK / 8;  // lanes a block
  uint8_t* srow = p.scale + static_cast<int64_t>(blockIdx.x) * (p.nvec / kGroup);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v - lane >= p.nvec) break;  // the same on every lane
    const bool live = v < p.nvec;
    float f[8];
    unpack8(u[i], f);
    if constexpr (NORM != 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], rstd);
      if (p.gamma != nullptr && live) {
        float g[8];
        unpack8(p.gamma[v], g);  // (a plain load: a read-only one need not stay behind the wait)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], g[j]);
      }
    }
    // the largest magnitude by its bits: infinities and NaN come out on top
    uint32_t am = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) am = max(am, __float_as_uint(f[j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 1; o < kGroup; o <<= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
    const int eb = static_cast<int>(am >> 23);
    const bool bad = eb == 255;
    int X = eb - 127 - 8;
    if (X < -127) X = -127;
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - X) << 23);  // 2^-X, X in [-127, 119]
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = bad ? 0u : e4m3x2(__fmul_rn(f[2 * j], inv), __fmul_rn(f[2 * j + 1], inv));
    if (live) {
      p.codes[at + v] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      if ((lane & (kGroup - 1)) == 0) srow[v / kGroup] = static_cast<uint8_t>(bad ? 255 : X + 127);
    }
  }
}

template <int NORM, int BLK>
cudaError_t launch(const QuantArgs& p, int64_t T, int sm_count, cudaStream_t s) {
  // few rows: every vector a thread of its own, for the shortest way through a
  // row; many: four a thread, for more loads in flight and shorter merges
  const bool few = T < 4 * sm_count && p.nvec <= 1024;
  const int nv = few ? 1 : (p.nvec <= 4096 ? 4 : 8);
  const int threads = ((p.nvec + nv - 1) / nv + 31) / 32 * 32;
  const unsigned grid = static_cast<unsigned>(T);
  if (nv == 1) return launch_dependent(quant_kernel<NORM, 1, BLK>, grid, threads, 0, s, p);
  if (nv == 4) return launch_dependent(quant_kernel<NORM, 4, BLK>, grid, threads, 0, s, p);
  return launch_dependent(quant_kernel<NORM, 8, BLK>, grid, threads, 0, s, p);
}

template <int NORM>
cudaError_t launch_blk(const QuantArgs& p, int64_t T, int64_t block, int sm_count, cudaStream_t s) {
  return block == 64 ? launch<NORM, 64>(p, T, sm_count, s) : launch<NORM, 32>(p, T, sm_count, s);
}

}  // namespace

rnl_status launch_quant_mxfp8(const void* x, const void* residual, void* x_sum, const void* gamma, int64_t T,
                              int64_t K, bool norm, float eps, int mode, int64_t block, uint8_t* codes,
                              uint8_t* scale, cudaStream_t s) {
  DeviceInfo dev;
  const rnl_status st = current_device(&dev);
  if (st != RNL_OK) return st;
  QuantArgs p;
  p.x = static_cast<const uint4*>(x);
  p.residual = static_cast<const uint4*>(residual);
  p.x_sum = static_cast<uint4*>(x_sum);
  p.gamma = static_cast<const uint4*>(gamma);
  p.nvec = static_cast<int>(K / 8);
  p.inv_d = static_cast<float>(1.0 / static_cast<double>(K));
  p.eps = eps;
  p.codes = reinterpret_cast<uint2*>(codes);
  p.scale = scale;
  trace_before(s);
  cudaError_t e;
  if (!norm)
    e = launch_blk<0>(p, T, block, dev.sm_count, s);
  else if (mode == RNL_NORM_RSQRT)
    e = launch_blk<1>(p, T, block, dev.sm_count, s);
  else
    e = launch_blk<2>(p, T, block, dev.sm_count, s);
  trace_after(s, norm ? "add_norm_mxfp8" : "quant_mxfp8");
  return e == cudaSuccess ? RNL_OK : RNL_ERR_LAUNCH;
}

}  // namespace rnl
