// ropeaxes.cu -- the V stage after the qkv projection (qkvrope.cu) with
// positions of several axes (time, height and width of a video, row and column
// of an image):
//
//   y [T, (Hq + 2 Hkv) * D] bf16: q heads, then k heads, then v heads
//   q / k head row h:  z = h, or with gammas bf16((h * rsqrt(mean(h^2) + eps)) * gamma)
//                      o[i]       = bf16(z[i] c_i - z[i + D/2] s_i)
//                      o[i + D/2] = bf16(z[i + D/2] c_i + z[i] s_i),  i < D/2
//   with (c_i, s_i) in column i of the angle table's row positions[axis(i), t];
//   v heads are copied.
//
// HBM bound: every head row is read once and written once, the table's rows
// come from L2.  A warp takes one token's heads in groups of 4 loads; D / 16
// lanes hold a head, each 8 elements (16 bytes) of its lower half and the 8
// rotation partners, so that the rotation needs no shuffle.  A token's angles
// are gathered once a warp: 8 pairs a lane, four 16-byte loads where the lane's
// pairs share an axis, 16 loads otherwise.  The sums of squares are added in
// the order of qkvrope.cu's kernel (its lane's R = D / 64 elements of either
// half, then a tree over its 32 lanes), so that one axis gives the same bits.
// Measured: 18433 tokens of 48 heads of 64 without norm 43 us (5.2 TB/s); 4096
// tokens of 48 heads of 128 with norm 31 us, where loads wait for the norm's
// arithmetic (32768 tokens: 4.5 TB/s, without norm 5.5).
#include <cuda_bf16.h>

#include <atomic>

#include "internal.h"
#include "ptx.cuh"

namespace rnl {
namespace {

__device__ unsigned int g_err_axes;  // kErrArg | site: a position outside [0, P)
std::atomic<bool> g_launched{false};

constexpr int kWarps = 4;
constexpr int kMinCtas = 5;  // by registers (102); 4 for head_dim 64 without it, 47 against 43 us at 18433 tokens
constexpr int kGroups = 4;  // head groups a warp has in flight

struct AxisMap {
  uint8_t a[128];  // axis of pair i, i < D/2
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float bf16_round(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }

template <int D>
__global__ void __launch_bounds__(kWarps * 32, kMinCtas)
    qkv_rope_axes_kernel(const __nv_bfloat16* __restrict__ y, int64_t T, int Hq, int Hkv, int parts, int per,
                         const __nv_bfloat16* __restrict__ q_gamma, const __nv_bfloat16* __restrict__ k_gamma,
                         float eps, const int* __restrict__ pos, const float* __restrict__ cs, int P,
                         __nv_bfloat16* __restrict__ q, __nv_bfloat16* __restrict__ k,
                         __nv_bfloat16* __restrict__ v, const __grid_constant__ AxisMap map) {
  constexpr int kLanes = D / 16;       // lanes a head
  constexpr int kHeads = 32 / kLanes;  // heads a group
  constexpr int kR = D / 64;           // elements of either half in a partial sum
  constexpr int kM = 8 / kR;           // partial sums a lane
  constexpr int kHalf = D / 2;
  const int lane = threadIdx.x & 31, sub = lane % kLanes;
  const int H = Hq + 2 * Hkv, nqk = Hq + Hkv;
  const int64_t wid = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (wid >= T * parts) return;
  const int64_t t = wid / parts;
  const int h0 = static_cast<int>(wid - t * parts) * per * kHeads;
  const int h1 = min(h0 + per * kHeads, H);  // the warp's heads [h0, h1)
  const __nv_bfloat16* yt = y + t * H * D + sub * 8;
  uint4 lo[kGroups], hi[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int h = h0 + g * kHeads + lane / kLanes;
    if (h < h1 && RNL_DCHECK(&g_err_axes, t < T && h >= 0 && h < H, 102)) {
      lo[g] = __ldg(reinterpret_cast<const uint4*>(yt + static_cast<int64_t>(h) * D));
      hi[g] = __ldg(reinterpret_cast<const uint4*>(yt + static_cast<int64_t>(h) * D + kHalf));
    }
  }
  float c[8], sn[8];
  bool p_ok = true;
  if (h0 < nqk) {  // some head of the warp is turned
    const int a0 = map.a[sub * 8];
    bool one = true;
#pragma unroll
    for (int e = 1; e < 8; ++e) one = one && map.a[sub * 8 + e] == a0;
    int p[8];
    p[0] = __ldg(pos + a0 * T + t);
#pragma unroll
    for (int e = 1; e < 8; ++e) p[e] = one ? p[0] : __ldg(pos + map.a[sub * 8 + e] * T + t);
    bool ok = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) ok = ok && p[e] >= 0 && p[e] < P;
    p_ok = __all_sync(0xffffffffu, ok);
    if (!p_ok) {  // nothing is read from the table; the caller gets RNL_ERR_ARG
      if (lane == 0) atomicCAS(&g_err_axes, 0u, kErrArg | (41u << 8));
    } else if (one) {
      const float4* row = reinterpret_cast<const float4*>(cs + static_cast<int64_t>(p[0]) * D + sub * 8);
      const float4 u0 = __ldg(row), u1 = __ldg(row + 1), w0 = __ldg(row + kHalf / 4), w1 = __ldg(row + kHalf / 4 + 1);
      c[0] = u0.x, c[1] = u0.y, c[2] = u0.z, c[3] = u0.w, c[4] = u1.x, c[5] = u1.y, c[6] = u1.z, c[7] = u1.w;
      sn[0] = w0.x, sn[1] = w0.y, sn[2] = w0.z, sn[3] = w0.w, sn[4] = w1.x, sn[5] = w1.y, sn[6] = w1.z, sn[7] = w1.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float* col = cs + static_cast<int64_t>(p[e]) * D + sub * 8 + e;
        c[e] = __ldg(col);
        sn[e] = __ldg(col + kHalf);
      }
    }
  }
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    if (h0 + g * kHeads >= h1) break;
    const int h = h0 + g * kHeads + lane / kLanes;
    const bool live = h < h1, turned = live && h < nqk, is_q = h < Hq;
    const __nv_bfloat16* gamma = is_q ? q_gamma : k_gamma;
    float fl[8], fh[8];
    unpack8(lo[g], fl);
    unpack8(hi[g], fh);
    if (q_gamma != nullptr || k_gamma != nullptr) {
      float part[kM];
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        part[m] = 0.f;
        if (turned) {
#pragma unroll
          for (int e = 0; e < kR; ++e) part[m] = fmaf(fl[m * kR + e], fl[m * kR + e], part[m]);
#pragma unroll
          for (int e = 0; e < kR; ++e) part[m] = fmaf(fh[m * kR + e], fh[m * kR + e], part[m]);
        }
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
        for (int m = 0; m < kM; ++m) part[m] += __shfl_xor_sync(0xffffffffu, part[m], o);
#pragma unroll
      for (int o = kM / 2; o > 0; o >>= 1)
#pragma unroll
        for (int m = 0; m < o; ++m) part[m] += part[m + o];
      if (turned && gamma != nullptr) {
        const float r = rsqrtf(part[0] * (1.0f / D) + eps);
        float gl[8], gh[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(gamma + sub * 8)), gl);
        unpack8(__ldg(reinterpret_cast<const uint4*>(gamma + kHalf + sub * 8)), gh);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          fl[e] = bf16_round(__fmul_rn(__fmul_rn(fl[e], r), gl[e]));
          fh[e] = bf16_round(__fmul_rn(__fmul_rn(fh[e], r), gh[e]));
        }
      }
    }
    if (!live || !RNL_DCHECK(&g_err_axes, h < H && sub * 8 + 8 <= kHalf, 103)) continue;
    if (!turned) {  // a v head: copied
      __nv_bfloat16* dst = v + (t * Hkv + (h - nqk)) * D + sub * 8;
      *reinterpret_cast<uint4*>(dst) = lo[g];
      *reinterpret_cast<uint4*>(dst + kHalf) = hi[g];
      continue;
    }
    if (!p_ok) continue;
    float ol[8], oh[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ol[e] = __fsub_rn(__fmul_rn(fl[e], c[e]), __fmul_rn(fh[e], sn[e]));
      oh[e] = __fadd_rn(__fmul_rn(fh[e], c[e]), __fmul_rn(fl[e], sn[e]));
    }
    __nv_bfloat16* dst = (is_q ? q + (t * Hq + h) * D : k + (t * Hkv + (h - Hq)) * D) + sub * 8;
    *reinterpret_cast<uint4*>(dst) = pack8(ol);
    *reinterpret_cast<uint4*>(dst + kHalf) = pack8(oh);
  }
}

template <int D>
void launch(const void* y, int64_t T, int64_t Hq, int64_t Hkv, const void* q_gamma, const void* k_gamma,
            float eps, const int32_t* positions, const float* cos_sin, int64_t max_pos, void* q, void* k,
            void* v, const AxisMap& map, cudaStream_t s) {
  constexpr int kHeads = 512 / D;  // heads a group
  const int64_t groups = (Hq + 2 * Hkv + kHeads - 1) / kHeads;
  const int64_t parts = (groups + kGroups - 1) / kGroups;  // warps a token, their groups spread evenly
  const int64_t per = (groups + parts - 1) / parts;
  const unsigned blocks = static_cast<unsigned>((T * parts + kWarps - 1) / kWarps);
  qkv_rope_axes_kernel<D><<<blocks, kWarps * 32, 0, s>>>(
      static_cast<const __nv_bfloat16*>(y), T, static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(parts), static_cast<int>(per),
      static_cast<const __nv_bfloat16*>(q_gamma), static_cast<const __nv_bfloat16*>(k_gamma), eps, positions, cos_sin,
      static_cast<int>(max_pos), static_cast<__nv_bfloat16*>(q), static_cast<__nv_bfloat16*>(k),
      static_cast<__nv_bfloat16*>(v), map);
}

}  // namespace

rnl_status launch_qkv_rope_axes(const void* y, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                                const void* q_gamma, const void* k_gamma, float eps,
                                const int32_t* positions, const uint8_t* axis_of_pair,
                                const float* cos_sin, int64_t max_pos, void* q, void* k, void* v,
                                cudaStream_t s) {
  if (T * (Hq + 2 * Hkv) == 0) return RNL_OK;
  g_launched.store(true, std::memory_order_relaxed);
  AxisMap map = {};
  for (int64_t i = 0; i < D / 2; ++i) map.a[i] = axis_of_pair[i];
  trace_before(s);
  if (D == 64)
    launch<64>(y, T, Hq, Hkv, q_gamma, k_gamma, eps, positions, cos_sin, max_pos, q, k, v, map, s);
  else if (D == 128)
    launch<128>(y, T, Hq, Hkv, q_gamma, k_gamma, eps, positions, cos_sin, max_pos, q, k, v, map, s);
  else
    launch<256>(y, T, Hq, Hkv, q_gamma, k_gamma, eps, positions, cos_sin, max_pos, q, k, v, map, s);
  const rnl_status st = cudaGetLastError() == cudaSuccess ? RNL_OK : RNL_ERR_LAUNCH;
  trace_after(s, "qkv_rope_axes");
  return st;
}

rnl_status read_clear_error_axes(unsigned int* word) {
  if (!g_launched.load(std::memory_order_relaxed)) return RNL_OK;
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_axes, sizeof v) != cudaSuccess) return RNL_ERR_LAUNCH;
  if (v != 0 && cudaMemcpyToSymbol(g_err_axes, &zero, sizeof zero) != cudaSuccess) return RNL_ERR_LAUNCH;
  *word = v;
  return RNL_OK;
}

}  // namespace rnl
