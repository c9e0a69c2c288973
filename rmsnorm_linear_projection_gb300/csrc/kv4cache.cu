// kv4cache.cu -- writing and reading back the 4-bit paged KV cache.
//
//   append: for row i of a sequence with r rows and cached length n (the r
//   rows counted), the token at position n - r + i gets, per head and block of
//   32 or 64 elements x of its k (v) row,
//     X     = floor(log2 max|x|) - 2, at least -127  (2 = E2M1's largest
//             exponent; an all-zero block gets -127)
//     scale = X + 127                                (the E8M0 byte; a block
//             with an infinity or NaN gets 255)
//     code  = E2M1(x * 2^-X)                         nearest even, saturating
//   gather: the same positions read back, value(code) * 2^X, exact in bf16.
//
// Both are bound by their bf16 traffic (2 bytes an element against 0.53 for
// codes and scales).  One warp takes 1024 elements of one row, of k and of v:
// every lane moves 8 elements (16 bytes of bf16, 4 bytes of codes) an access,
// eight accesses on their way at once, and the sequence is looked up once for
// both sides; the writer's loads do not wait for it.  Measured at a captured
// call, cold: prefixes of 9000 to 20000 tokens read back at 5.4 TB/s (10 of
// them: 6.35), prompts written and read back at 3.7 TB/s (20 of them: 4.95);
// 512 elements a warp were slower (50 against 43 us for either).
#include <atomic>

#include "kv4.cuh"

namespace rnl {
namespace {

using namespace kv4;

__device__ unsigned int g_err_kv4cache;
std::atomic<bool> g_launched{false};

constexpr int kCacheWarps = 4;
constexpr int kVecs = 4;  // 8-element vectors of a row that a lane takes

// The row and chunk of this warp.
__device__ __forceinline__ bool warp_job(const Args& a, int chunks, int& t, int& chunk) {
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kCacheWarps + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(a.n_rows) * chunks) return false;
  t = static_cast<int>(w / chunks);
  chunk = static_cast<int>(w - static_cast<int64_t>(t) * chunks);
  return true;
}

// The cache row of head 0 for row t, -1 where there is none.
__device__ __forceinline__ int64_t row_of(const Args& a, int t) {
  const int b = seq_of_row(a, t);
  if (b < 0) return -1;  // rows behind the last sequence are left alone
  Seq s;
  if (!load_seq(a, b, s, &g_err_kv4cache, 42) || t < s.row0) return -1;  // or cu_rows out of order
  const int pos = s.len - s.rows + (t - s.row0);
  if (pos < 0) {  // more rows than the length counts
    atomicCAS(&g_err_kv4cache, 0u, kErrArg | (43u << 8));
    return -1;
  }
  return token_row(a, b, pos, 0, &g_err_kv4cache, 44);
}

__global__ void __launch_bounds__(kCacheWarps * 32)
    kv4_append_kernel(const __nv_bfloat16* __restrict__ k, int64_t k_stride,
                      const __nv_bfloat16* __restrict__ v, int64_t v_stride, const Args a, int chunks) {
  int t, chunk;
  if (!warp_job(a, chunks, t, chunk)) return;
  const int n = a.Hkv * a.D;
  const int e0 = (chunk * kVecs * 32 + (threadIdx.x & 31)) * 8;
  const __nv_bfloat16* const src[2] = {k + t * k_stride, v + t * v_stride};
  uint4 x[2][kVecs];
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = e0 + i * 256;
      x[r][i] = e < n ? __ldg(reinterpret_cast<const uint4*>(src[r] + e)) : make_uint4(0, 0, 0, 0);
    }
  const int64_t row0 = row_of(a, t);
  if (row0 < 0) return;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const Side& side = r == 0 ? a.k : a.v;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = e0 + i * 256;
      float f[8];
      const uint32_t w[4] = {x[r][i].x, x[r][i].y, x[r][i].z, x[r][i].w};
      // the largest magnitude by its bits: a NaN or infinity gives exponent 255
      uint32_t am = 0;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        f[2 * p] = __uint_as_float(w[p] << 16);
        f[2 * p + 1] = __uint_as_float(w[p] & 0xFFFF0000u);
        am = max(am, max((w[p] << 16) & 0x7FFFFFFFu, w[p] & 0x7FFF0000u));
      }
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      if (a.block_shift == 6) am = max(am, __shfl_xor_sync(0xffffffffu, am, 4));
      const int eb = static_cast<int>(am >> 23);
      const int byte = eb == 255 ? 255 : max(eb - 2, 0);
      // 2^-X for X = byte - 127: exponent field 254 - byte, at least 1 (byte <= 252)
      const float inv = __uint_as_float(static_cast<uint32_t>(max(254 - byte, 1)) << 23);
#pragma unroll
      for (int p = 0; p < 8; ++p) f[p] = __fmul_rn(f[p], inv);
      if (e >= n) continue;
      const int head = e >> a.d_shift, d = e & (a.D - 1);
      const int64_t row = row0 + (static_cast<int64_t>(head) << a.page_shift);
      if (!RNL_DCHECK(&g_err_kv4cache, in_cache(a, row, 1) && head < a.Hkv && d + 8 <= a.D, 100)) continue;
      *reinterpret_cast<uint32_t*>(side.codes + ((row << a.d_shift) + d) / 2) = e2m1x8_code(f);
      if ((d & ((1 << a.block_shift) - 1)) == 0)
        side.scales[(row << (a.d_shift - a.block_shift)) + (d >> a.block_shift)] = static_cast<uint8_t>(byte);
    }
  }
}

__global__ void __launch_bounds__(kCacheWarps * 32)
    kv4_gather_kernel(const Args a, __nv_bfloat16* __restrict__ k, __nv_bfloat16* __restrict__ v, int chunks) {
  int t, chunk;
  if (!warp_job(a, chunks, t, chunk)) return;
  const int n = a.Hkv * a.D;
  const int e0 = (chunk * kVecs * 32 + (threadIdx.x & 31)) * 8;
  const int64_t row0 = row_of(a, t);
  if (row0 < 0) return;
  uint32_t c[2][kVecs], s[2][kVecs];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const Side& side = r == 0 ? a.k : a.v;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = e0 + i * 256;
      if (e < n) {
        const int head = e >> a.d_shift, d = e & (a.D - 1);
        const int64_t row = row0 + (static_cast<int64_t>(head) << a.page_shift);
        if (!RNL_DCHECK(&g_err_kv4cache, in_cache(a, row, 1) && head < a.Hkv && d + 8 <= a.D, 101)) return;
        c[r][i] = __ldg(reinterpret_cast<const uint32_t*>(side.codes + ((row << a.d_shift) + d) / 2));
        s[r][i] = __ldg(side.scales + (row << (a.d_shift - a.block_shift)) + (d >> a.block_shift));
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    __nv_bfloat16* dst = (r == 0 ? k : v) + static_cast<int64_t>(t) * n;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = e0 + i * 256;
      if (e >= n) break;
      uint32_t h[4], o[4];
      e2m1x8_to_half(c[r][i], h);
      const float p = e8m0_value(s[r][i]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[q]));
        const __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(f.x, p), __fmul_rn(f.y, p));
        o[q] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(dst + e) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

inline int chunks_of(const rnl_kv4_cache& c) {
  return static_cast<int>((c.n_kv_heads * c.head_dim + kVecs * 256 - 1) / (kVecs * 256));
}
inline unsigned blocks_of(const rnl_kv4_seqs& q, int chunks) {
  return static_cast<unsigned>((q.n_rows * chunks + kCacheWarps - 1) / kCacheWarps);
}

}  // namespace

rnl_status launch_kv4_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const rnl_kv4_cache& c, const rnl_kv4_seqs& q, cudaStream_t s) {
  g_launched.store(true, std::memory_order_relaxed);
  const int chunks = chunks_of(c);
  trace_before(s);
  kv4_append_kernel<<<blocks_of(q, chunks), kCacheWarps * 32, 0, s>>>(
      static_cast<const __nv_bfloat16*>(k), k_stride, static_cast<const __nv_bfloat16*>(v), v_stride,
      make_args(c, q), chunks);
  const rnl_status st = cudaGetLastError() == cudaSuccess ? RNL_OK : RNL_ERR_LAUNCH;
  trace_after(s, "kv4_append");
  return st;
}

rnl_status launch_kv4_gather(const rnl_kv4_cache& c, const rnl_kv4_seqs& q, void* k_out, void* v_out,
                             cudaStream_t s) {
  g_launched.store(true, std::memory_order_relaxed);
  const int chunks = chunks_of(c);
  trace_before(s);
  kv4_gather_kernel<<<blocks_of(q, chunks), kCacheWarps * 32, 0, s>>>(
      make_args(c, q), static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out), chunks);
  const rnl_status st = cudaGetLastError() == cudaSuccess ? RNL_OK : RNL_ERR_LAUNCH;
  trace_after(s, "kv4_gather");
  return st;
}

rnl_status read_clear_error_kv4cache(unsigned int* word) {
  if (!g_launched.load(std::memory_order_relaxed)) return RNL_OK;
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_kv4cache, sizeof v) != cudaSuccess) return RNL_ERR_LAUNCH;
  if (v != 0 && cudaMemcpyToSymbol(g_err_kv4cache, &zero, sizeof zero) != cudaSuccess)
    return RNL_ERR_LAUNCH;
  *word = v;
  return RNL_OK;
}

}  // namespace rnl
