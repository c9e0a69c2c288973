// kv4.cuh -- device-side pieces of the 4-bit paged KV cache that its writer,
// its reader and the attention kernels share: the element format and the walk
// from a row of the call to its sequence and page.
//
// Format (MX with E2M1 elements): a block of 32 or 64 elements of one token's
// head row shares the power of two 2^X; element = E2M1 value (0, 0.5, 1, 1.5,
// 2, 3, 4, 6 and their negatives) * 2^X.  Two significant bits: the product is
// exact in bf16 and in binary32, and the E2M1 value alone is exact in binary16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace rnl {
namespace kv4 {

// One side (keys or values) of the cache: codes [pages, Hkv, page, D / 2],
// scale bytes [pages, Hkv, page, D / block].
struct Side {
  uint8_t* codes;
  uint8_t* scales;
};

// The cache and the sequences of a call, as the kernels take them.
struct Args {
  Side k, v;
  int n_pages, Hkv, page, page_shift;  // page = tokens a page, a power of two
  int D, d_shift, block_shift;         // D = 1 << d_shift; log2 of the elements a scale covers
  const int* table;                    // [n_seqs, max_pages]
  const int* lens;                     // [n_seqs]
  const int* cu;                       // [n_seqs + 1] or null: one row a sequence
  int n_seqs, max_pages;
  int n_rows;
};

inline Args make_args(const rnl_kv4_cache& c, const rnl_kv4_seqs& q) {
  Args a;
  a.k = {static_cast<uint8_t*>(c.k_codes), static_cast<uint8_t*>(c.k_scales)};
  a.v = {static_cast<uint8_t*>(c.v_codes), static_cast<uint8_t*>(c.v_scales)};
  a.n_pages = static_cast<int>(c.n_pages);
  a.Hkv = static_cast<int>(c.n_kv_heads);
  a.page = static_cast<int>(c.page_size);
  a.page_shift = 0;
  while ((1 << a.page_shift) < a.page) ++a.page_shift;
  a.D = static_cast<int>(c.head_dim);
  a.d_shift = c.head_dim == 64 ? 6 : c.head_dim == 128 ? 7 : 8;
  a.block_shift = c.block == 64 ? 6 : 5;
  a.table = q.block_table;
  a.lens = q.seq_lens;
  a.cu = q.cu_rows;
  a.n_seqs = static_cast<int>(q.n_seqs);
  a.max_pages = static_cast<int>(q.max_pages);
  a.n_rows = static_cast<int>(q.n_rows);
  return a;
}

// First row, row count and cached length of sequence b; false (and the error
// word set) where the device-side data is out of range: the caller leaves
// that sequence alone.
struct Seq {
  int row0, rows, len;
};
__device__ __forceinline__ bool load_seq(const Args& a, int b, Seq& s, unsigned int* err, uint32_t site) {
  s.row0 = a.cu != nullptr ? __ldg(a.cu + b) : b;
  const int end = a.cu != nullptr ? __ldg(a.cu + b + 1) : b + 1;
  s.rows = end - s.row0;
  s.len = __ldg(a.lens + b);
  const bool ok = s.row0 >= 0 && end >= s.row0 && end <= a.n_rows && s.len >= 0 &&
                  s.len <= static_cast<int64_t>(a.max_pages) * a.page;
  if (!ok) {
    atomicCAS(err, 0u, kErrArg | (site << 8));
    s.rows = 0;
    s.len = 0;
  }
  return ok;
}

// The sequence that row t belongs to: the last b with cu[b] <= t, found by
// the whole warp (32 probes a step).  -1 where no sequence covers the row.
__device__ __forceinline__ int seq_of_row(const Args& a, int t) {
  if (a.cu == nullptr) return t < a.n_seqs ? t : -1;
  int lo = 0, n = a.n_seqs;  // the answer + 1 lies in [lo, lo + n]
  const int lane = threadIdx.x & 31;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lo + (lane + 1) * step - 1;  // last index of this lane's part
    const bool le = i < lo + n ? __ldg(a.cu + i) <= t : false;
    const int full = __popc(__ballot_sync(0xffffffffu, le));
    const int left = n - full * step;
    lo += full * step;
    n = left < step - 1 ? left : step - 1;
    if (n < 0) n = 0;
  }
  const int b = lo - 1;
  if (b < 0 || t >= __ldg(a.cu + b + 1)) return -1;
  return b;
}

// The cache row (page * Hkv + head) * page + offset of token position pos, or
// -1 for a page id outside the cache (error word set).
__device__ __forceinline__ int64_t token_row(const Args& a, int b, int pos, int head, unsigned int* err,
                                             uint32_t site) {
  const int p = __ldg(a.table + static_cast<int64_t>(b) * a.max_pages + (pos >> a.page_shift));
  if (p < 0 || p >= a.n_pages) {
    atomicCAS(err, 0u, kErrArg | (site << 8));
    return -1;
  }
  return ((static_cast<int64_t>(p) * a.Hkv + head) << a.page_shift) + (pos & (a.page - 1));
}

// Whether n tokens from cache row `row` on lie in the cache (for the debug build's checks).
__device__ __forceinline__ bool in_cache(const Args& a, int64_t row, int n) {
  return row >= 0 && row + n <= (static_cast<int64_t>(a.n_pages) * a.Hkv << a.page_shift);
}

// 8 codes -> 4 half2 of consecutive elements (exact).
__device__ __forceinline__ void e2m1x8_to_half(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// 8 values -> 8 codes (element 0 in the lowest nibble), round to nearest
// even, saturating at 6.
__device__ __forceinline__ uint32_t e2m1x8_code(const float (&f)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return w;
}

// 2^(byte - 127) in binary32 (byte 0 is the subnormal 2^-127; byte 255, the
// E8M0 NaN, gives an infinity, so that what it scales is not finite).
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

// ---- attention (kv4attn.cu, kv4prompt.cu)
constexpr float kLn2 = 0.6931471805599453f;

struct AttnParams {
  const __nv_bfloat16* q;
  int64_t q_stride;
  __nv_bfloat16* out;
  float* lse;
  float* part;   // partial sums: 2 slots a CTA
  int4* rec;     // [CTAs]: the cut item a CTA begins (item, sequence, last CTA), .x = -1: none
  float scale_log2;
  int Hq, G;
  int causal, window;
  int few;  // sequences of up to this many rows (times G) are the few-row kernel's, the others the prompt kernel's
};

// mbar_wait (ptx.cuh) for waits that are short and many: a tight loop first, in
// which a poll costs few issue slots, the timer only after it.
__device__ __forceinline__ bool quick_wait(uint32_t bar, uint32_t parity, volatile int* abort, unsigned int* err,
                                           uint32_t site) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 n;\n\t"
      "mov.b32 n, 0;\n\t"
      "POLL:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "@p bra DONE;\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.lt.u32 q, n, 256;\n\t"
      "@q bra POLL;\n\t"
      "DONE:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000)
      : "memory");
  return ok != 0 || mbar_wait(bar, parity, abort, err, site);
}

// After a wait has given up: what the CTA still has in flight is waited for all
// the same (with a limit of its own), before its shared memory or TMEM goes back.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > kWaitLimitNs) return;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ __half2 h2(uint32_t a) { return *reinterpret_cast<const __half2*>(&a); }
__device__ __forceinline__ uint32_t u32(__half2 a) { return *reinterpret_cast<const uint32_t*>(&a); }

// 2^x; results below binary32's normal range become 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^(byte - 127) with 0 for byte 0 (and an infinity for 255, E8M0's NaN).
__device__ __forceinline__ float byte_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// 2^e; the clamp is reached only where what it scales vanishes anyway.
__device__ __forceinline__ float pow2i(int e) {
  return __uint_as_float(static_cast<uint32_t>(min(max(e, -126), 127) + 127) << 23);
}
// 2^e for |e| up to 250, subnormal or infinite outside binary32's range.
__device__ __forceinline__ float pow2w(int e) { return pow2i(e / 2) * pow2i(e - e / 2); }

// Eight dims of row r of key head kvh: sums v over weights ll with maximum mm.
template <int D>
__device__ __forceinline__ void store_row(const AttnParams& p, const Seq& s, int kvh, int r, int d,
                                          const float (&v)[8], float mm, float ll) {
  const int tok = r / p.G;
  const int64_t row = static_cast<int64_t>(s.row0 + tok) * p.Hq + kvh * p.G + (r - tok * p.G);
  const float inv = ll != 0.f ? 1.f / ll : 0.f;
  uint32_t w[4];
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * y] * inv, v[2 * y + 1] * inv);
    w[y] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p.out + row * D + d) = make_uint4(w[0], w[1], w[2], w[3]);
  if (d == 0 && p.lse != nullptr) p.lse[row] = ll != 0.f ? mm * kLn2 + logf(ll) : -INFINITY;
}

// Rows taken by themselves.  The rows of an item share their operands, and with
// them the reference scale R: E2M1 * 2^(X - R + 13) is exact in binary16 for
// X >= R - kSpread only.  Where a token that some of the rows do not read (later
// in a causal prompt, older than their window) is so much larger than others,
// R would be that token's and the rest would vanish for those rows too.  The
// kernels see that from the scale bytes of the tiles that the mask cuts, and
// such an item's rows are computed by one_row instead.
constexpr int kSpread = 36;

// So are rows with scores this large (in log2 units): the exponents of their
// weights come from one FMA, score times factor less the rounded maximum, which
// is half a step of the maximum off, from here on enough to take the largest
// weight out of binary16 or to nothing.
constexpr float kTopScore = 4194304.f;

// A warp computes row r of key head kvh over the tokens of [lo, hi) that it
// reads, in FP32 straight from the cache: a token a lane for the scores, D / 32
// dims a lane for the sums v.  m is the maximum in log2 units, l the sum of the
// weights 2^(x - m).
template <int D>
__device__ __forceinline__ void one_row(const Args& a, const AttnParams& p, const Seq& s, int b, int kvh, int r,
                                        int lo, int hi, unsigned int* err, uint32_t site, float& m, float& l,
                                        float (&v)[D / 32]) {
  const int lane = threadIdx.x & 31;
  const int tok_q = r / p.G;
  const int pos = p.causal ? s.len - s.rows + tok_q : s.len - 1;
  lo = max(max(lo, 0), p.window > 0 ? pos - p.window + 1 : 0);
  hi = min(hi, pos + 1);
  const __nv_bfloat16* q = p.q + (s.row0 + tok_q) * p.q_stride + static_cast<int64_t>(kvh * p.G + (r - tok_q * p.G)) * D;
  uint32_t am = 0;
  for (int i = lane; i < D / 2; i += 32) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(q) + i);
    am = max(am, max((w << 16) & 0x7FFFFFFFu, w & 0x7FFF0000u));
  }
  // q is taken times 2^-e, below 2, and a block's scale times 2^-16, so that no sum overflows
  const int e = max(static_cast<int>(__reduce_max_sync(0xffffffffu, am) >> 23), 1) - 127;
  const float q1 = pow2i(-e / 2), q2 = pow2i(-e - (-e) / 2);
  const float f1 = pow2i((e + 16) / 2), f2 = pow2i(e + 16 - (e + 16) / 2);
  const int n_blocks = D >> a.block_shift, words = 1 << (a.block_shift - 3);
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) v[i] = 0.f;
  for (int t0 = lo; t0 < hi; t0 += 32) {
    const int64_t row = t0 + lane < hi ? token_row(a, b, t0 + lane, kvh, err, site) : -1;
    float x = -INFINITY;
    if (row >= 0) {
      const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.k.codes + row * (D / 2));
      float sum = 0.f;
      bool finite = true;
#pragma unroll 1
      for (int c = 0; c < n_blocks; ++c) {
        const uint32_t byte = __ldg(a.k.scales + row * n_blocks + c);
        finite = finite && byte != 255u && __ldg(a.v.scales + row * n_blocks + c) != 255u;
        float part = 0.f;
#pragma unroll 1
        for (int w = c * words; w < (c + 1) * words; ++w) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(q) + w);
          const uint32_t qw[4] = {u.x, u.y, u.z, u.w};
          uint32_t h[4];
          e2m1x8_to_half(__ldg(codes + w), h);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float2 k2 = __half22float2(h2(h[y]));
            part = fmaf(__uint_as_float(qw[y] << 16) * q1 * q2, k2.x, part);
            part = fmaf(__uint_as_float(qw[y] & 0xFFFF0000u) * q1 * q2, k2.y, part);
          }
        }
        sum = fmaf(part, byte_scale(byte) * (1.f / 65536.f), sum);
      }
      x = finite ? sum * p.scale_log2 * f1 * f2 : NAN;
    }
    float mx = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
    const float al = ex2(m - mu), w = ex2(x - mu);
    m = mn;
    float all = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    l = fmaf(l, al, all);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) v[i] *= al;
#pragma unroll 1
    for (int j = 0; j < 32; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const int64_t rj = __shfl_sync(0xffffffffu, row, j);
      if (wj == 0.f) continue;
      const uint8_t* c = a.v.codes + rj * (D / 2) + lane * (D / 64);
      uint32_t code;
      if constexpr (D == 64) code = __ldg(c);
      else if constexpr (D == 128) code = __ldg(reinterpret_cast<const uint16_t*>(c));
      else code = __ldg(reinterpret_cast<const uint32_t*>(c));
      const float f = wj * byte_scale(__ldg(a.v.scales + rj * n_blocks + ((lane * (D / 32)) >> a.block_shift)));
      uint32_t h[4];
      e2m1x8_to_half(code, h);
#pragma unroll
      for (int i = 0; i < D / 32; i += 2) {
        const float2 z = __half22float2(h2(h[i / 2]));
        v[i] = fmaf(z.x, f, v[i]);
        v[i + 1] = fmaf(z.y, f, v[i + 1]);
      }
    }
  }
}

// one_row's result as an output row, or as row i of a partial of `rows` rows.
template <int D>
__device__ __forceinline__ void store_one_row(const AttnParams& p, const Seq& s, int kvh, int r, float m, float l,
                                              const float (&v)[D / 32], float* partial, int i, int rows) {
  const int lane = threadIdx.x & 31, d = lane * (D / 32);
  if (partial != nullptr) {
#pragma unroll
    for (int x = 0; x < D / 32; ++x) partial[i * D + d + x] = v[x];
    if (lane == 0) {
      partial[rows * D + i] = m;
      partial[rows * D + rows + i] = l;
    }
    return;
  }
  const int tok = r / p.G;
  const int64_t row = static_cast<int64_t>(s.row0 + tok) * p.Hq + kvh * p.G + (r - tok * p.G);
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int x = 0; x < D / 32; x += 2)
    *reinterpret_cast<__nv_bfloat162*>(p.out + row * D + d + x) = __floats2bfloat162_rn(v[x] * inv, v[x + 1] * inv);
  if (lane == 0 && p.lse != nullptr) p.lse[row] = l != 0.f ? m * kLn2 + logf(l) : -INFINITY;
}

__device__ __forceinline__ int64_t range_start(int64_t units, int c, int n) { return units * c / n; }

}  // namespace kv4

// Sequences of more than p.few rows (kv4prompt.cu), head_dim 64 or 128.
bool kv4_prompt_fits(int64_t D);
size_t kv4_prompt_workspace_bytes(int64_t D);
rnl_status launch_kv4_prompt(const kv4::AttnParams& p, const kv4::Args& a, int block, void* ws,
                             const DeviceInfo& dev, cudaStream_t s);

}  // namespace rnl
