// kv4attn.cu -- attention over the 4-bit paged KV cache (kv4.cuh):
//
//   out[t, h] = sum_j p_j v[j] / sum_j p_j,   p_j = exp(scale q[t, h] . k[j] - max)
//
// over the tokens j of the row's sequence that the mask leaves it.
#include "kv4.cuh"

namespace rnl {
namespace {

using namespace kv4;

__device__ unsigned int g_err_kv4attn;

constexpr int kSimpleWarps = 4;

// One CTA per (row, query head); its warps take every fourth token, the
// running maximum, sum and weighted values in binary32 registers.
template <int D>
__global__ void __launch_bounds__(kSimpleWarps * 32)
    kv4_attn_simple_kernel(const __nv_bfloat16* __restrict__ q, int64_t q_stride, int Hq, float scale_log2,
                           bool causal, int window, const Args a, __nv_bfloat16* __restrict__ out,
                           float* __restrict__ lse) {
  constexpr int R = D / 32;  // dims per lane
  const int t = blockIdx.x / Hq, h = blockIdx.x - t * Hq;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = seq_of_row(a, t);
  if (b < 0) return;
  Seq s;
  if (!load_seq(a, b, s, &g_err_kv4attn, 45)) return;
  if (t < s.row0) return;
  const int kvh = h / (Hq / a.Hkv);
  int lo = 0, hi = s.len;
  if (causal) {
    const int pos = s.len - s.rows + (t - s.row0);
    hi = pos + 1;
    if (window > 0 && pos + 1 > window) lo = pos + 1 - window;
  }
  float qf[R], acc[R];
#pragma unroll
  for (int e = 0; e < R; ++e) {
    qf[e] = __bfloat162float(q[t * q_stride + static_cast<int64_t>(h) * D + lane * R + e]) * scale_log2;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int sd = D >> a.block_shift, sj = (lane * R) >> a.block_shift;
  for (int j = lo + warp; j < hi; j += kSimpleWarps) {
    const int64_t row = token_row(a, b, j, kvh, &g_err_kv4attn, 46);
    if (row < 0) continue;
    auto value = [&](const Side& side, int e, float sc) {
      const int d = lane * R + e;
      const uint32_t byte = side.codes[(row * D + d) / 2];
      const uint32_t c = (d & 1) ? byte >> 4 : byte & 15;
      const float mag = (c & 7) < 2 ? 0.5f * (c & 7) : (1.f + 0.5f * (c & 1)) * static_cast<float>(1 << (((c & 7) >> 1) - 1));
      return ((c & 8) ? -mag : mag) * sc;
    };
    const float ks = e8m0_value(a.k.scales[row * sd + sj]), vs = e8m0_value(a.v.scales[row * sd + sj]);
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < R; ++e) dot = fmaf(qf[e], value(a.k, e, ks), dot);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    const float mn = fmaxf(m, dot);
    const float f = exp2f(m - mn), p = exp2f(dot - mn);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < R; ++e) acc[e] = fmaf(p, value(a.v, e, vs), acc[e] * f);
    m = mn;
  }
  __shared__ float sm[kSimpleWarps], sl[kSimpleWarps], so[kSimpleWarps][D];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < R; ++e) so[warp][lane * R + e] = acc[e];
  __syncthreads();
  float mm = -INFINITY, ll = 0.f;
  for (int w = 0; w < kSimpleWarps; ++w) mm = fmaxf(mm, sm[w]);
  float f[kSimpleWarps];
  for (int w = 0; w < kSimpleWarps; ++w) {
    f[w] = sl[w] != 0.f ? exp2f(sm[w] - mm) : 0.f;
    ll += sl[w] * f[w];
  }
  const int64_t o = (static_cast<int64_t>(t) * Hq + h) * D;
  for (int d = threadIdx.x; d < D; d += kSimpleWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kSimpleWarps; ++w) x = fmaf(so[w][d], f[w], x);
    out[o + d] = __float2bfloat16_rn(ll != 0.f ? x / ll : 0.f);
  }
  if (lse != nullptr && threadIdx.x == 0)
    lse[static_cast<int64_t>(t) * Hq + h] = ll != 0.f ? mm * 0.6931471805599453f + logf(ll) : -INFINITY;
}

}  // namespace

size_t kv4_attn_workspace_bytes(int64_t T, int64_t D, int64_t Hq, int64_t Hkv) { return 0; }

rnl_status launch_kv4_attention(const Kv4AttnArgs& x, const rnl_kv4_cache& c, const rnl_kv4_seqs& q,
                                cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>(q.n_rows * x.Hq);
  const float sl = x.scale * 1.4426950408889634f;
  const Args a = make_args(c, q);
  const auto* qp = static_cast<const __nv_bfloat16*>(x.q);
  auto* op = static_cast<__nv_bfloat16*>(x.out);
  const int hq = static_cast<int>(x.Hq), w = static_cast<int>(x.window);
  trace_before(s);
  if (a.D == 64)
    kv4_attn_simple_kernel<64><<<blocks, kSimpleWarps * 32, 0, s>>>(qp, x.q_stride, hq, sl, x.causal, w, a, op, x.lse);
  else if (a.D == 128)
    kv4_attn_simple_kernel<128><<<blocks, kSimpleWarps * 32, 0, s>>>(qp, x.q_stride, hq, sl, x.causal, w, a, op, x.lse);
  else
    kv4_attn_simple_kernel<256><<<blocks, kSimpleWarps * 32, 0, s>>>(qp, x.q_stride, hq, sl, x.causal, w, a, op, x.lse);
  const rnl_status st = cudaGetLastError() == cudaSuccess ? RNL_OK : RNL_ERR_LAUNCH;
  trace_after(s, "kv4_attn");
  return st;
}

rnl_status read_clear_error_kv4attn(unsigned int* word) {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_kv4attn, sizeof v) != cudaSuccess) return RNL_ERR_LAUNCH;
  if (v != 0 && cudaMemcpyToSymbol(g_err_kv4attn, &zero, sizeof zero) != cudaSuccess)
    return RNL_ERR_LAUNCH;
  *word = v;
  return RNL_OK;
}

}  // namespace rnl
