// moe.cu -- the two ends of the grouped products: tokens to experts (top-k of
// the router's logits, softmax weights, the rows grouped by expert) and the
// weighted sum of a token's expert rows back.
//
// Routing (bound by latency: a few MB are read).  32 warps a CTA and 64 tokens, so
// that a warp has two tokens to choose for; with 8 warps of 8 tokens each, and
// the counts added up by as few threads, the two launches took 19.3 and 14.9 us
// for 8192 tokens over 128 experts, now 9.6 to 11 each (17.7 us a call in a graph).
// One warp a token: a lane holds every 32nd logit as an order-preserving integer, and
// k rounds of two warp reductions take the largest key and, among equals, the lowest
// expert.  The rows are grouped by a
// stable counting sort, (token, place) order within an expert: each CTA counts
// its tokens' choices, then adds up the counts of the CTAs before it and ranks
// its own choices warp by warp (match_any).  Nothing depends on the order of
// atomics: shared-memory atomics only count.  Both steps are one launch while a
// single CTA's tokens suffice, else two.
#include <cuda_bf16.h>

#include <atomic>

#include "internal.h"
#include "ptx_more.cuh"

namespace rnl {
namespace {

__device__ unsigned int g_err_moe;
std::atomic<bool> g_launched{false};

constexpr int kThreadsR = 1024;
constexpr int kWarpsR = kThreadsR / 32;
constexpr int kMinTokens = 64;  // tokens a CTA; more when there would be over kMaxBlocks CTAs
constexpr int kMaxBlocks = 256;

// Keys in the order of the logits; 0 for what is never chosen (NaN, -infinity).
// -0 counts as +0.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  if (v != v || u == 0xff800000u) return 0u;
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

struct RouteArgs {
  const float* logits;
  int64_t T;
  int E, k, per;  // per: tokens a CTA
  int renorm;
  int32_t* ids;
  float* weights;
  int32_t* offsets;
  int32_t* rows;
  int32_t* slots;
  int32_t* hist;  // [CTA][E]
};

// exp(v - m) with infinities of the same sign at distance 0
__device__ __forceinline__ float soft(float v, float m) { return v == m ? 1.0f : expf(v - m); }

template <int VPL>
__device__ __forceinline__ void load_keys(const RouteArgs& p, int64_t t, int lane, uint32_t (&key)[VPL]) {
  const float* l = p.logits + t * p.E;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < p.E ? key_of(l[e]) : 0u;
  }
}

// One token's choices from its keys (which are used up); lane j < k gets the j-th
// one's key, expert and weight (key 0: none).  VPL: logits a lane.
template <int VPL>
__device__ __forceinline__ void choose(const RouteArgs& p, int lane, uint32_t (&key)[VPL], uint32_t& my_key,
                                       int& my_id, float& my_w) {
  my_key = 0u;
  my_id = -1;
  float mx = 0.f, sum = 0.f;
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const uint32_t m = __reduce_max_sync(0xffffffffu, best);
    if (m == 0u) break;  // the same on every lane
    const uint32_t e = __reduce_min_sync(0xffffffffu, best == m ? static_cast<uint32_t>(lane + 32 * at) : 0xffffffffu);
    if (j == 0) {
      mx = logit_of(m);
      if (!p.renorm) {  // the softmax' sum over all experts
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (key[i] != 0u) sum += soft(logit_of(key[i]), mx);
      }
    }
    if (lane == j) {
      my_key = m;
      my_id = static_cast<int>(e);
    }
    // (a select for each, not a store to key[e / 32]: the keys stay in registers)
    const uint32_t gone = (e & 31u) == static_cast<uint32_t>(lane) ? e >> 5 : 0xffffffffu;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      uint32_t k = key[i];
      asm("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %1, %2;\n\tselp.u32 %0, 0, %0, p;\n\t}" : "+r"(k) : "r"(gone), "r"(i));
      key[i] = k;
    }
  }
  const float mine = my_key != 0u ? soft(logit_of(my_key), mx) : 0.f;
  if (p.renorm) sum = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  my_w = my_key != 0u ? mine / sum : 0.f;
}

// Counts of this CTA's choices into cnt [E] (shared), ids and weights out.
template <int VPL>
__device__ void choose_all(const RouteArgs& p, int64_t t0, int64_t t1, int* cnt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += kThreadsR) cnt[e] = 0;
  __syncthreads();
  constexpr bool kAhead = VPL <= 8;  // the next token's logits while this one's are looked through
  uint32_t key[VPL], next[kAhead ? VPL : 1];
  int64_t t = t0 + warp;
  if (kAhead && t < t1) load_keys<VPL>(p, t, lane, key);
  for (; t < t1; t += kWarpsR) {
    if constexpr (kAhead) {
      if (t + kWarpsR < t1) load_keys<VPL>(p, t + kWarpsR, lane, next);
    } else {
      load_keys<VPL>(p, t, lane, key);
    }
    uint32_t my_key;
    int id;
    float w;
    choose<VPL>(p, lane, key, my_key, id, w);
    if (lane < p.k) {
      p.ids[t * p.k + lane] = id;
      p.weights[t * p.k + lane] = w;
      if (id >= 0) atomicAdd(cnt + id, 1);
    }
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = next[i];
    }
  }
  __syncthreads();
}

// Warps that rank a CTA's choices: their counts, E values each, stay in 48 KB.
__host__ __device__ inline int rank_warps(int E) { return E <= 256 ? kWarpsR : 8; }

// before[e]: rows of expert e of the CTAs before this one; then the first row of
// expert e of this CTA.  Shared: before [E], total [E], wcnt [warps][E].
__device__ void place_all(const RouteArgs& p, int64_t t0, int64_t t1, int* before, int* total, int* wcnt) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ int warp_sum[kWarpsR];
  // exclusive scan of the totals over the experts
  int carry = 0;
  for (int e0 = 0; e0 < p.E; e0 += kThreadsR) {
    const int e = e0 + threadIdx.x;
    const int own = e < p.E ? total[e] : 0;
    int v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    int add = carry, all = carry;
    for (int i = 0; i < kWarpsR; ++i) {
      if (i < warp) add += warp_sum[i];
      all += warp_sum[i];
    }
    if (e < p.E) {
      before[e] += add + v - own;
      if (blockIdx.x == 0) p.offsets[e] = add + v - own;
    }
    carry = all;
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[p.E] = carry;
  // rows behind the last expert's
  for (int64_t i = carry + static_cast<int64_t>(blockIdx.x) * kThreadsR + threadIdx.x; i < p.T * p.k;
       i += static_cast<int64_t>(gridDim.x) * kThreadsR)
    p.rows[i] = -1;
  // each ranking warp takes an equal run of the CTA's choices, 32 at least
  const int64_t all_n = (t1 - t0) * p.k;
  const int rw = static_cast<int>(min(static_cast<int64_t>(rank_warps(p.E)), max(int64_t{1}, (all_n + 31) / 32)));
  const int64_t n = warp < rw ? all_n : 0;
  const int64_t run = ((n + rw - 1) / rw + 31) / 32 * 32;
  const int64_t i0 = t0 * p.k + warp * run;
  const int64_t end = t1 * p.k;
  const int64_t i1 = i0 + run < end ? i0 + run : end;  // (run 0 for the other warps: nothing)
  for (int i = threadIdx.x; i < rw * p.E; i += kThreadsR) wcnt[i] = 0;
  __syncthreads();
  int* mine = wcnt + (warp < rw ? warp : 0) * p.E;
  for (int64_t i = i0 + lane; i < i1; i += 32) {
    const int id = p.ids[i];
    if (id >= 0) atomicAdd(mine + id, 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreadsR) {
    int at = before[e];
    for (int w = 0; w < rw; ++w) {
      const int c = wcnt[w * p.E + e];
      wcnt[w * p.E + e] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int64_t b = i0; b < i1; b += 32) {
    const int64_t i = b + lane;
    int id = i < i1 ? p.ids[i] : -1;
    if (!RNL_DCHECK(&g_err_moe, id >= -1 && id < p.E, 216)) id = -1;
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int pos = -1;
    if (id >= 0) pos = mine[id] + rank;
    __syncwarp();
    if (id >= 0 && rank == 0) mine[id] += __popc(same);
    __syncwarp();
    if (i < i1) {
      p.slots[i] = pos;
      if (pos >= 0 && RNL_DCHECK(&g_err_moe, pos < p.T * p.k, 217)) p.rows[pos] = static_cast<int32_t>(i / p.k);
    }
  }
}

__device__ __forceinline__ void token_range(const RouteArgs& p, int64_t& t0, int64_t& t1) {
  t0 = static_cast<int64_t>(blockIdx.x) * p.per;
  t1 = t0 + p.per < p.T ? t0 + p.per : p.T;
}

template <int VPL>
__global__ void __launch_bounds__(kThreadsR) route_choose_kernel(RouteArgs p) {
  extern __shared__ int sm[];
  grid_dependency_wait();
  grid_launch_dependents();
  int64_t t0, t1;
  token_range(p, t0, t1);
  choose_all<VPL>(p, t0, t1, sm);
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < p.E; e += kThreadsR) p.hist[static_cast<int64_t>(blockIdx.x) * p.E + e] = sm[e];
    return;
  }
  int* before = sm + p.E;
  for (int e = threadIdx.x; e < p.E; e += kThreadsR) before[e] = 0;
  __syncthreads();
  place_all(p, t0, t1, before, sm, sm + 2 * p.E);
}

__global__ void __launch_bounds__(kThreadsR) route_place_kernel(RouteArgs p) {
  extern __shared__ int sm[];
  int* total = sm;
  int* before = sm + p.E;
  for (int e = threadIdx.x; e < 2 * p.E; e += kThreadsR) sm[e] = 0;
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  // lane groups of the block share the CTAs' counts out; additions of integers
  const int B = gridDim.x;
  const int lanes = p.E < kThreadsR ? p.E : kThreadsR;  // threads over the experts
  const int parts = kThreadsR / lanes;
  const int part = threadIdx.x / lanes;
  if (part < parts)
    for (int e = threadIdx.x % lanes; e < p.E; e += lanes) {
      int all = 0, bef = 0;
#pragma unroll 8
      for (int b = part; b < B; b += parts) {
        const int c = p.hist[static_cast<int64_t>(b) * p.E + e];
        all += c;
        if (b < static_cast<int>(blockIdx.x)) bef += c;
      }
      if (parts > 1) {
        atomicAdd(total + e, all);
        atomicAdd(before + e, bef);
      } else {
        total[e] = all;
        before[e] = bef;
      }
    }
  __syncthreads();
  int64_t t0, t1;
  token_range(p, t0, t1);
  place_all(p, t0, t1, before, total, sm + 2 * p.E);
}

int route_blocks(int64_t T, int* per) {
  int64_t n = (T + kMaxBlocks - 1) / kMaxBlocks;
  if (n < kMinTokens) n = kMinTokens;
  *per = static_cast<int>(n);
  return static_cast<int>((T + n - 1) / n);
}

// ------------------------------------------------------------------ combine
// One thread a 16-byte vector of a token's output: its k rows' vectors are
// loaded four at a time and added in FP32 in the order of the places.  Bound by
// HBM: 8192 tokens x 8 rows of 4096 in 104 us, 6.4 TB/s.
__global__ void __launch_bounds__(256)
    combine_kernel(const uint4* y, int64_t M, int nvec, const int32_t* slots, const float* weights, int64_t total,
                   int k, const uint4* residual, uint4* out) {
  // (plain loads: read-only ones need not stay behind the wait)
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= total) return;
  const int64_t t = i / nvec;
  const int v = static_cast<int>(i - t * nvec);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  uint4 res = make_uint4(0u, 0u, 0u, 0u);
  if (residual != nullptr) res = residual[i];
  for (int j0 = 0; j0 < k; j0 += 4) {
    uint4 u[4];
    float w[4];
    bool on[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      on[j] = false;
      if (j0 + j < k) {
        const int s = slots[t * k + j0 + j];
        w[j] = weights[t * k + j0 + j];
        on[j] = s >= 0 && s < M;
        if (!on[j] && s != -1) atomicCAS(&g_err_moe, 0u, kErrArg | (214u << 8));
        if (on[j]) u[j] = y[static_cast<int64_t>(s) * nvec + v];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (on[j]) {
        const uint32_t q[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          acc[2 * h] = fmaf(w[j], __uint_as_float(q[h] << 16), acc[2 * h]);
          acc[2 * h + 1] = fmaf(w[j], __uint_as_float(q[h] & 0xFFFF0000u), acc[2 * h + 1]);
        }
      }
  }
  const uint32_t q[4] = {res.x, res.y, res.z, res.w};
  uint32_t o[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    if (residual != nullptr) {
      acc[2 * h] += __uint_as_float(q[h] << 16);
      acc[2 * h + 1] += __uint_as_float(q[h] & 0xFFFF0000u);
    }
    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * h], acc[2 * h + 1]);
    o[h] = *reinterpret_cast<const uint32_t*>(&b);
  }
  out[i] = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace

size_t moe_route_workspace_bytes(int64_t T, int64_t E) {
  int per;
  const int blocks = T > 0 ? route_blocks(T, &per) : 0;
  return blocks > 1 ? static_cast<size_t>(blocks) * E * 4 : 0;
}

rnl_status launch_moe_route(const float* logits, int64_t T, int64_t E, int64_t k, int renorm, int32_t* ids,
                            float* weights, int32_t* offsets, int32_t* rows, int32_t* slots, void* ws,
                            cudaStream_t s) {
  RouteArgs p;
  p.logits = logits;
  p.T = T;
  p.E = static_cast<int>(E);
  p.k = static_cast<int>(k);
  p.renorm = renorm;
  p.ids = ids;
  p.weights = weights;
  p.offsets = offsets;
  p.rows = rows;
  p.slots = slots;
  p.hist = static_cast<int32_t*>(ws);
  const int blocks = route_blocks(T > 0 ? T : 1, &p.per);
  g_launched.store(true, std::memory_order_relaxed);
  const size_t smem = static_cast<size_t>(E) * 4 * (2 + rank_warps(static_cast<int>(E)));  // at most 40 KB
  trace_before(s);
  cudaError_t e;
  if (E <= 32)
    e = launch_dependent(route_choose_kernel<1>, blocks, kThreadsR, smem, s, p);
  else if (E <= 64)
    e = launch_dependent(route_choose_kernel<2>, blocks, kThreadsR, smem, s, p);
  else if (E <= 128)
    e = launch_dependent(route_choose_kernel<4>, blocks, kThreadsR, smem, s, p);
  else if (E <= 256)
    e = launch_dependent(route_choose_kernel<8>, blocks, kThreadsR, smem, s, p);
  else if (E <= 512)
    e = launch_dependent(route_choose_kernel<16>, blocks, kThreadsR, smem, s, p);
  else
    e = launch_dependent(route_choose_kernel<32>, blocks, kThreadsR, smem, s, p);
  trace_after(s, "moe_route");
  if (e == cudaSuccess && blocks > 1) {
    trace_before(s);
    e = launch_dependent(route_place_kernel, blocks, kThreadsR, smem, s, p);
    trace_after(s, "moe_route_place");
  }
  return e == cudaSuccess ? RNL_OK : RNL_ERR_LAUNCH;
}

rnl_status launch_moe_combine(const void* y, int64_t M, int64_t N, const int32_t* slots, const float* weights,
                              int64_t T, int64_t k, const void* residual, void* out, cudaStream_t s) {
  const int64_t total = T * (N / 8);
  if (total == 0) return RNL_OK;
  g_launched.store(true, std::memory_order_relaxed);
  trace_before(s);
  const cudaError_t e = launch_dependent(combine_kernel, static_cast<unsigned>((total + 255) / 256), 256, 0, s,
                                         static_cast<const uint4*>(y), M, static_cast<int>(N / 8), slots, weights,
                                         total, static_cast<int>(k), static_cast<const uint4*>(residual),
                                         static_cast<uint4*>(out));
  trace_after(s, "moe_combine");
  return e == cudaSuccess ? RNL_OK : RNL_ERR_LAUNCH;
}

rnl_status read_clear_error_moe(unsigned int* word) {
  if (!g_launched.load(std::memory_order_relaxed)) return RNL_OK;
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_moe, sizeof v) != cudaSuccess) return RNL_ERR_LAUNCH;
  if (v != 0 && cudaMemcpyToSymbol(g_err_moe, &zero, sizeof zero) != cudaSuccess) return RNL_ERR_LAUNCH;
  *word = v;
  return RNL_OK;
}

}  // namespace rnl
