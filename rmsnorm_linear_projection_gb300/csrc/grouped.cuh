// grouped.cuh -- what the grouped products (grouped.cu, groupedmx.cu) share:
// the tiles of ragged groups, the work list over them and the epilogue stores.
//
//   out[i] = x[rows[i]] W[e]^T   for the rows i of expert e, offsets[e] <= i < offsets[e + 1]
//
// Weight rows stand on the tensor core's M side (128 TMEM lanes a CTA), the
// group's rows on its N side, because N may be any multiple of 16 (of 32 on a CTA
// pair): a group of 5 rows costs a 16-wide product instead of a 128-row one, and a large group is
// cut into equal tiles of at most kTile rows.  How many rows an expert has is
// known on the device only: every CTA reads the offsets and builds the table
// of the groups' first tiles itself.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "gemm_common.cuh"
#include "ptx.cuh"

namespace rnl {
namespace grouped {

constexpr int kMaxExperts = 1024;
constexpr int kEpiWarps = 8;
// token tiles of a group walked before the next weight rows: their operand
// (16 x 256 rows of 4096 bf16: 34 MB) stays in L2 while the weight passes
constexpr int kSuper = 16;

// The groups: off[e] rows before expert e, pre[e] tiles before it (both E + 1 values).
struct Groups {
  const int* off;
  const int* pre;
  int E;
  int num_f;  // feature tiles
};

// One output tile: rows [row0, row0 + valid) of the grouped order against the
// weight rows of feature tile f of expert e; n: valid rounded up to the step of
// the product's N side (16 on one CTA, 32 on a pair).
struct Tile {
  int e, f, row0, valid, n;
};

__device__ __forceinline__ int token_tiles(int cnt, int tile) { return (cnt + tile - 1) / tile; }

// Fills off and pre (shared memory, E + 1 values each) from the offsets; called
// by every thread of the block, which must synchronise afterwards.  Offsets
// that decrease or leave [0, M] are reported, and no tile is made.
__device__ __forceinline__ void build_groups(const int32_t* __restrict__ offsets, int E, int M, int num_f,
                                             int tile, int* off, int* pre, unsigned int* err, uint32_t site) {
  for (int i = threadIdx.x; i <= E; i += blockDim.x) off[i] = offsets[i];
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int64_t base = 0;
    bool bad = off[0] < 0 || off[E] > M;
    for (int i0 = 0; i0 < E; i0 += 32) {
      const int i = i0 + lane;
      const int64_t cnt = i < E ? static_cast<int64_t>(off[i + 1]) - off[i] : 0;
      bad |= cnt < 0;
      int64_t t = cnt > 0 ? (cnt + tile - 1) / tile * num_f : 0;
      const int64_t own = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += v;
      }
      if (i < E) pre[i] = static_cast<int>(base + t - own);
      base += __shfl_sync(0xffffffffu, t, 31);
    }
    bad = __any_sync(0xffffffffu, bad) || base > 0x7fffffff;
    if (bad) {
      for (int i = lane; i <= E; i += 32) pre[i] = 0;
      if (lane == 0) atomicCAS(err, 0u, kErrArg | (site << 8));
    } else if (lane == 0) {
      pre[E] = static_cast<int>(base);
    }
  }
}

template <int kTile, int kStep>
__device__ __forceinline__ Tile tile_at(const Groups& g, int t) {
  static_assert(kTile % kStep == 0, "tiles of whole steps");
  int lo = 0, hi = g.E;  // the last e with pre[e] <= t (empty groups have no tile)
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (g.pre[m] <= t)
      lo = m;
    else
      hi = m;
  }
  Tile r;
  r.e = lo;
  const int loc = t - g.pre[lo];
  const int cnt = g.off[lo + 1] - g.off[lo];
  const int nt = token_tiles(cnt, kTile);
  const int ns = ((cnt + nt - 1) / nt + kStep - 1) / kStep * kStep;  // (nt - 1) ns < cnt, as ns <= kTile
  const int super = loc / (kSuper * g.num_f);
  const int gm = min(nt - super * kSuper, kSuper);
  const int in = loc - super * kSuper * g.num_f;
  const int tt = super * kSuper + in % gm;
  r.f = in / gm;
  r.row0 = g.off[lo] + tt * ns;
  r.valid = min(ns, cnt - tt * ns);
  r.n = (r.valid + kStep - 1) / kStep * kStep;
  return r;
}

// The work list of `units` workers (CTAs or CTA pairs) over T tiles of num_kb
// k-blocks: the first tiles go round the workers whole; the k-blocks of the
// last units .. 2 units - 1 tiles (of all, when there are fewer) are cut into
// equal ranges, so that no worker waits through a partial wave.  A range that
// does not hold its last tile's end leaves that tile's partial sums to the
// worker that does, which has a HIGHER index; a worker makes its partial sums
// first and finishes a tile of others last, so waiting goes to lower indices
// only and never round in a circle, whatever else holds the GPU's SMs.
struct Sched {
  int units;
  int dp;      // tiles that go whole
  int sk;      // tiles whose k-blocks are cut into ranges
  int sk_units;  // workers that get a range
  int num_kb;
  __device__ __forceinline__ Sched(int tiles, int workers, int kbs) {
    units = workers;
    num_kb = kbs;
    dp = tiles >= 2 * workers ? (tiles / workers - 1) * workers : 0;
    sk = tiles - dp;
    // a range of fewer than 4 k-blocks is not worth its joining
    const int64_t most = static_cast<int64_t>(sk) * kbs / 4;
    sk_units = most < 1 ? 1 : (most < workers ? static_cast<int>(most) : workers);
  }
  __device__ __forceinline__ int64_t start(int u) const {
    return static_cast<int64_t>(u) * sk * num_kb / sk_units;
  }
};

enum : int { kWhole = 0, kFinish = 1, kPartial = 2 };

struct Item {
  int tile, kb0, kb1, kind;
  int first;  // kFinish: the lowest worker that holds a part of the tile
};

// The items of one worker, in order.
struct Walk {
  int n;
  int unit, n_sk, n_dp, tile_lo;
  int64_t u0, u1;
  bool fin_last;
  __device__ __forceinline__ Walk(const Sched& s, int u) {
    unit = u;
    n_dp = u < s.dp ? (s.dp - u + s.units - 1) / s.units : 0;
    n_sk = 0;
    u0 = u1 = 0;
    tile_lo = 0;
    fin_last = false;
    if (u < s.sk_units && s.sk > 0) {
      u0 = s.start(u);
      u1 = s.start(u + 1);
      if (u1 > u0) {
        tile_lo = static_cast<int>(u0 / s.num_kb);
        n_sk = static_cast<int>((u1 - 1) / s.num_kb) - tile_lo + 1;
        fin_last = u0 > static_cast<int64_t>(tile_lo) * s.num_kb &&
                   u1 >= static_cast<int64_t>(tile_lo + 1) * s.num_kb;
      }
    }
    n = n_sk + n_dp;
  }
  __device__ __forceinline__ Item at(const Sched& s, int it) const {
    Item w;
    w.first = unit;
    int j;  // index among the range's tiles, highest first
    const int early = fin_last ? n_sk - 1 : n_sk;
    if (it < early) {
      j = it;
    } else if (it < early + n_dp) {
      w.tile = unit + (it - early) * s.units;
      w.kb0 = 0;
      w.kb1 = s.num_kb;
      w.kind = kWhole;
      return w;
    } else {
      j = n_sk - 1;
    }
    const int t = tile_lo + (n_sk - 1 - j);
    const int64_t ts = static_cast<int64_t>(t) * s.num_kb;
    w.tile = s.dp + t;
    w.kb0 = static_cast<int>(u0 > ts ? u0 - ts : 0);
    w.kb1 = static_cast<int>(u1 < ts + s.num_kb ? u1 - ts : s.num_kb);
    w.kind = w.kb1 < s.num_kb ? kPartial : (w.kb0 > 0 ? kFinish : kWhole);
    if (w.kind == kFinish) {
      int q = unit - 1;
      while (s.start(q) > ts) --q;
      w.first = q;
    }
    return w;
  }
};

// x * sigmoid(x) * u; the exponential is good to a few units of FP32's last
// place times |g|, far inside the bf16 rounding that follows.
__device__ __forceinline__ float swiglu_of(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// Writes 32 columns (rows row0 + col .. of the output) of a warp's 32 TMEM
// lanes (32 weight rows; feat: the lane's feature) as bf16.  Neighbouring lanes
// exchange a value each, so that every store takes two features of one row.
__device__ __forceinline__ void store_cols(__nv_bfloat16* __restrict__ out, int N, int64_t row0, int valid, int col,
                                           int feat, int lane, const uint32_t (&r)[32]) {
  if ((N & 1) == 0) {
    const bool odd = lane & 1;
    // the column pair's first row for even lanes, its second one for odd ones
    __nv_bfloat16* dst = out + (row0 + col + (odd ? 1 : 0)) * N + (feat & ~1);
    const bool f_ok = (feat | 1) < N;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? r[j] : r[j + 1], 1);
      const uint32_t word = odd ? gemm::bf16x2_bits(__uint_as_float(got), __uint_as_float(r[j + 1]))
                                : gemm::bf16x2_bits(__uint_as_float(r[j]), __uint_as_float(got));
      if (f_ok && col + j + (odd ? 1 : 0) < valid)
        *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(j) * N) = word;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (feat < N && col + j < valid)
        out[(row0 + col + j) * N + feat] = __float2bfloat16_rn(__uint_as_float(r[j]));
  }
}

// The same for gate and up sums: lanes 0-15 of the warp hold the gates of 16
// features, lanes 16-31 their ups.  feat: of lane & 15; F: features of a row, a
// multiple of 16.
__device__ __forceinline__ void store_cols_swiglu(__nv_bfloat16* __restrict__ out, int F, int64_t row0, int valid,
                                                  int col, int feat, int lane, const uint32_t (&r)[32]) {
  const bool hi = lane & 16, odd = lane & 1;
  const int sub = (hi ? 1 : 0) + (odd ? 2 : 0);  // the row of four that this lane stores
  __nv_bfloat16* dst = out + (row0 + col + sub) * F + (feat & ~1);
  const bool f_ok = feat < F;
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    float v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // lanes 0-15 take column j + 2h, lanes 16-31 the next one
      const uint32_t a = r[j + 2 * h], b = r[j + 2 * h + 1];
      const float got = __uint_as_float(__shfl_xor_sync(0xffffffffu, hi ? a : b, 16));
      v[h] = hi ? swiglu_of(got, __uint_as_float(b)) : swiglu_of(__uint_as_float(a), got);
    }
    const float got = __shfl_xor_sync(0xffffffffu, odd ? v[0] : v[1], 1);
    const uint32_t word = odd ? gemm::bf16x2_bits(got, v[1]) : gemm::bf16x2_bits(v[0], got);
    if (f_ok && col + j + sub < valid) *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(j) * F) = word;
  }
}

}  // namespace grouped
}  // namespace rnl
