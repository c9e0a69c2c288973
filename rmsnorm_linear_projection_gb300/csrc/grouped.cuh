// grouped.cuh -- pieces of the grouped products (grouped.cu): the tiles of ragged groups,
// the work list over them and the epilogue stores.
//
//   out[i] = x[rows[i]] W[e]^T   for the rows i of expert e, offsets[e] <= i < offsets[e + 1]
//
// Weight rows stand on the tensor core's M side (256 of a CTA pair, 128 TMEM lanes
// each), the group's rows on its N side, because N may be any multiple of 32: a group
// of 5 rows costs a 32-wide product instead of a 256-row one, and a large group is
// cut into near-equal tiles of at most kTile rows.  How many rows an expert has is
// known on the device only: every CTA reads the offsets and builds the table
// of the groups' first tiles itself.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "gemm_common.cuh"
#include "joinflag.h"
#include "ptx_more.cuh"

namespace rnl {
namespace grouped {

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
// the product's N side (32).
struct Tile {
  int e, f, row0, valid, n;
};

__device__ __forceinline__ int token_tiles(int cnt, int tile) { return (cnt + tile - 1) / tile; }

// Fills off and pre (shared memory, E + 1 values each) from the offsets; called
// by every thread of the block, which must synchronise afterwards (warp 0, which
// writes pre, need not).  (offsets without __restrict__: read-only loads need not stay
// behind the wait for the kernel before.)  Offsets
// that decrease or leave [0, M] are reported, and no tile is made.
__device__ __forceinline__ void build_groups(const int32_t* offsets, int E, int M, int num_f,
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
    __syncwarp();
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
  // the group's steps are dealt out to its tiles as evenly as whole steps allow:
  // 900 rows in steps of 32 are 256 + 3 x 224, not 3 x 256 + 132 (32 experts of them
  // 113.6 -> 111.3 us, of 520 rows 76.7 -> 74.0; MXFP8 65536 rows over 128 experts
  // 347 -> 340)
  const int nt = token_tiles(cnt, kTile);
  const int steps = (cnt + kStep - 1) / kStep;
  const int each = steps / nt, more = steps - each * nt;
  const int super = loc / (kSuper * g.num_f);
  const int gm = min(nt - super * kSuper, kSuper);
  const int in = loc - super * kSuper * g.num_f;
  const int tt = super * kSuper + in % gm;
  r.f = in / gm;
  const int first = (tt * each + min(tt, more)) * kStep;
  r.row0 = g.off[lo] + first;
  r.valid = min((each + (tt < more ? 1 : 0)) * kStep, cnt - first);
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
  int sk_units;  // workers that get a range: share k-blocks, the first `more` of them one more
  int share, more;
  int num_kb;
  __device__ __forceinline__ void set(int tiles, int workers, int kbs) {
    units = workers;
    num_kb = kbs;
    dp = tiles >= 2 * workers ? (tiles / workers - 1) * workers : 0;
    sk = tiles - dp;
    // a range of fewer than 4 k-blocks is not worth its joining
    const int total = sk * kbs;  // below 2^31: sk < 2 * 128, K at most RNL_GROUPED_MAX_K
    sk_units = max(1, min(total / 4, workers));
    share = total / sk_units;
    more = total - share * sk_units;
  }
  // first k-block (of the flattened sk tiles) of worker u's range
  __device__ __forceinline__ int start(int u) const { return u * share + min(u, more); }
};

enum : int { kWhole = 0, kFinish = 1, kPartial = 2 };

// What a worker does to one tile: k-blocks [kb0, kb1) of it.
struct Item {
  Tile t;
  int kb0, kb1, kind;
  int first;  // kFinish: the lowest worker that holds a part of the tile (else the worker itself)
};

// One side's visit of a join's flag (joinflag.h): leaves v there (the epoch: partial
// sums are handed over, what this thread has seen written stands before it; or
// join_gave_up), or 0 where the other side has been.
__device__ __forceinline__ void join_visit(uint64_t* f, uint64_t v, uint64_t epoch) {
  uint64_t found;
  asm volatile("atom.acq_rel.gpu.global.exch.b64 %0, [%1], %2;" : "=l"(found) : "l"(f), "l"(v) : "memory");
  if (join_is_second(found, epoch)) *reinterpret_cast<volatile uint64_t*>(f) = 0;
}

// The items of one worker, in order: what they are made from, and the first kTable of
// them (in shared memory, filled by one warp).
constexpr int kTable = 16;  // (with 32 the table costs a stage of the pipeline from 86 experts on, with 16 from 150)
struct Plan {
  Sched s;
  int n;
  int unit, n_sk, n_dp, tile_lo, u0, u1;
  int fin_last;
  int4 table[kTable][2];

  __device__ __forceinline__ void set(int tiles, int workers, int kbs, int u) {
    s.set(tiles, workers, kbs);
    unit = u;
    n_dp = u < s.dp ? (s.dp - u + s.units - 1) / s.units : 0;
    n_sk = 0;
    u0 = u1 = 0;
    tile_lo = 0;
    fin_last = 0;
    if (u < s.sk_units && s.sk > 0) {
      u0 = s.start(u);
      u1 = s.start(u + 1);
      if (u1 > u0) {
        tile_lo = u0 / s.num_kb;
        n_sk = (u1 - 1) / s.num_kb - tile_lo + 1;
        fin_last = u0 > tile_lo * s.num_kb && u1 >= (tile_lo + 1) * s.num_kb;
      }
    }
    n = n_sk + n_dp;
  }
};

template <int kTile, int kStep>
__device__ __forceinline__ Item make_item(const Plan& p, const Groups& g, int it) {
  const Sched& s = p.s;
  Item w;
  w.first = p.unit;
  int j;  // index among the range's tiles, highest first
  const int early = p.fin_last ? p.n_sk - 1 : p.n_sk;
  if (it < early) {
    j = it;
  } else if (it < early + p.n_dp) {
    w.t = tile_at<kTile, kStep>(g, p.unit + (it - early) * s.units);
    w.kb0 = 0;
    w.kb1 = s.num_kb;
    w.kind = kWhole;
    return w;
  } else {
    j = p.n_sk - 1;
  }
  const int t = p.tile_lo + (p.n_sk - 1 - j);
  const int ts = t * s.num_kb;
  w.t = tile_at<kTile, kStep>(g, s.dp + t);
  w.kb0 = max(p.u0 - ts, 0);
  w.kb1 = min(p.u1 - ts, s.num_kb);
  w.kind = w.kb1 < s.num_kb ? kPartial : (w.kb0 > 0 ? kFinish : kWhole);
  if (w.kind == kFinish) {
    int q = p.unit - 1;
    while (s.start(q) > ts) --q;
    w.first = q;
  }
  return w;
}

// The flags that a warp has not visited when it leaves its worker's items at item
// `it`: of the worker's own partial sums, which are its first item, and of the parts
// that its last item joins.  (Not inline: the registers are the items' own.)
template <int kTile, int kStep>
__device__ __noinline__ void give_up_joins(const Plan& p, const Groups& g, int it, int lane, uint64_t* flags, int step,
                                           uint64_t epoch) {
  if (it == 0 && lane == 0 && make_item<kTile, kStep>(p, g, 0).kind == kPartial)
    join_visit(flags + static_cast<int64_t>(p.unit) * step, join_gave_up(epoch), epoch);
  if (!p.fin_last) return;
  const Item last = make_item<kTile, kStep>(p, g, p.n - 1);
  for (int q = last.first + lane; q < p.unit; q += 32)
    join_visit(flags + static_cast<int64_t>(q) * step, join_gave_up(epoch), epoch);
}

// Fills the plan and its table: by one warp, after build_groups' (the same warp's)
// part.  Every warp for itself, it took 1.3 to 2.3 us of a launch.
template <int kTile, int kStep>
__device__ __forceinline__ void make_plan(Plan& p, const Groups& g, int workers, int kbs, int unit, int lane) {
  if (lane == 0) p.set(g.pre[g.E], workers, kbs, unit);
  __syncwarp();
  if (lane < p.n && lane < kTable) {
    const Item w = make_item<kTile, kStep>(p, g, lane);
    p.table[lane][0] = make_int4(w.t.e, w.t.f, w.t.row0, w.t.valid);
    p.table[lane][1] = make_int4(w.kb0, w.kb1, w.kind, w.first);
  }
}

// The items one after the other: the first ones from the plan's table; behind them
// a warp works out 32 at once, one a lane, and hands them round (one by one they
// cost each role about 0.8 us a tile).
template <int kTile, int kStep>
struct Walk {
  const Plan& p;
  const Groups& g;
  int n, lane;
  Item mine;
  __device__ __forceinline__ Walk(const Plan& plan, const Groups& gr, int ln) : p(plan), g(gr), n(plan.n), lane(ln) {}
  // Item `it`, the same on every lane; called by the whole warp, for it = 0, 1, ...
  __device__ __forceinline__ Item at(int it) {
    Item w;
    if (it < kTable) {
      const int4 a = p.table[it][0], b = p.table[it][1];
      w.t.e = a.x, w.t.f = a.y, w.t.row0 = a.z, w.t.valid = a.w;
      w.kb0 = b.x, w.kb1 = b.y, w.kind = b.z, w.first = b.w;
    } else {
      const int from = (it - kTable) & 31;
      if (from == 0 && it + lane < n) mine = make_item<kTile, kStep>(p, g, it + lane);
      w.t.e = __shfl_sync(0xffffffffu, mine.t.e, from);
      w.t.f = __shfl_sync(0xffffffffu, mine.t.f, from);
      w.t.row0 = __shfl_sync(0xffffffffu, mine.t.row0, from);
      w.t.valid = __shfl_sync(0xffffffffu, mine.t.valid, from);
      w.kb0 = __shfl_sync(0xffffffffu, mine.kb0, from);
      w.kb1 = __shfl_sync(0xffffffffu, mine.kb1, from);
      w.kind = __shfl_sync(0xffffffffu, mine.kind, from);
      w.first = __shfl_sync(0xffffffffu, mine.first, from);
    }
    w.t.n = (w.t.valid + kStep - 1) / kStep * kStep;
    return w;
  }
};

// v[i] = g * sigmoid(g) * u of 16 gates and ups, over FP32's whole range: u * g /
// (1 + exp(-g)) for gates of -80 and more.  Below, sigmoid(g) is exp(g) to FP32's last
// bit, and leaves FP32's range (from -87 on) before silu(g) u with a large u does (from
// -185): with q = exp(g / 4) two of its factors go to g and two to u (q^2 still holds
// 15 bits at -185), so that nothing is lost in front of the product.  A warp votes once
// whether any of its 16 columns holds such a gate, since they are rare: a form for the
// whole range throughout cost 1.5 % of a prompt (8192 tokens over 32 experts 263.7
// against 259.2 us), and a branch or a correctly rounded division for each value
// keeps a thread's columns from overlapping.  Which form a value takes goes by its own
// gate alone.  The exponentials are good to 8 + |g| units of FP32's last place, the
// reciprocal to one, both far inside the bf16 rounding that follows.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void swiglu_cols(const float (&g)[16], const float (&u)[16], float (&v)[16]) {
  constexpr float kLog2e = 1.44269504f;
  float least = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    v[j] = g[j] * rcp_approx(1.0f + exp2_approx(g[j] * -kLog2e)) * u[j];
    least = fminf(least, g[j]);
  }
  if (__any_sync(0xffffffffu, least < -80.f)) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float q = exp2_approx(g[j] * (0.25f * kLog2e)), q2 = q * q;
      if (g[j] < -80.f) v[j] = (g[j] * q2) * (u[j] * q2);
    }
  }
}

// Stores words w[i] at dst + i * step, i < n, of the lanes that are on; whole: of
// all lanes, n = COUNT (no predicates, so that the stores go out back to back).
template <int COUNT>
__device__ __forceinline__ void store_words(__nv_bfloat16* dst, int64_t step, const uint32_t (&w)[COUNT], bool on,
                                            int n) {
  if (__all_sync(0xffffffffu, on && n >= COUNT)) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) *reinterpret_cast<uint32_t*>(dst + i * step) = w[i];
  } else if (on) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
      if (i < n) *reinterpret_cast<uint32_t*>(dst + i * step) = w[i];
  }
}

// Writes 32 columns (rows row0 + col .. of the output) of a warp's 32 TMEM
// lanes (32 weight rows; feat: the lane's feature) as bf16.  Neighbouring lanes
// exchange a value each, so that every store takes two features of one row; all
// exchanges come before the stores (one by one in turn they took 130 cycles
// each).
__device__ __forceinline__ void store_cols(__nv_bfloat16* __restrict__ out, int N, int64_t row0, int valid, int col,
                                           int feat, int lane, const uint32_t (&r)[32]) {
  if ((N & 1) == 0) {
    const int odd = lane & 1;  // takes the column pair's second row
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? r[2 * j] : r[2 * j + 1], 1);
      w[j] = odd ? gemm::bf16x2_bits(__uint_as_float(got), __uint_as_float(r[2 * j + 1]))
                 : gemm::bf16x2_bits(__uint_as_float(r[2 * j]), __uint_as_float(got));
    }
    store_words<16>(out + (row0 + col + odd) * N + (feat & ~1), 2 * static_cast<int64_t>(N), w, (feat | 1) < N,
                    (valid - col - odd + 1) >> 1);
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
  float g[16], u[16], v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {  // lanes 0-15 take column 2j, lanes 16-31 the next one
    const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? r[2 * j] : r[2 * j + 1], 16);
    g[j] = __uint_as_float(hi ? got : r[2 * j]);
    u[j] = __uint_as_float(hi ? r[2 * j + 1] : got);
  }
  swiglu_cols(g, u, v);
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float got = __shfl_xor_sync(0xffffffffu, odd ? v[2 * j] : v[2 * j + 1], 1);
    w[j] = odd ? gemm::bf16x2_bits(got, v[2 * j + 1]) : gemm::bf16x2_bits(v[2 * j], got);
  }
  store_words<8>(out + (row0 + col + sub) * F + (feat & ~1), 4 * static_cast<int64_t>(F), w, feat < F,
                 (valid - col - sub + 3) >> 2);
}

}  // namespace grouped
}  // namespace rnl
