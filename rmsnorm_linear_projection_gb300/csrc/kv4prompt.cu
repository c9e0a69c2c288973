// kv4prompt.cu -- attention over the 4-bit paged KV cache for sequences with
// many rows in the call (prompts, chunks of prompts, cross attention), on the
// fifth-generation tensor cores.  The formulas, operands and scales are those
// of kv4attn.cu: E2M1 values times 2^(X - R + 13) in binary16, where R is the
// tile's largest scale (keys) or the largest so far (values), exact down to
// 2^-36 of it (kv4.cuh, kSpread); queries scaled by a power of two per row.
//
// A CTA works on 256 rows (token x query head of one key head), two tiles of
// 128, against tiles of 128 tokens in steps of 64:
//   warps 0-3, 4-7   softmax of the two row tiles, a thread a row: a step's
//                    scores from TMEM, weights back to TMEM as binary16 (the A
//                    operand of the second product), the sums rescaled there
//                    when the maximum grew by about 2^9
//   warps 8-11,      keys and values, a thread a token: codes and scales from a
//     12-15          ring in shared memory, converted and scaled into the
//                    operands there (128-byte swizzle; keys K-major, values
//                    MN-major, the same bytes in the same order)
//   warps 16, 17     (TMEM allocation and) a row tile's tcgen05.mma each:
//                    S = Q K^T (both from shared memory), O += P V (P from TMEM)
//   warp 18          bulk copies of the next tiles' codes and scales into the ring
//   warp 19          walks the CTA's range and tells the others its runs
// TMEM, per row tile: two buffers of 64 columns of scores (a step's weights
// take the first 32 of its buffer), and D columns of sums.  The scores of a
// step are computed while the softmax works on the step before, so that it
// does not wait for the tensor core and its barriers.
//
// The weights are 2^(x - m + 7) with m at most 9 behind the true maximum:
// binary16 holds them with 11 bits down to 2^-21 of the largest, or less.
//
// Rows later in a causal prompt read more tokens.  An item is a pair of row
// groups, one from either end, so that all items of a sequence have about the
// same number of tiles; the tiles of all items are dealt to the CTAs in equal
// contiguous ranges.  A group that is cut leaves FP32 partial sums, joined by
// a dependent kernel.
//
// Measured (two prompts of 1000 to 2048 rows over 6000 to 10240 tokens, G = 4,
// D = 128): 375 to 379 us, 995 to 1006 TFLOP/s, tensor pipe 46 % active; a tile takes
// 1.9 us where the products alone would take 1.1.  What it waits for is the softmax (a
// thread a row: exponentials, conversions, TMEM reads) beside 8 to 10 us a run, in
// which a run's queries and first scores wait for the output of the run before.  With
// a window of 4096 tokens (2048 and 1500 rows over 10240 and 8000): 300 us against 127.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv4.cuh"

namespace rnl {
namespace {

using namespace kv4;

__device__ unsigned int g_err_kv4prompt;
std::atomic<bool> g_launched{false};

constexpr int kT = 128;            // tokens a tile of operands
constexpr int kU = 64;             // tokens a step of products and softmax
constexpr int kGroup = 256;        // rows a CTA holds
constexpr int kSoftWarps = 8;
constexpr int kFillWarps = 4;      // for the keys, and as many for the values
constexpr int kValueWarp = kSoftWarps + kFillWarps;
constexpr int kMmaWarp = kValueWarp + kFillWarps;
constexpr int kLoadWarp = kMmaWarp + 2;
constexpr int kWalkWarp = kLoadWarp + 1;
constexpr int kMaxRing = 6;
constexpr int kPWarps = 20;        // five warpgroups
constexpr int kPThreads = kPWarps * 32;
// registers a thread after the roles part, within what the block is launched with
constexpr int kLaunchRegs = 96, kSoftRegs = 136, kFillRegs = 64, kMmaRegs = 72;
static_assert(8 * kSoftRegs + 8 * kFillRegs + 4 * kMmaRegs <= kPWarps * kLaunchRegs, "register file");
// What a group costs beside its tiles (queries, output), in tiles.  12 prompts of
// 300 to 1500 rows: 330 us, with 3 tiles 338, 5 345, 7 359; 6 of 100 to 800 rows
// over 1000 to 9000 tokens, D = 64: 125 us, with 3 tiles 136, 5 121.
constexpr int kGroupCost = 4;
constexpr int kMaxPromptCtas = 160;
constexpr float kTop = 7.f;        // weights are scaled by 2^7: room for 2^9 above the maximum in use

template <int D>
struct PCfg {
  static constexpr uint32_t kTileBytes = 128u * D * 2;    // Q_i, K or V in shared memory
  static constexpr uint32_t kHalf = 128u * 128;           // bytes between blocks of 64 dims
  // The ring's places hold a tile's keys (codes, scales, and the values' scales)
  // or its values (codes, scales), by turns; as many as there is room for.
  static constexpr uint32_t kRawCodes = 128u * D / 2, kRawScales = 128u * D / 32;
  static constexpr uint32_t kRaw = kRawCodes + 2 * kRawScales;
  static constexpr int kRing = D == 128 ? 3 : kMaxRing;
  static constexpr size_t kSmem = 1024 + 6 * static_cast<size_t>(kTileBytes) + kRing * kRaw;
  static constexpr int kSlot = kGroup * (D + 2);          // floats of a partial: sums, maxima, weights
};

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A group's tokens in tiles.
struct Span {
  Seq s;
  int groups;
};
__device__ __forceinline__ bool load_span(const Args& a, const AttnParams& p, int b, Span& w) {
  if (!load_seq(a, b, w.s, &g_err_kv4prompt, 48) || w.s.rows * p.G <= p.few) return false;
  w.groups = (w.s.rows * p.G + kGroup - 1) / kGroup;
  return true;
}
__device__ __forceinline__ void group_tokens(const AttnParams& p, const Seq& s, int g, int& lo, int& hi) {
  lo = 0;
  hi = s.len;
  if (p.causal) {
    const int last = min((g + 1) * kGroup, s.rows * p.G) - 1;
    hi = max(0, s.len - s.rows + last / p.G + 1);
    if (p.window > 0) lo = max(0, s.len - s.rows + g * kGroup / p.G + 1 - p.window);
  }
}
// The tokens that every row of the group reads.
__device__ __forceinline__ void common_tokens(const AttnParams& p, const Seq& s, int g, int& lo, int& hi) {
  lo = 0;
  hi = s.len;
  if (p.causal) {
    const int last = min((g + 1) * kGroup, s.rows * p.G) - 1;
    hi = max(0, s.len - s.rows + g * kGroup / p.G + 1);
    if (p.window > 0) lo = max(0, s.len - s.rows + last / p.G + 1 - p.window);
  }
}
__device__ __forceinline__ int tiles_between(int lo, int hi) {
  return hi > lo ? (hi + kT - 1) / kT - lo / kT : 1;  // at least one: rows without a token still get zeros
}
__device__ __forceinline__ int group_tiles(const AttnParams& p, const Seq& s, int g) {
  int lo, hi;
  group_tokens(p, s, g, lo, hi);
  return tiles_between(lo, hi);
}
// Units of a pair of groups: at least both groups' tiles and costs.  Causal
// rows: the first group and the last, were it full; with a window also at most
// twice the tiles that a window and a group's tokens can touch.
__device__ __forceinline__ int pair_units(const AttnParams& p, const Span& w) {
  int t;
  if (p.causal) {
    const int hi = max(0, w.s.len - w.s.rows + (w.groups * kGroup - 1) / p.G + 1);
    const int last = min((w.groups > 1 ? 1 : w.groups) * kGroup, w.s.rows * p.G) - 1;
    const int first = max(0, w.s.len - w.s.rows + last / p.G + 1);
    t = tiles_between(0, first) + tiles_between(0, hi) + 3;
    if (p.window > 0) t = min(t, 2 * ((p.window + (kGroup - 1) / p.G + 1 + 2 * kT - 2) / kT) + 1);
  } else {
    t = 2 * tiles_between(0, w.s.len);
  }
  return t + 2 * kGroupCost;
}

// Units of a head's items: the pairs, and the middle group alone where the
// number of groups is odd.
__device__ __forceinline__ int64_t head_units(const AttnParams& p, const Span& w) {
  return static_cast<int64_t>(pair_units(p, w)) * (w.groups / 2) +
         ((w.groups & 1) ? kGroupCost + group_tiles(p, w.s, w.groups / 2) : 0);
}

// Walks a CTA's range: next() gives its next run of one group's tiles.
struct Walk {
  int b, head, pair, off;  // place: units into the pair's item
  int64_t at, left;        // of the range's units: where, and how many are left
  Span w;
  // the run
  int group, lo, hi;       // tokens of the group
  int tile, n, all;        // first tile in the group, tiles, tiles of the group
  int64_t unit;            // where the run's first tile stands
  int seq, kvh;
};
__device__ __forceinline__ bool next_run(const Args& a, const AttnParams& p, Walk& c) {
  while (c.left > 0) {
    const int g0 = c.w.groups - 1 - c.pair, g1 = c.pair;
    const int n0 = group_tiles(p, c.w.s, g0), n1 = g1 < g0 ? group_tiles(p, c.w.s, g1) : 0;
    const int z0 = kGroupCost + n0, z1 = g1 < g0 ? kGroupCost + n1 : 0;
    if (c.off < z0 + z1) {
      const bool second = c.off >= z0;
      int o = second ? c.off - z0 : c.off;
      if (o < kGroupCost) {
        const int d = kGroupCost - o;
        c.left -= d;
        c.at += d;
        c.off += d;
        o = kGroupCost;
        if (c.left <= 0) return false;
      }
      c.group = second ? g1 : g0;
      c.all = second ? n1 : n0;
      c.tile = o - kGroupCost;
      c.n = static_cast<int>(min(static_cast<int64_t>(c.all - c.tile), c.left));
      if (c.n <= 0) return false;
      group_tokens(p, c.w.s, c.group, c.lo, c.hi);
      c.unit = c.at;
      c.seq = c.b;
      c.kvh = c.head;
      c.left -= c.n;
      c.at += c.n;
      c.off += c.n;
      return true;
    }
    const int rest = g1 < g0 ? max(pair_units(p, c.w) - c.off, 0) : 0;
    c.left -= rest;
    c.at += rest;
    c.off = 0;
    if (++c.pair == (c.w.groups + 1) / 2) {
      c.pair = 0;
      if (++c.head == a.Hkv) {
        c.head = 0;
        if (c.left <= 0) return false;
        do {
          if (++c.b >= a.n_seqs) {
            c.left = 0;
            return false;
          }
        } while (!load_span(a, p, c.b, c.w));
      }
    }
  }
  return false;
}

// The walk from unit `off` of sequence b's items on.
__device__ __forceinline__ Walk walk_from(const AttnParams& p, int b, const Span& w, int64_t off, int64_t at,
                                          int64_t left) {
  Walk c;
  c.b = b;
  c.w = w;
  const int64_t per_head = head_units(p, w);
  const int len = pair_units(p, w);
  // (64-bit divisions are slow, and everyone waits for the first run)
  c.head = off >> 32 || per_head >> 32
               ? static_cast<int>(off / per_head)
               : static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(per_head));
  const int64_t in_head = off - c.head * per_head;
  const int64_t pair = in_head >> 32 ? in_head / len : static_cast<uint32_t>(in_head) / static_cast<uint32_t>(len);
  c.pair = static_cast<int>(min(pair, static_cast<int64_t>(w.groups / 2)));
  c.off = static_cast<int>(in_head - static_cast<int64_t>(c.pair) * len);
  c.at = at;
  c.left = left;
  return c;
}

// A run as the roles read it.
struct Run {
  int row0, rows, len;         // the sequence
  int groups, group, seq, kvh;
  int lo, tile, n, all;        // tokens from lo on, in tiles: first, number, number of the whole group
  int hi, stop;
  int common_lo, common_hi;    // the tokens that every row of the group reads
  int64_t unit;
};
constexpr int kRuns = 4;

struct __align__(16) PCtrl {
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_done[2][2];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t raw_full[kMaxRing], raw_empty[kMaxRing];
  uint64_t run_full[kRuns], run_empty[kRuns];
  uint64_t drained[2];          // a row tile's products, after a wait has given up
  Run run[kRuns];
  // first token, the group's tokens, 1: a run's first tile, 2: no more tiles, 4: with
  // tokens that only some of the rows read; the run's number (up to 31) from bit 8 on
  int4 raw_info[kMaxRing];
  uint32_t alone;               // runs whose rows have to be taken by themselves (one_row)
  float k_info[4];   // score factor of tile x at x % 4
  int v_info[4];     // the values' reference scale byte
  int top[2][2][kFillWarps], stop[2], done[2][2];
  long long sum[kPWarps];
  long long off;
  uint32_t tmem;
  Span w;
  int b, abort;
};

// Low word of a shared-memory descriptor: start address and leading offset
// (between blocks of 64 elements of an MN-major operand; 16 bytes, unused, for
// a K-major one).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lead >> 4) << 16);
}
// kind::f16, binary16 A and B, fp32 accumulator of M x N; B MN-major if asked.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}
// The products of one 16-wide step; descriptors as their low words (address
// and leading offset) with constant high words, so that a step costs a 32-bit
// addition each.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups, version, 128-byte swizzle
template <uint32_t IDESC>
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "mov.b64 da, {%1, %4};\n\t"
      "mov.b64 db, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(accumulate), "n"(kDescHi), "r"(IDESC)
      : "memory");
}
// A from TMEM (binary16 pairs, lane = row), B from shared memory.
template <uint32_t IDESC>
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "mov.b64 db, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(accumulate), "n"(kDescHi), "r"(IDESC)
      : "memory");
}
// tcgen05.wait::ld that the loaded registers depend on: nothing reads them earlier.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st_32cols(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t site) {
  return __all_sync(0xffffffffu, quick_wait(bar, parity, abort, &g_err_kv4prompt, site));
}

// The same for waits with slack: the warp sleeps between polls.
__device__ __forceinline__ bool idle_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t site) {
  for (int n = 0; n < 64; ++n) {
    if (mbar_try_wait(bar, parity)) break;
    __nanosleep(64);
  }
  return warp_wait(bar, parity, abort, site);
}

// Named barriers.  A warp that polls takes issue slots from those that work:
// of the warps that wait for the same thing one polls, the others stand at a
// named barrier, which costs nothing.  1-2: a row tile's warps, 3-4: the warps
// that fill keys, values; 5: both row tiles' warps, once.
template <int WARPS>
__device__ __forceinline__ void meet(int bar) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(bar), "n"(WARPS * 32) : "memory");
}

// Where 16-byte chunk c (8 dims) of row r of a 128-row operand lies: blocks of
// 64 dims, rows of 128 bytes, chunks permuted by row % 8.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return static_cast<uint32_t>(c >> 3) * PCfg<D>::kHalf + static_cast<uint32_t>(r) * 128u +
         static_cast<uint32_t>(((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// N bytes (1, 2 or 4) in one word.
template <int N>
__device__ __forceinline__ uint32_t ld_shared(uint32_t addr) {
  uint32_t v;
  if constexpr (N == 4) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  } else if constexpr (N == 2) {
    uint16_t h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr) : "memory");
    v = h;
  } else {
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  }
  return v;
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// The rows of the CTA's runs in ctrl.alone by themselves, a softmax warp a row.
// After all runs: this takes as long as it takes, and nothing waits for it.
template <int D>
__device__ __noinline__ void runs_by_rows(const Args& a, const AttnParams& p, const PCtrl& ctrl, int64_t u0, int64_t u1) {
  using C = PCfg<D>;
  Walk walk = walk_from(p, ctrl.b, ctrl.w, ctrl.off, u0, u1 - u0);
  for (int nth = 0; next_run(a, p, walk); ++nth) {
    if ((ctrl.alone >> min(nth, 31) & 1) == 0) continue;
    const Seq& s = walk.w.s;
    const int from = (walk.lo / kT + walk.tile) * kT;
    float* slot = p.part + static_cast<int64_t>(2 * blockIdx.x + (nth > 0)) * C::kSlot;
    for (int rg = threadIdx.x >> 5; rg < kGroup; rg += kSoftWarps) {
      const int r = walk.group * kGroup + rg;
      if (r >= s.rows * p.G) break;
      float m, l, v[D / 32];
      one_row<D>(a, p, s, walk.seq, walk.kvh, r, from, min(from + walk.n * kT, walk.hi), &g_err_kv4prompt, 51, m, l, v);
      store_one_row<D>(p, s, walk.kvh, r, m, l, v, walk.n == walk.all ? nullptr : slot, rg, kGroup);
    }
  }
}

template <int D, int BS>
__global__ void __launch_bounds__(kPThreads, 1)
    kv4_prompt_kernel(const __grid_constant__ Args a, const __grid_constant__ AttnParams p) {
  using C = PCfg<D>;
  constexpr int kSB = D / BS;
  constexpr uint32_t kTileBytes = C::kTileBytes;
  constexpr int kRing = C::kRing;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PCtrl ctrl;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sq = base, sk = base + 2 * kTileBytes, sv = base + 4 * kTileBytes;
  const uint8_t* const raws = smem_raw + (base - smem_u32(smem_raw)) + 6 * kTileBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile int* abort = &ctrl.abort;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctrl.q_full[i]), 4);
      mbar_init(smem_u32(&ctrl.s_full[i][0]), 1);
      mbar_init(smem_u32(&ctrl.s_full[i][1]), 1);
      mbar_init(smem_u32(&ctrl.o_done[i][0]), 1);
      mbar_init(smem_u32(&ctrl.o_done[i][1]), 1);
      mbar_init(smem_u32(&ctrl.p_full[i][0]), 4);
      mbar_init(smem_u32(&ctrl.p_full[i][1]), 4);
      mbar_init(smem_u32(&ctrl.k_full[i]), kFillWarps);
      mbar_init(smem_u32(&ctrl.k_empty[i]), 2);
      mbar_init(smem_u32(&ctrl.v_full[i]), kFillWarps);
      mbar_init(smem_u32(&ctrl.v_empty[i]), 2);
      mbar_init(smem_u32(&ctrl.drained[i]), 1);
    }
    for (int i = 0; i < kRuns; ++i) {
      mbar_init(smem_u32(&ctrl.run_full[i]), 1);
      mbar_init(smem_u32(&ctrl.run_empty[i]), kSoftWarps + 3);  // softmax, products, loads
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(smem_u32(&ctrl.raw_full[i]), 1);
      mbar_init(smem_u32(&ctrl.raw_empty[i]), kFillWarps);
    }
    ctrl.abort = 0;
    ctrl.alone = 0;
    ctrl.b = -1;
    fence_mbar_init();
  }
  // ---- this CTA's range (as kv4attn.cu, units of this kernel)
  auto units_of = [&](int b, Span& w) -> long long {
    if (b >= a.n_seqs || !load_span(a, p, b, w)) return 0;
    return head_units(p, w) * a.Hkv;
  };
  Span mine;
  const long long mine_units = units_of(tid, mine);
  long long sum = mine_units;
  for (int b = tid + kPThreads; b < a.n_seqs; b += kPThreads) {
    Span w;
    sum += units_of(b, w);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) ctrl.sum[warp] = sum;
  __syncthreads();
  long long units = 0;
#pragma unroll 1
  for (int i = 0; i < kPWarps; ++i) units += ctrl.sum[i];
  const int cta = blockIdx.x;
  const int ctas =
      static_cast<int>(min(static_cast<long long>(gridDim.x), (units + kGroupCost) / (1 + kGroupCost)));
  grid_launch_dependents();
  if (tid == 0) p.rec[cta] = make_int4(-1, 0, 0, 0);
  if (cta >= ctas) return;  // the whole CTA
  const int64_t u0 = range_start(units, cta, ctas), u1 = range_start(units, cta + 1, ctas);
  long long before = 0;
#pragma unroll 1
  for (int start = 0; start < a.n_seqs; start += kPThreads) {
    Span w = mine;
    const long long u = start == 0 ? mine_units : units_of(start + tid, w);
    long long inc = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    __syncthreads();
    if (lane == 31) ctrl.sum[warp] = inc;
    __syncthreads();
    long long all = 0;
#pragma unroll 1
    for (int i = 0; i < kPWarps; ++i) {
      if (i < warp) inc += ctrl.sum[i];
      all += ctrl.sum[i];
    }
    inc += before;
    if (u0 >= inc - u && u0 < inc) {
      ctrl.b = start + tid;
      ctrl.off = u0 - (inc - u);
      ctrl.w = w;
    }
    __syncthreads();
    if (ctrl.b >= 0) break;
    before += all;
  }
  if (ctrl.b < 0) return;  // lengths changed under the call
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&ctrl.tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl.tmem;

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------- softmax
    regs_inc<kSoftRegs>();
    const int i = warp >> 2;                    // row tile
    const int rw = (warp & 3) * 32 + lane;      // row in it
    const bool polls = (warp & 3) == 1 + i;     // for the tile's four warps
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + i * 128, to = tmem + lanes + 256 + i * D;
    // a bit a buffer: the phase of its next scores; the phase of its last sums is
    // the other one (a barrier a buffer each: a parity tells two phases apart)
    uint32_t s_phase = 0;
    int count = 0;         // tiles so far
    // a wait that gives up (a bug) ends every later wait at once: the loops run
    // on to their ends, so that the warp-wide instructions stay together
    for (int nth = 0;; ++nth) {
      const Run& run = ctrl.run[nth % kRuns];
      if (polls) {
        warp_wait(smem_u32(&ctrl.run_full[nth % kRuns]), (nth / kRuns) & 1, abort, 63);
        if (lane == 0) ctrl.done[i][nth & 1] = run.stop || *abort;
      }
      meet<4>(1 + i);
      if (ctrl.done[i][nth & 1]) break;  // all four warps alike
      const int n_tiles = run.n;
      const int all_rows = run.rows * p.G, r0 = run.group * kGroup;
      if (r0 + i * 128 >= all_rows) {  // no row of this tile
        count += n_tiles;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctrl.run_empty[nth % kRuns]));
        continue;
      }
      const int r = r0 + i * 128 + rw;
      const int rc = min(r, all_rows - 1), tok_q = rc / p.G;
      const int head = run.kvh * p.G + (rc - tok_q * p.G);  // of the thread's row
      const int pos = p.causal ? run.len - run.rows + tok_q : run.len - 1;
      const int first = p.window > 0 ? pos - p.window + 1 : 0;  // first token the row reads
      float f_row;
      {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (run.row0 + tok_q) * p.q_stride +
                                                          static_cast<int64_t>(head) * D);
        uint4 w[D / 8];
        uint32_t am = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) w[c] = __ldg(src + c);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
          for (int y = 0; y < 4; ++y) am = max(am, max((x[y] << 16) & 0x7FFFFFFFu, x[y] & 0x7FFF0000u));
        }
        const int e = 141 - max(static_cast<int>(am >> 23), 1);
        const float s1 = p.scale_log2 < 0.f ? -pow2i(e / 2) : pow2i(e / 2), s2 = pow2i(e - e / 2);
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
          uint32_t h[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            h[y] = pack_half2(__uint_as_float(x[y] << 16) * s1 * s2, __uint_as_float(x[y] & 0xFFFF0000u) * s1 * s2);
          st_shared16(sq + i * kTileBytes + chunk_at<D>(rw, c), h[0], h[1], h[2], h[3]);
        }
        f_row = fabsf(p.scale_log2) * pow2w(-e);
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctrl.q_full[i]));

      float m = -INFINITY, l = 0.f;
      bool large = false;
      int ref_v = 13;
      int tok0 = (run.lo / kT + run.tile) * kT;
      for (int u = 0; u < 2 * n_tiles; ++u, tok0 += kU) {
        const int buf = u & 1;
        if (polls) warp_wait(smem_u32(&ctrl.s_full[i][buf]), (s_phase >> buf) & 1, abort, 49);
        meet<4>(1 + i);
        s_phase ^= 1u << buf;
        tc_fence_after();
        const int info = (count + (u >> 1)) & 3;
        float f = f_row * ctrl.k_info[info];
        if (f < 1e-37f) f = 1e-37f;  // not 0, for masked scores (-infinity) times it
        const int new_v = ctrl.v_info[info];
        const uint32_t tsu = ts + buf * kU;
        float alpha = 1.f;
        auto step = [&](auto masked) {  // kept apart: the mask's tests stay out of whole steps
          constexpr bool kMasked = decltype(masked)::value;
          auto seen = [&](int tok, float v, float other) { return !kMasked || (tok <= pos && tok >= first) ? v : other; };
          // The maximum in use serves while the row's weights stay within
          // binary16, about 2^9 above it, which one pass over the scores finds
          // while it computes them; where it does not (a run's first step, or a
          // row of the warp far above what it saw) the maximum is taken first.
          bool exact = __any_sync(0xffffffffu, m == -INFINITY);
          uint32_t h[32];  // the row's weights, binary16 pairs
          for (;;) {
            uint32_t s[32];
            if (exact) {
              float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                tmem_ld_32cols(tsu + 32 * c, s);
                tmem_ld_wait(s);
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                  const int tok = tok0 + 32 * c + x;
                  mx[(x >> 1) & 3] = fmaxf(mx[(x >> 1) & 3], fmaxf(seen(tok, __uint_as_float(s[x]), -INFINITY),
                                                                   seen(tok + 1, __uint_as_float(s[x + 1]), -INFINITY)));
                }
              }
              const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * f;
              if (top > m) {
                alpha = ex2(m - top);
                m = top;
                l *= alpha;
                large |= fabsf(top) >= kTopScore;
              }
            }
            const float bias = kTop - (m == -INFINITY ? 0.f : m);
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t s1[32];
            tmem_ld_32cols(tsu, s);
            tmem_ld_wait(s);
            tmem_ld_32cols(tsu + 32, s1);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (c == 1) tmem_ld_wait(s1);
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                const int tok = tok0 + 32 * c + 2 * x;
                const uint32_t a0 = c ? s1[2 * x] : s[2 * x], a1 = c ? s1[2 * x + 1] : s[2 * x + 1];
                const float e0 = seen(tok, ex2(fmaf(__uint_as_float(a0), f, bias)), 0.f);
                const float e1 = seen(tok + 1, ex2(fmaf(__uint_as_float(a1), f, bias)), 0.f);
                sum[2 * (x & 1)] += e0;
                sum[2 * (x & 1) + 1] += e1;
                h[16 * c + x] = pack_half2(e0, e1);
              }
            }
            // The weights are positive: none is beyond binary16 (65504) if their
            // sum is not, so that the sum says whether the maximum in use still
            // serves.
            const float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
            if (!exact && __any_sync(0xffffffffu, !(all < 65504.f))) {
              exact = true;
              continue;
            }
            l += all;
            break;
          }
          tmem_st_32cols(tsu, h);  // into columns whose scores have been read
        };
        if (__all_sync(0xffffffffu, tok0 + kU - 1 <= pos && tok0 >= first))
          step(std::false_type{});
        else
          step(std::true_type{});
        if (new_v != ref_v) {
          alpha *= pow2i(ref_v - new_v);
          ref_v = new_v;
        }
        // the sums so far, rescaled: after the step before (the earlier ones are
        // done: this step's scores came after them)
        if (u > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          warp_wait(smem_u32(&ctrl.o_done[i][buf ^ 1]), ((s_phase >> (buf ^ 1)) & 1) ^ 1u, abort, 67);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t s[32];
            tmem_ld_32cols(to + 32 * c, s);
            tmem_ld_wait(s);
#pragma unroll
            for (int x = 0; x < 32; ++x) s[x] = __float_as_uint(__uint_as_float(s[x]) * alpha);
            tmem_st_32cols(to + 32 * c, s);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctrl.p_full[i][buf]));
      }
      count += n_tiles;
#pragma unroll
      for (int buf = 0; buf < 2; ++buf)
        warp_wait(smem_u32(&ctrl.o_done[i][buf]), ((s_phase >> buf) & 1) ^ 1u, abort, 50);
      tc_fence_after();
      if (large && r < all_rows) atomicOr(&ctrl.alone, 1u << min(nth, 31));
      // rows that are taken by themselves later are stored there alone
      const bool stored = RNL_DCHECK(&g_err_kv4prompt,
                                     cta < kMaxPromptCtas && run.row0 + (all_rows - 1) / p.G < a.n_rows && head < p.Hq, 110) &&
                          r < all_rows && (*const_cast<volatile uint32_t*>(&ctrl.alone) >> min(nth, 31) & 1) == 0;
      // sums stand for value * 2^(ref_v - 127 - 13), weights and sums both times 2^7
      const bool complete = run.n == run.all;
      const float inv = complete ? (l != 0.f ? 1.f / l : 0.f) : 1.f / 128.f;
      const float fa = pow2i((ref_v - 140) / 2), fb = pow2i(ref_v - 140 - (ref_v - 140) / 2);
      const int64_t orow = static_cast<int64_t>(run.row0 + tok_q) * p.Hq + head;
      float* slot = p.part + static_cast<int64_t>(2 * cta + (nth > 0)) * C::kSlot;
      const int rg = i * 128 + rw;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t s[32];
        tmem_ld_32cols(to + 32 * c, s);
        tmem_ld_wait(s);
        float v[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) v[x] = __uint_as_float(s[x]) * inv * fa * fb;
        if (stored) {
          if (complete) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + 32 * c);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[8 * y + 2 * x], v[8 * y + 2 * x + 1]);
                w[x] = *reinterpret_cast<const uint32_t*>(&b2);
              }
              dst[y] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            float4* dst = reinterpret_cast<float4*>(slot + rg * D + 32 * c);
#pragma unroll
            for (int y = 0; y < 8; ++y) dst[y] = make_float4(v[4 * y], v[4 * y + 1], v[4 * y + 2], v[4 * y + 3]);
          }
        }
      }
      tc_fence_before();  // the next run's products overwrite these sums
      if (stored) {
        const float lt = l * (1.f / 128.f);
        if (complete) {
          if (p.lse != nullptr) p.lse[orow] = lt != 0.f ? m * kLn2 + logf(lt) : -INFINITY;
        } else {
          slot[kGroup * D + rg] = m;
          slot[kGroup * D + kGroup + rg] = lt;
        }
      }
      // a group that begins here and goes on in later CTAs
      if (i == 0 && rw == 0 && run.tile == 0 && !complete) {
        const int64_t end = run.unit + run.all;
        p.rec[cta] = make_int4(run.kvh * run.groups + run.group, run.seq,
                               static_cast<int>((end * ctas - 1) / units), nth > 0);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctrl.run_empty[nth % kRuns]));
    }
    meet<kSoftWarps>(5);  // every tile has been filled: the upper rows' warps may be ahead of the others
    if (*const_cast<volatile uint32_t*>(&ctrl.alone) != 0) runs_by_rows<D>(a, p, ctrl, u0, u1);
  } else if (warp < kMmaWarp) {
    // ---------------------------------------------- codes to binary16 tiles
    regs_dec<kFillRegs>();
    const bool values = warp >= kValueWarp;
    const int tk = tid - (values ? kValueWarp : kSoftWarps) * 32;  // token in the tile
    const int fw = warp - (values ? kValueWarp : kSoftWarps);
    const uint32_t tiles = values ? sv : sk;
    const uint32_t full = smem_u32(values ? ctrl.v_full : ctrl.k_full);
    const uint32_t empty = smem_u32(values ? ctrl.v_empty : ctrl.k_empty);
    auto top_of = [](uint32_t w) {
      uint32_t t = 0;
#pragma unroll
      for (int x = 0; x < kSB; ++x) t = max(t, (w >> (8 * x)) & 0xFFu);
      return t;
    };
    // 255 less the smallest byte that is not 0, or 0
    auto low_of = [](uint32_t w) {
      uint32_t t = 0;
#pragma unroll
      for (int x = 0; x < kSB; ++x) t = max(t, (255u - ((w >> (8 * x)) & 0xFFu)) % 255u);
      return t;
    };
    // A token with a block that is not finite (scale byte 255), keys or values: its
    // keys become NaN operands, so that exactly the rows that read it get a weight
    // that is not a number; its values become zeros.
    auto bad_bytes = [](uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & w & 0x80808080u; };
    auto clean = [&](uint32_t w) { return w & ~((bad_bytes(w) >> 7) * 255u); };
    // Of the token's 16-byte runs of codes a warp's lanes take different ones at
    // a time (run c + tk/2), and their 8-dim chunks are permuted by the token's
    // number: reads and writes free of bank conflicts.
    const uint32_t row_at = tiles + static_cast<uint32_t>(tk) * 128u;
    const uint32_t swz = static_cast<uint32_t>(tk & 7) << 4;
    const uint32_t zero = static_cast<uint32_t>(p.causal) >> 1;
    int ref_v = 13;
    int common_v = 13;  // the same over the tiles that every row reads whole
    for (int count = 0, rs = values ? 1 : 0, rp = 0;; ++count) {
      const int stage = count & 1;
      if (fw == 3) {  // polling warps on different schedulers
        idle_wait(smem_u32(&ctrl.raw_full[rs]), rp, abort, 60);
        if (lane == 0) ctrl.stop[values] = (ctrl.raw_info[rs].w & 2) || *abort;
      }
      meet<kFillWarps>(3 + values);
      if (ctrl.stop[values]) break;  // all four warps alike
      const int4 info = ctrl.raw_info[rs];
      const uint32_t raw = smem_u32(raws) + rs * C::kRaw;
      const bool live = info.x + tk >= info.y && info.x + tk < info.z;
      auto scale_word = [&](uint32_t of) -> uint32_t {
        return live ? ld_shared<kSB>(of + tk * kSB) : 0u;  // else: whatever stands there gives zero operands
      };
      uint32_t word = scale_word(raw + C::kRawCodes);
      // the tile's largest scales, over the four warps; the keys' warps look at
      // the values' too, for the softmax
      const uint32_t own = __reduce_max_sync(0xffffffffu, top_of(clean(word)));
      uint32_t other = 0;
      // whether what only some rows read may be too far above the rest (kv4.cuh, kSpread)
      const bool spread = (info.w & 4) || (values && !(info.w & 1) && ref_v > common_v);
      const uint32_t low = spread ? __reduce_max_sync(0xffffffffu, low_of(clean(word))) : 0u;
      if (values) {
        word = clean(word);
      } else {
        const uint32_t word_v = scale_word(raw + C::kRawCodes + C::kRawScales);
        other = __reduce_max_sync(0xffffffffu, top_of(clean(word_v)));
        if ((bad_bytes(word) | bad_bytes(word_v)) != 0) word = 0xFFFFFFFFu;
      }
      uint4 c[D / 32];
#pragma unroll
      for (int x = 0; x < D / 32; ++x)
        c[x] = ld_shared16(raw + tk * (D / 2) + (((x + (tk >> 1)) & (D / 32 - 1)) << 4));
      // The warp has read the place once the codes are in registers.  Program order
      // alone does not see to that: the loads may be moved to where the codes are
      // used, past the arrival, and then read what the next copy brings.  So the
      // arrival depends on them (`zero` is 0, which the compiler does not know).
      uint32_t read = info.w;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) read |= c[x].x | c[x].y | c[x].z | c[x].w;
      const bool done = __all_sync(0xffffffffu, (read & zero) == 0);
      if (lane == 0 && done) {
        ctrl.top[values][stage][fw] = static_cast<int>(own | (other << 8) | (low << 16));
        mbar_arrive(smem_u32(&ctrl.raw_empty[rs]));
      }
      if (fw == 3) idle_wait(empty + 8 * stage, ((count >> 1) & 1) ^ 1u, abort, 52);
      meet<kFillWarps>(3 + values);
      int top = 0, top_v = 0, bottom = 255;
#pragma unroll
      for (int x = 0; x < kFillWarps; ++x) {
        const int t = ctrl.top[values][stage][x];
        top = max(top, t & 0xFF);
        top_v = max(top_v, values ? t & 0xFF : (t >> 8) & 0xFF);
        bottom = min(bottom, 255 - (t >> 16));
      }
      const int before = ref_v;
      ref_v = max((info.w & 1) ? 13 : ref_v, top_v);
      bool alone = spread && top - bottom > kSpread;
      if (values) {
        const bool first = info.w & 1, cut = info.w & 4;
        common_v = max(first ? 13 : common_v, cut ? 13 : top_v);
        alone = (cut && !first && ref_v - before > kSpread) || (spread && ref_v > common_v && ref_v - bottom > kSpread);
      }
      if (alone && tk == 0) atomicOr(&ctrl.alone, 1u << (info.w >> 8));
      const int ref = values ? ref_v : max(top, 13);
      if (tk == 0 && !values) {
        ctrl.k_info[count & 3] = pow2w(ref - 140);
        ctrl.v_info[count & 3] = ref_v;
      }
      const float fr = word == 0xFFFFFFFFu ? NAN : pow2i(140 - ref);
      const uint32_t at = row_at + stage * kTileBytes;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const int r = (x + (tk >> 1)) & (D / 32 - 1);
        const uint32_t w[4] = {c[x].x, c[x].y, c[x].z, c[x].w};
        const float z = byte_scale((word >> (8 * (r * 32 / BS))) & 0xFFu) * fr;
        const __half2 m2 = h2(pack_half2(z, z));
        const uint32_t dst = at + (r >> 1) * C::kHalf;
        const uint32_t first = (static_cast<uint32_t>(r & 1) << 6) ^ swz;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t h[4];
          e2m1x8_to_half(w[y], h);
          st_shared16(dst + (first ^ (y << 4)), u32(__hmul2(h2(h[0]), m2)), u32(__hmul2(h2(h[1]), m2)),
                      u32(__hmul2(h2(h[2]), m2)), u32(__hmul2(h2(h[3]), m2)));
        }
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * stage);
      rs += 2;  // keys and values by turns
      if (rs >= kRing) {
        rs -= kRing;
        rp ^= 1;
      }
    }
  } else {
    // ------------------------------------------------------------ products
    regs_dec<kMmaRegs>();
    if (warp < kLoadWarp) {
      // A warp for each row tile: while the products of one tile run (issuing
      // them blocks), the other's warp waits for its tile's weights.
      const int i = warp - kMmaWarp;
      constexpr uint32_t kDescQK = idesc_f16(128, kU, false), kDescPV = idesc_f16(128, D, true);
      int count = 0;             // tiles so far
      uint32_t q_phase = 0, p_phase = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
        ok = __all_sync(0xffffffffu, quick_wait(smem_u32(bar), parity, abort, &g_err_kv4prompt, site)) && ok;
        return ok;
      };
      const uint32_t q_lo = desc_lo(sq, 16) + i * (kTileBytes >> 4), k_lo = desc_lo(sk, 16),
                     v_lo = desc_lo(sv, C::kHalf);
      const uint32_t ts = tmem + i * 128, to = tmem + 256 + i * D;
      constexpr uint32_t kStep = kU * 128 >> 4;  // a step's rows of an operand
      auto scores = [&](int stage, int half) {
        if (!RNL_DCHECK(&g_err_kv4prompt, stage < 2 && half < 2 && i * 128 + (half + 1) * kU <= 256, 108)) return;
        const uint32_t kd = k_lo + stage * (kTileBytes >> 4) + half * kStep;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint32_t at = ((x >> 2) * C::kHalf + (x & 3) * 32) >> 4;
          umma_ss<kDescQK>(ts + half * kU, q_lo + at, kd + at, x > 0);
        }
        umma_commit(smem_u32(&ctrl.s_full[i][half]));
      };
      auto sums = [&](int stage, int half, bool fresh) {
        if (!RNL_DCHECK(&g_err_kv4prompt, stage < 2 && half < 2 && 256 + (i + 1) * D <= 512, 109)) return;
        const uint32_t vd = v_lo + stage * (kTileBytes >> 4) + half * kStep;
#pragma unroll
        for (int x = 0; x < kU / 16; ++x)
          umma_ts<kDescPV>(to, ts + half * kU + 8 * x, vd + ((x * 2048u) >> 4), !fresh || x > 0);
        umma_commit(smem_u32(&ctrl.o_done[i][half]));
      };
      for (int nth = 0; ok; ++nth) {
        if (!wait(&ctrl.run_full[nth % kRuns], (nth / kRuns) & 1, 64)) break;
        const Run& run = ctrl.run[nth % kRuns];
        if (run.stop) break;
        const int n_tiles = run.n;
        const bool rows = run.rows * p.G - run.group * kGroup > i * 128;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctrl.run_empty[nth % kRuns]));
        if (!rows) {  // nothing to do for this row tile: hand the operands back
          for (int k = 0; k < n_tiles && ok; ++k, ++count) {
            if (!wait(&ctrl.k_full[count & 1], (count >> 1) & 1, 55) || !wait(&ctrl.v_full[count & 1], (count >> 1) & 1, 57))
              break;
            if (lane == 0) {
              mbar_arrive(smem_u32(&ctrl.k_empty[count & 1]));
              mbar_arrive(smem_u32(&ctrl.v_empty[count & 1]));
            }
          }
          continue;
        }
        if (!wait(&ctrl.q_full[i], q_phase, 54) || !wait(&ctrl.k_full[count & 1], (count >> 1) & 1, 55)) break;
        q_phase ^= 1u;
        tc_fence_after();
        if (elect_one()) {
          scores(count & 1, 0);
          scores(count & 1, 1);
          umma_commit(smem_u32(&ctrl.k_empty[count & 1]));
        }
        __syncwarp();
        // a step's sums, then the scores two steps on, into the same columns
        for (int u = 0; u < 2 * n_tiles; ++u) {
          const int half = u & 1, t = count + (u >> 1);
          const bool more = u + 2 < 2 * n_tiles;
          if (half == 0) {
            if (!wait(&ctrl.v_full[t & 1], (t >> 1) & 1, 57)) break;
            if (more && !wait(&ctrl.k_full[(t + 1) & 1], ((t + 1) >> 1) & 1, 58)) break;
          }
          // a barrier a buffer: the softmax may be a step ahead
          if (!wait(&ctrl.p_full[i][half], (p_phase >> half) & 1, 56)) break;
          p_phase ^= 1u << half;
          tc_fence_after();
          if (elect_one()) {
            sums(t & 1, half, u == 0);
            if (more) scores((t + 1) & 1, half);
            if (half == 1) {
              umma_commit(smem_u32(&ctrl.v_empty[t & 1]));
              if (more) umma_commit(smem_u32(&ctrl.k_empty[(t + 1) & 1]));
            }
          }
          __syncwarp();
        }
        count += n_tiles;
      }
      // the last arrival on this CTA's barriers
      if (ok && count > 0) wait(&ctrl.v_empty[(count - 1) & 1], ((count - 1) >> 1) & 1, 59);
      if (!ok) {  // whatever has been issued
        if (elect_one()) umma_commit(smem_u32(&ctrl.drained[i]));
        __syncwarp();
        drain_wait(smem_u32(&ctrl.drained[i]), 0);
      }
    } else if (warp == kLoadWarp) {
      // ------------------------------------------------ codes from the pages
      // A bulk copy a lane: of a page's codes, scales or (with the keys) the
      // values' scales.
      const int chunk_tokens = min(kT, a.page);
      const int what = lane & 3, chunk_at = (lane >> 2) * chunk_tokens;
      const int row_bytes = what == 0 ? D / 2 : kSB;
      const uint32_t bytes = static_cast<uint32_t>(chunk_tokens * row_bytes);
      const uint32_t dst0 = smem_u32(raws) + (what == 0 ? 0 : C::kRawCodes + (what - 1) * C::kRawScales) +
                            (lane >> 2) * bytes;
      int rs = 0;
      uint32_t rp = 1;
      auto stage_up = [&]() {
        if (++rs == kRing) {
          rs = 0;
          rp ^= 1u;
        }
      };
      bool ok = true;
      for (int nth = 0; ok; ++nth) {
        ok = idle_wait(smem_u32(&ctrl.run_full[nth % kRuns]), (nth / kRuns) & 1, abort, 65);
        const Run& run = ctrl.run[nth % kRuns];
        if (!ok || run.stop) break;
        const int n_tiles = run.n, lo = run.lo, hi = run.hi, kvh = run.kvh;
        const int common_lo = run.common_lo, common_hi = run.common_hi;
        const int* table = a.table + static_cast<int64_t>(run.seq) * a.max_pages;
        int tok0 = (lo / kT + run.tile) * kT;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctrl.run_empty[nth % kRuns]));
        auto page_of = [&](int t0) {
          const int tok = t0 + chunk_at;
          return chunk_at < kT && tok < hi && tok + chunk_tokens > lo ? __ldg(table + (tok >> a.page_shift)) : -2;
        };
        int page = page_of(tok0);
        for (int k = 0; k < n_tiles && ok; ++k, tok0 += kT) {
          const int next = k + 1 < n_tiles ? page_of(tok0 + kT) : -2;  // a tile early
          const bool there = page >= 0 && page < a.n_pages;
          if (!there && page != -2) atomicCAS(&g_err_kv4prompt, 0u, kErrArg | (51u << 8));
          const int64_t row = ((static_cast<int64_t>(page) * a.Hkv + kvh) << a.page_shift) +
                              ((tok0 + chunk_at) & (a.page - 1));
#pragma unroll
          for (int v = 0; v < 2; ++v) {  // keys, values
            bool mine = there && what < (v ? 2 : 3);
            const uint8_t* src = what == 0 ? (v ? a.v.codes : a.k.codes) : (v || what == 2 ? a.v.scales : a.k.scales);
            ok = idle_wait(smem_u32(&ctrl.raw_empty[rs]), rp, abort, 61);
            if (!ok) break;
            if (!RNL_DCHECK(&g_err_kv4prompt,
                            rs >= 0 && rs < kRing && (!there || (chunk_at + chunk_tokens <= kT && in_cache(a, row, chunk_tokens))),
                            107))
              mine = false;
            const uint32_t total = __reduce_add_sync(0xffffffffu, mine ? bytes : 0u);
            const uint32_t bar = smem_u32(&ctrl.raw_full[rs]);
            if (lane == 0) {
              const bool cut = max(tok0, lo) < common_lo || min(tok0 + kT, hi) > common_hi;
              ctrl.raw_info[rs] = make_int4(tok0, lo, hi, (k == 0) | cut << 2 | min(nth, 31) << 8);
              mbar_arrive_expect_tx(bar, total);
            }
            __syncwarp();
            if (mine) bulk_copy_g2s(dst0 + rs * C::kRaw, src + row * row_bytes, bytes, bar);
            if (v == 0) stage_up();
          }
          stage_up();
          page = next;
        }
      }
      for (int v = 0; v < 2 && ok; ++v) {
        ok = idle_wait(smem_u32(&ctrl.raw_empty[rs]), rp, abort, 61);
        if (!ok) break;
        if (lane == 0) {
          ctrl.raw_info[rs] = make_int4(0, 0, 0, 2);
          mbar_arrive(smem_u32(&ctrl.raw_full[rs]));
        }
        stage_up();
      }
      if (!ok)  // the last copies of every place, of this round or the one before
        for (int x = 0; x < kRing; ++x) drain_wait(smem_u32(&ctrl.raw_full[x]), x < rs ? rp ^ 1u : rp);
    } else if (warp == kWalkWarp && lane == 0) {
      // ------------------------------------------------ the range's runs
      Walk walk = walk_from(p, ctrl.b, ctrl.w, ctrl.off, u0, u1 - u0);
      for (int nth = 0, more = 1; more; ++nth) {
        more = next_run(a, p, walk);
        // (a run that is still read must not change: the others end by `abort`)
        if (!mbar_wait(smem_u32(&ctrl.run_empty[nth % kRuns]), ((nth / kRuns) & 1) ^ 1, abort, &g_err_kv4prompt, 66))
          break;
        Run& run = ctrl.run[nth % kRuns];
        run.stop = !more;
        if (more) {
          run.row0 = walk.w.s.row0, run.rows = walk.w.s.rows, run.len = walk.w.s.len;
          run.groups = walk.w.groups, run.group = walk.group, run.seq = walk.seq, run.kvh = walk.kvh;
          run.lo = walk.lo, run.hi = walk.hi, run.tile = walk.tile, run.n = walk.n, run.all = walk.all;
          run.unit = walk.unit;
          common_tokens(p, walk.w.s, walk.group, run.common_lo, run.common_hi);
        }
        mbar_arrive(smem_u32(&ctrl.run_full[nth % kRuns]));
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the groups that were cut, pieces in CTA order.
template <int D>
__global__ void __launch_bounds__(512)
    kv4_prompt_join_kernel(const Args a, const AttnParams p) {
  using C = PCfg<D>;
  grid_launch_dependents();
  grid_dependency_wait();
  const int first = blockIdx.x >> 2, part = blockIdx.x & 3;  // 4 CTAs a group, 64 rows each
  const int4 rec = p.rec[first];
  if (rec.x < 0) return;
  Span w;
  load_span(a, p, rec.y, w);
  const int kvh = rec.x / w.groups, group = rec.x - kvh * w.groups;
  const int all_rows = w.s.rows * p.G, r0 = group * kGroup;
  if (!RNL_DCHECK(&g_err_kv4prompt, rec.z >= first && rec.z < kMaxPromptCtas && r0 < all_rows && kvh < a.Hkv, 111)) return;
  constexpr int kTpr = D / 8;
  for (int x = threadIdx.x; x < 64 * kTpr; x += 512) {
    const int r = part * 64 + x / kTpr, d = (x % kTpr) * 8;
    if (r0 + r >= all_rows) continue;
    auto slot = [&](int c) { return p.part + static_cast<int64_t>(2 * c + (c == first ? rec.w : 0)) * C::kSlot; };
    float mm = -INFINITY, ll = 0.f, v[8] = {};
    for (int c = first; c <= rec.z; ++c) mm = fmaxf(mm, slot(c)[kGroup * D + r]);
#pragma unroll 2
    for (int c = first; c <= rec.z; ++c) {
      const float* s = slot(c);
      const float pm = s[kGroup * D + r], pl = s[kGroup * D + kGroup + r];
      const float4 y = *reinterpret_cast<const float4*>(s + r * D + d);
      const float4 z = *reinterpret_cast<const float4*>(s + r * D + d + 4);
      const float f = pl != 0.f ? ex2(pm - mm) : 0.f;  // 0: nothing read there
      ll += pl * f;
      v[0] += y.x * f, v[1] += y.y * f, v[2] += y.z * f, v[3] += y.w * f;
      v[4] += z.x * f, v[5] += z.y * f, v[6] += z.z * f, v[7] += z.w * f;
    }
    store_row<D>(p, w.s, kvh, r0 + r, d, v, mm, ll);
  }
}

// The roles' register shares add up to what the block is launched with only if
// the kernel was built with kLaunchRegs: checked once, before a first launch.
template <int D, int BS>
bool built_as_planned() {
  static const bool ok = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, kv4_prompt_kernel<D, BS>) == cudaSuccess && at.numRegs == kLaunchRegs;
  }();
  return ok;
}

template <int D, int BS>
rnl_status launch(const AttnParams& p, const Args& a, const DeviceInfo& dev, cudaStream_t s) {
  const rnl_status st =
      ensure_smem_attr(reinterpret_cast<const void*>(kv4_prompt_kernel<D, BS>), dev.device, PCfg<D>::kSmem);
  if (st != RNL_OK) return st;
  if (!built_as_planned<D, BS>()) return RNL_ERR_LAUNCH;
  const int ctas = std::min(dev.sm_count, kMaxPromptCtas);
  trace_before(s);
  kv4_prompt_kernel<D, BS><<<ctas, kPThreads, PCfg<D>::kSmem, s>>>(a, p);
  cudaError_t e = cudaGetLastError();
  trace_after(s, "kv4_prompt");
  if (e != cudaSuccess) return RNL_ERR_LAUNCH;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(4 * ctas);
  cfg.blockDim = dim3(512);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  trace_before(s);
  e = cudaLaunchKernelEx(&cfg, kv4_prompt_join_kernel<D>, a, p);
  trace_after(s, "kv4_prompt_join");
  return e == cudaSuccess ? RNL_OK : RNL_ERR_LAUNCH;
}

}  // namespace

bool kv4_prompt_fits(int64_t D) { return D == 64 || D == 128; }

size_t kv4_prompt_workspace_bytes(int64_t D) {
  const size_t slot = static_cast<size_t>(kGroup) * (static_cast<size_t>(D) + 2) * 4;
  return kMaxPromptCtas * (sizeof(int4) + 2 * slot);
}

rnl_status launch_kv4_prompt(const AttnParams& p0, const Args& a, int block, void* ws, const DeviceInfo& dev,
                             cudaStream_t s) {
  g_launched.store(true, std::memory_order_relaxed);
  AttnParams p = p0;
  p.rec = static_cast<int4*>(ws);
  p.part = reinterpret_cast<float*>(p.rec + kMaxPromptCtas);
  if (a.D == 64) return block == 64 ? launch<64, 64>(p, a, dev, s) : launch<64, 32>(p, a, dev, s);
  return block == 64 ? launch<128, 64>(p, a, dev, s) : launch<128, 32>(p, a, dev, s);
}

rnl_status read_clear_error_kv4prompt(unsigned int* word) {
  if (!g_launched.load(std::memory_order_relaxed)) return RNL_OK;
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_kv4prompt, sizeof v) != cudaSuccess) return RNL_ERR_LAUNCH;
  if (v != 0 && cudaMemcpyToSymbol(g_err_kv4prompt, &zero, sizeof zero) != cudaSuccess)
    return RNL_ERR_LAUNCH;
  *word = v;
  return RNL_OK;
}

}  // namespace rnl
