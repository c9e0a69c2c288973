// kv4attn.cu -- attention over the 4-bit paged KV cache (kv4.cuh):
//
//   out[t, h] = sum_j p_j v[j] / sum_j p_j,   p_j = exp(scale q[t, h] . k[j] - max)
//
// over the tokens j of the row's sequence that the mask leaves it, for calls
// of few rows a sequence (single tokens, drafts): the cache is read once and
// its bytes at HBM rate are the floor, so what counts is how few instructions
// a byte of codes costs.
//
// Rows and items.  The G = Hq / Hkv query heads of one key head and the rows of
// one sequence form one list of rows (row r: token r / G, head r % G); an item
// is (sequence, key head, 4, 8 or 16 of these rows).  Every item's tokens are cut
// into tiles of TT; all items' tiles, one after the other, are dealt to the
// CTAs in equal contiguous ranges, whatever the lengths are, so that no SM
// waits for a long sequence.  An item that lies in one range is written by its
// CTA; one that is cut leaves partial sums (FP32, with their maxima) in the
// workspace, and a second, dependent kernel joins them in CTA order.
//
// A warp owns a tile at a time: bulk copies (codes and scales, a page each)
// bring its keys and its values into the warp's two buffers; the next tile's
// keys are requested when these have been read, then its values.
//
// The products run on mma.sync m16n8k16 with binary16 operands, transposed, so
// that the query rows are the narrow side (8) and tokens and dims the wide one:
//   S^T = K Q^T   A = 16 tokens of keys, B = 8 query rows
//   O^T = V^T P^T A = 16 dims of values over 16 tokens, B = the weights
// A's registers come straight from the codes: E2M1 pairs convert to half2 in
// one instruction, a half2 multiplication applies the block's scale, and the
// order of dims (in S) and of tokens (in O) is free, so every lane reads whole
// 4- to 16-byte runs of codes.  tcgen05 would need both operands written to
// shared memory as binary16 first, 8 times the bytes the codes have.
//
// Measured (G = 4, D = 128, cold caches): 8 sequences of 131072 tokens 242 us,
// 4.7 TB/s of cache: latency, 59 % of the issue slots with three warps a
// scheduler that wait for their own chains (tensor pipe 25 %, conversions); 32
// sequences of 4 rows over 2000 to 9000 tokens 95 us, the same with two warps a
// scheduler (16 rows take 255 registers; tensor pipe 35 %).  head_dim 256: 64
// sequences of 1 to 16384 tokens 261 us against 174 of bytes; prompts come here too
// (kv4prompt.cu has no form for them) and read the cache once per 16 rows: 2048 and
// 1500 rows over 10240 and 8000 tokens, G = 2, 5.0 ms.
//
// Scales.  2^X of a block does not fit binary16's range, 2^(X - R) does, where
// R is the largest X of the tile (keys) or of the tiles so far (values): an
// operand is E2M1 * 2^(X - R + 13), exact down to 2^-36 of the largest (kv4.cuh,
// kSpread), and 2^(R - 13) goes into the FP32 factors of the scores and of the
// sums.  Query rows are scaled by a power of two of their own, weights by 2^15
// (p <= 1, so that weights down to 2^-29 keep all 11 bits).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv4.cuh"

namespace rnl {
namespace {

using namespace kv4;

__device__ unsigned int g_err_kv4attn;
std::atomic<bool> g_launched{false};

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCtas = 640;                              // partial-sum slots in the workspace

// What an item costs a CTA beside its tiles (queries, joining the warps), in
// tiles: counted when the tiles are dealt out.  64 sequences of 1 to 16384 tokens
// (60 us now): 58 us, with 2 tiles 88, 4 68, 9 60, 14 64.
constexpr int kItemCost = 6;

template <int D, int NT>
struct Cfg {
  static constexpr int TT = D == 256 ? 32 : 64;  // tokens a tile
  // NT = 0: 4 rows, twice in the 8 columns of a product; the second copy takes
  // the odd dims of the sums, so that they need one product instead of two
  static constexpr int kRows = NT == 0 ? 4 : 8 * NT;
  static constexpr int kTiles = NT == 0 ? 1 : NT;   // column tiles of 8
  static constexpr int kCodeBytes = TT * D / 2;                 // codes of a tile, keys or values
  static constexpr int kSideBytes = kCodeBytes + TT * D / 32;   // and scales, room for blocks of 32
  static constexpr int kPitch = D + 4;     // floats between rows of the merge buffer
  static constexpr int kSlot = kRows * (D + 2);  // floats of a partial: sums, maxima, weights
  static constexpr size_t kSmem = kWarps * 2 * kSideBytes + kWarps * kRows * kPitch * 4;
  static constexpr int kJoin = D * kTiles > 256 ? 2 : 4;  // thread groups that join pieces (static shared memory)
  // CTAs an SM, by what their registers leave: 2 with 255 registers a thread for 16 rows (3, with spills:
  // 117 against 93 us at 32 x 4 rows, D = 128), 3 for up to 8 (4: 68 against 60 us at 8 rows, D = 128)
  static constexpr int kMinCtas = NT == 2 ? 2 : 3;
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// What of a sequence the call's rows read, in tiles.
struct Span {
  Seq s;
  int groups;     // row groups of kRows
  int lo, hi;     // tokens that any row reads
  int t0, tiles;  // first tile, number of tiles (at least 1: an item without tokens still writes zeros)
};
template <int D, int NT>
__device__ __forceinline__ bool load_span(const Args& a, const AttnParams& p, int b, Span& w) {
  constexpr int TT = Cfg<D, NT>::TT;
  if (!load_seq(a, b, w.s, &g_err_kv4attn, 45) || w.s.rows == 0 || w.s.rows * p.G > p.few) return false;
  w.groups = (w.s.rows * p.G + Cfg<D, NT>::kRows - 1) / Cfg<D, NT>::kRows;
  w.lo = 0;
  w.hi = w.s.len;
  if (p.causal && p.window > 0) w.lo = max(0, w.s.len - w.s.rows + 1 - p.window);
  w.t0 = w.lo / TT;
  w.tiles = max(1, (w.hi + TT - 1) / TT - w.t0);
  return true;
}

// A place among all tiles, and what is left of the CTA's range from there on
// (in tiles, items counted as kItemCost more): at an end where left <= 0.
struct Cursor {
  int b, head, group, tile, left;
  Span w;
};
// n tiles of the range further.
template <int D, int NT>
__device__ __forceinline__ void skip(const Args& a, const AttnParams& p, Cursor& c, int n) {
  while (c.left > 0) {
    const int here = c.w.tiles - c.tile;
    if (n < here) {
      c.tile += n;
      c.left -= n;
      return;
    }
    n -= here;
    c.left -= here + kItemCost;
    c.tile = 0;
    if (++c.group < c.w.groups) continue;
    c.group = 0;
    if (++c.head == a.Hkv && c.left > 0) {
      c.head = 0;
      do {
        if (++c.b >= a.n_seqs) {
          c.left = 0;
          return;
        }
      } while (!load_span<D, NT>(a, p, c.b, c.w));
    }
  }
}

// The place of unit `off` of sequence b's items, u0 of the range [u0, u1); `at`:
// where its first tile stands.
template <int D, int NT>
__device__ __forceinline__ Cursor cursor_at(int b, const Span& w, long long off, int64_t u0, int64_t u1, int64_t& at) {
  Cursor c;
  c.b = b;
  c.w = w;
  // (a 64-bit division is slow)
  const int item = off >> 32 ? static_cast<int>(off / (c.w.tiles + kItemCost))
                             : static_cast<int>(static_cast<uint32_t>(off) / (c.w.tiles + kItemCost));
  c.head = item / c.w.groups;
  c.group = item - c.head * c.w.groups;
  c.tile = static_cast<int>(off - static_cast<long long>(item) * (c.w.tiles + kItemCost)) - kItemCost;
  c.left = static_cast<int>(u1 - u0);
  at = u0;
  if (c.tile < 0) {
    at -= c.tile;
    c.left += c.tile;
    c.tile = 0;
  }
  return c;
}

// The rows of the CTA's segments in `alone` (bit: number, up to 31) by
// themselves, a warp a row.
template <int D, int NT>
__device__ __noinline__ void segments_by_rows(const Args& a, const AttnParams& p, int b, const Span& first, long long off,
                                              int64_t u0, int64_t u1, uint32_t alone) {
  using C = Cfg<D, NT>;
  int64_t at;
  Cursor cur = cursor_at<D, NT>(b, first, off, u0, u1, at);
  for (int seg = 0; cur.left > 0; ++seg) {
    const int n = min(cur.w.tiles - cur.tile, cur.left);
    if (alone >> min(seg, 31) & 1) {
      const Seq& s = cur.w.s;
      const int from = (cur.w.t0 + cur.tile) * C::TT;
      float* slot = p.part + static_cast<int64_t>(2 * blockIdx.x + (seg > 0)) * C::kSlot;
      for (int i = threadIdx.x >> 5; i < C::kRows; i += kWarps) {
        const int r = cur.group * C::kRows + i;
        if (r >= s.rows * p.G) break;
        float m, l, v[D / 32];
        one_row<D>(a, p, s, cur.b, cur.head, r, from, min(from + n * C::TT, cur.w.hi), &g_err_kv4attn, 46, m, l, v);
        store_one_row<D>(p, s, cur.head, r, m, l, v, n == cur.w.tiles ? nullptr : slot, i, C::kRows);
      }
    }
    skip<D, NT>(a, p, cur, n);
  }
}

// MIXED: the rows of a sequence may differ in what they read (several causal
// rows).  64 sequences of 1 to 16384 tokens, Hkv = 8, a row each: 149 us with it
// (given with cu_rows), 142 without.
template <int D, int NT, int BS, bool MIXED>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kMinCtas)
    kv4_attn_kernel(const __grid_constant__ Args a, const __grid_constant__ AttnParams p) {
  using C = Cfg<D, NT>;
  constexpr int TT = C::TT, kRows = C::kRows, kPitch = C::kPitch, T8 = C::kTiles;
  constexpr bool kTwin = NT == 0;   // both parities in one product
  constexpr int kCodeBytes = C::kCodeBytes, kSideBytes = C::kSideBytes;
  constexpr int KS = D / 16;        // k-steps of the scores, and groups of 16 dims of the sums
  constexpr int MS = TT / 16;       // groups of 16 tokens a tile
  constexpr int kKB = D / 8;        // code bytes a lane takes of a key (8, 16, 32)
  constexpr int kVB = D / 16;       // of a value (4, 8, 16)
  constexpr int kKW = kKB / 4, kVW = kVB / 4;
  constexpr int kScalesPerLane = D == 256 ? 2 : 1;  // 32-element parts of a lane's key dims
  constexpr int kSB = D / BS;                       // scale bytes a token
  constexpr int kSW = (TT * kSB + 127) / 128;       // words of scales a lane looks over (1 or 2)
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kWarps * 2];
  __shared__ float sh_ml[2][kWarps][2][kRows];
  __shared__ long long sh_sum[kWarps];
  __shared__ int sh_b, sh_abort;
  __shared__ uint32_t sh_alone;  // segments whose rows are taken by themselves in the end
  __shared__ long long sh_off;
  __shared__ Span sh_w;
  float* merge = reinterpret_cast<float*>(smem + kWarps * 2 * kSideBytes);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = lane >> 2, j = lane & 3;

  if (tid == 0) {
    for (int i = 0; i < kWarps * 2; ++i) mbar_init(smem_u32(&full[i]), 1);
    sh_abort = 0;
    sh_b = -1;
    sh_alone = 0;
    fence_mbar_init();
  }
  // ---- this CTA's range of tiles
  auto units_of = [&](int b, Span& w) -> long long {
    if (b >= a.n_seqs || !load_span<D, NT>(a, p, b, w)) return 0;
    return static_cast<long long>(w.tiles + kItemCost) * w.groups * a.Hkv;
  };
  Span mine;
  const long long mine_units = units_of(tid, mine);
  long long sum = mine_units;
  for (int b = tid + kThreads; b < a.n_seqs; b += kThreads) {
    Span w;
    sum += units_of(b, w);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sh_sum[warp] = sum;
  __syncthreads();
  long long units = 0;
  for (int i = 0; i < kWarps; ++i) units += sh_sum[i];
  // at least a tile a warp for every CTA that works
  const int cta = blockIdx.x;
  const int ctas = static_cast<int>(
      min(static_cast<long long>(gridDim.x), (units + kWarps + kItemCost - 1) / (kWarps + kItemCost)));
  grid_launch_dependents();
  if (tid == 0) p.rec[cta] = make_int4(-1, 0, 0, 0);
  // (launched early, beside the prompt kernel's join: both are done before this
  // grid is, so that what follows in the stream comes after them)
  if (cta >= ctas) {
    grid_dependency_wait();
    return;  // the whole CTA
  }
  const int64_t u0 = range_start(units, cta, ctas), u1 = range_start(units, cta + 1, ctas);
  long long before = 0;
  for (int base = 0; base < a.n_seqs; base += kThreads) {
    Span w = mine;
    const long long u = base == 0 ? mine_units : units_of(base + tid, w);
    long long inc = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    __syncthreads();
    if (lane == 31) sh_sum[warp] = inc;
    __syncthreads();
    for (int i = 0; i < warp; ++i) inc += sh_sum[i];
    long long all = 0;
    for (int i = 0; i < kWarps; ++i) all += sh_sum[i];
    inc += before;
    if (u0 >= inc - u && u0 < inc) {
      sh_b = base + tid;
      sh_off = u0 - (inc - u);
      sh_w = w;
    }
    __syncthreads();
    if (sh_b >= 0) break;
    before += all;
  }
  if (sh_b < 0) {  // lengths changed under the call
    grid_dependency_wait();
    return;
  }
  int64_t at;  // where the range's first tile stands
  Cursor cur = cursor_at<D, NT>(sh_b, sh_w, sh_off, u0, u1, at);  // the CTA's place

  // ---- the warp's buffers: a tile of keys and a tile of values, each fetched
  // again as soon as it has been read
  const uint32_t buf = smem_u32(smem) + warp * 2 * kSideBytes;
  uint8_t* const ks = smem + warp * 2 * kSideBytes;
  uint8_t* const vs = ks + kSideBytes;
  const uint32_t bar_k = smem_u32(&full[warp * 2]), bar_v = bar_k + 8;
  uint32_t phase = 0;  // of both
  // copies of a tile: a page's codes and scales on two lanes
  const int chunk_tokens = min(TT, a.page);
  const bool is_code = (lane & 1) == 0;
  const int chunk_at = (lane >> 1) * chunk_tokens;
  const int row_bytes = is_code ? D / 2 : kSB;
  const uint32_t copy_bytes = static_cast<uint32_t>(chunk_tokens * row_bytes);
  const uint32_t copy_dst = buf + (is_code ? 0 : kCodeBytes) + (lane >> 1) * copy_bytes;
  const uint8_t* const src_k = is_code ? a.k.codes : a.k.scales;
  const uint8_t* const src_v = is_code ? a.v.codes : a.v.scales;
  Cursor ahead = cur;      // the next tile to fetch
  int page = -1;           // this lane's page of it, -1: none
  int page_off = 0;        // tokens into the page, and its key head
  int page_head = 0;
  auto locate = [&]() {    // the table's entry is looked up a tile early
    page = -1;
    if (ahead.left <= 0) return;
    const int tok = (ahead.w.t0 + ahead.tile) * TT + chunk_at;
    page_off = tok & (a.page - 1);
    page_head = ahead.head;
    // (not what lies wholly in front of a window: that page may have been given back)
    if (chunk_at < TT && tok < ahead.w.hi && tok + chunk_tokens > ahead.w.lo)
      page = __ldg(a.table + static_cast<int64_t>(ahead.b) * a.max_pages + (tok >> a.page_shift));
    else
      page = -2;
  };
  int64_t fetch_at = 0;      // byte offset of this lane's copy
  uint32_t fetch_lanes = 0;  // the lanes that have one
  auto fetch_keys = [&]() {  // and settle the place that the values' copies use too
    const bool ok = page >= 0 && page < a.n_pages &&
                    RNL_DCHECK(&g_err_kv4attn,
                               chunk_at + chunk_tokens <= TT &&
                                   in_cache(a, ((static_cast<int64_t>(page) * a.Hkv + page_head) << a.page_shift) + page_off,
                                            chunk_tokens),
                               104);
    if (!ok && page != -2 && (page < 0 || page >= a.n_pages)) atomicCAS(&g_err_kv4attn, 0u, kErrArg | (46u << 8));  // a page id outside the cache
    fetch_lanes = __ballot_sync(0xffffffffu, ok);
    fetch_at = (((static_cast<int64_t>(page) * a.Hkv + page_head) << a.page_shift) + page_off) * row_bytes;
    if (lane == 0)
      mbar_arrive_expect_tx(bar_k, __popc(fetch_lanes) / 2 * (chunk_tokens * (D / 2 + kSB)));
    __syncwarp();
    if (ok) bulk_copy_g2s(copy_dst, src_k + fetch_at, copy_bytes, bar_k);
  };
  auto fetch_values = [&]() {
    if (lane == 0)
      mbar_arrive_expect_tx(bar_v, __popc(fetch_lanes) / 2 * (chunk_tokens * (D / 2 + kSB)));
    __syncwarp();
    if (fetch_lanes >> lane & 1) bulk_copy_g2s(copy_dst + kSideBytes, src_v + fetch_at, copy_bytes, bar_v);
  };
  skip<D, NT>(a, p, ahead, warp);
  locate();
  __syncthreads();  // barriers initialised
  if (ahead.left > 0) {
    fetch_keys();
    fetch_values();
    skip<D, NT>(a, p, ahead, kWarps);
    locate();
  }

  bool gave_up = false;  // a wait of this warp ran out: it fetches no more and runs to its end, phase as it was
  int done = 0;      // tiles of the range before the current segment
  int seg = 0;
  while (cur.left > 0) {
    // ---- a segment: the range's tiles of one item
    const int seg_tiles = min(cur.w.tiles - cur.tile, cur.left);
    const int kvh = cur.head;
    const int all_rows = cur.w.s.rows * p.G;
    const int r0 = cur.group * kRows;
    // queries: lane (n, j) holds dims [j D/4, (j + 1) D/4) of row n of each tile of 8
    uint32_t qf[T8][KS][2];
    float f_row[T8][2];  // score factors of rows 2j and 2j + 1
    int pos[T8][2];      // last token they read
#pragma unroll
    for (int t = 0; t < T8; ++t) {
      const int r = min(r0 + t * 8 + (kTwin ? n & 3 : n), all_rows - 1);
      const int tok = r / p.G;
      const __nv_bfloat16* src = p.q + (cur.w.s.row0 + tok) * p.q_stride +
                                 static_cast<int64_t>(kvh * p.G + (r - tok * p.G)) * D + j * (D / 4);
      uint32_t w[D / 8];
      uint32_t am = 0;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(src) + i);
        w[4 * i] = x.x;
        w[4 * i + 1] = x.y;
        w[4 * i + 2] = x.z;
        w[4 * i + 3] = x.w;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) am = max(am, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      const int eb = static_cast<int>(am >> 23);
      // exponent field 127 + 14 for the largest: times 2^(141 - eb), in two steps
      const int e = 141 - max(eb, 1);
      // the scale's sign goes with the query: score factors are then positive
      const float s1 = p.scale_log2 < 0.f ? -pow2i(e / 2) : pow2i(e / 2), s2 = pow2i(e - e / 2);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        qf[t][i >> 1][i & 1] = pack_half2(__uint_as_float(w[i] << 16) * s1 * s2,
                                          __uint_as_float(w[i] & 0xFFFF0000u) * s1 * s2);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int er = __shfl_sync(0xffffffffu, e, (2 * j + h) * 4);
        f_row[t][h] = fabsf(p.scale_log2) * pow2w(-er);
        const int rr = min(r0 + t * 8 + (kTwin ? 2 * (j & 1) : 2 * j) + h, all_rows - 1);
        pos[t][h] = p.causal ? cur.w.s.len - cur.w.s.rows + rr / p.G : cur.w.s.len - 1;
      }
    }
    const int r_last = min(r0 + kRows, all_rows) - 1;
    const int pos_min = p.causal ? cur.w.s.len - cur.w.s.rows + r0 / p.G : cur.w.s.len - 1;
    const int pos_max = p.causal ? cur.w.s.len - cur.w.s.rows + r_last / p.G : cur.w.s.len - 1;
    const int win = p.window > 0 ? p.window : 0x40000000;

    constexpr int KO = kTwin ? KS / 2 : KS;  // accumulators of 4
    float o[T8][KO][4];
    float m[T8][2], l[T8][2];
#pragma unroll
    for (int t = 0; t < T8; ++t) {
#pragma unroll
      for (int i = 0; i < KO; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }
    // tokens that some row of the group reads
    const int seen_lo = max(cur.w.lo, pos_min - win + 1), seen_hi = min(cur.w.hi, pos_max + 1);
    int ref_v = MIXED ? 0 : 13;  // 0: no tile yet; else at least 13 (below, the factor 2^(140 - ref) would leave binary32)
    int common_v = 13;     // the same over the tiles that every row reads whole
    bool alone = false;    // the rows have to be taken by themselves (one_row)

    for (int i = (warp - done % kWarps + kWarps) % kWarps; i < seg_tiles; i += kWarps) {
      const int tok0 = (cur.w.t0 + cur.tile + i) * TT;
      // a tile that no row of this group reads (causal, earlier rows): nothing
      const bool any = tok0 < seen_hi && tok0 + TT > seen_lo;
      const bool whole = tok0 + TT - 1 <= pos_min && tok0 > pos_max - win;
      const bool cut = MIXED && pos_min != pos_max && !whole;  // with tokens that only some of the rows read
      const bool edge = tok0 < seen_lo || tok0 + TT > seen_hi || cut;
      // largest scale byte of a side; at an edge of what the rows read, the
      // scale bytes of tokens that no row reads become 0 first, so that
      // whatever stands there gives zero operands.  A block that is not finite
      // (byte 255) becomes zeros too, and the rows that read its token get a
      // normaliser that is not a number
      // `low`: the smallest byte that is not 0 where `edge` (MIXED), else 256
      auto top_scale = [&](uint8_t* scales, bool edge, int& low) {
        uint32_t* sc = reinterpret_cast<uint32_t*>(scales) + lane;
        uint32_t w[kSW];
#pragma unroll
        for (int y = 0; y < kSW; ++y) {
          const bool has = (y * 32 + lane) * 4 < TT * kSB;
          w[y] = has ? sc[y * 32] : 0u;
          if (edge) {
            uint32_t keep = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int tok = tok0 + ((y * 32 + lane) * 4 + x) / kSB;
              if (tok >= seen_lo && tok < seen_hi) keep |= 0xFFu << (8 * x);
            }
            w[y] &= keep;
            if (has) sc[y * 32] = w[y];
          }
        }
        low = 256;
        if (edge) {
          if constexpr (MIXED) {
            uint32_t t = 0xFFFFFFFFu;
#pragma unroll
            for (int y = 0; y < kSW; ++y) t = __vminu4(t, __vsub4(w[y], 0x01010101u));  // 0 becomes 255
            t = __vminu4(t, t >> 16 | 0xFFFF0000u);
            low = static_cast<int>(__reduce_min_sync(0xffffffffu, min(t & 0xFFu, (t >> 8) & 0xFFu))) + 1;
          }
          fence_proxy_async_shared();  // the next copy into this buffer comes after these writes
          __syncwarp();
        }
        auto top = [&]() {
          uint32_t t = w[0];
          if constexpr (kSW == 2) t = __vmaxu4(t, w[1]);
          t = __vmaxu4(t, t >> 16);
          return static_cast<int>(__reduce_max_sync(0xffffffffu, max(t & 0xFFu, (t >> 8) & 0xFFu)));
        };
        const int all = top();
        if (all != 255) return all;
        uint64_t bad = 0;
#pragma unroll
        for (int y = 0; y < kSW; ++y) {
          uint32_t keep = 0;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if ((w[y] >> (8 * x) & 0xFFu) == 255u)
              bad |= 1ull << ((y * 32 + lane) * 4 + x) / kSB;
            else
              keep |= 0xFFu << (8 * x);
          }
          w[y] &= keep;
          if ((y * 32 + lane) * 4 < TT * kSB) sc[y * 32] = w[y];
        }
        bad = static_cast<uint64_t>(__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(bad >> 32))) << 32 |
              __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(bad));
        fence_proxy_async_shared();
        __syncwarp();
#pragma unroll
        for (int t = 0; t < T8; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int lo = max(pos[t][h] - win + 1 - tok0, 0), hi = min(pos[t][h] - tok0, TT - 1);
            if (hi >= lo && (bad & (~0ull << lo) & (~0ull >> (63 - hi))) != 0) l[t][h] = NAN;
          }
        return top();
      };
      gave_up |= !quick_wait(bar_k, phase & 1, &sh_abort, &g_err_kv4attn, 47);
      float s[T8][MS][4];
      float f_tile = 0.f;
      if (any) {
        int low;
        const int ref_k = max(top_scale(ks + kCodeBytes, edge, low), 13);
        alone |= cut && ref_k - low > kSpread;
        const float fk = pow2i(140 - ref_k);
        f_tile = pow2w(ref_k - 140);
        // ---- scores, transposed: 16 tokens x 8 rows
        // tokens of a group of 16: matrix row x is token x/2 (x even) or 4 + (x/2 ^ 1)
        // (x odd), plus 8 for x >= 8: reads of keys free of bank conflicts
        const int tk = (n & 1) ? 4 + ((n >> 1) ^ 1) : (n >> 1);
        const uint8_t* c0 = ks + tk * (D / 2) + j * kKB;
        const uint8_t* sc0 = ks + kCodeBytes + tk * kSB + j * (D / 4) / BS;
#pragma unroll
        for (int ms = 0; ms < MS; ++ms) {
          uint32_t w0[kKW], w1[kKW];
          const uint8_t* c = c0 + ms * 8 * D;
          if constexpr (kKW == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(c), y = *reinterpret_cast<const uint2*>(c + 4 * D);
            w0[0] = x.x, w0[1] = x.y, w1[0] = y.x, w1[1] = y.y;
          } else {
#pragma unroll
            for (int x = 0; x < kKW / 4; ++x) {
              const uint4 u = reinterpret_cast<const uint4*>(c)[x], y = reinterpret_cast<const uint4*>(c + 4 * D)[x];
              w0[4 * x] = u.x, w0[4 * x + 1] = u.y, w0[4 * x + 2] = u.z, w0[4 * x + 3] = u.w;
              w1[4 * x] = y.x, w1[4 * x + 1] = y.y, w1[4 * x + 2] = y.z, w1[4 * x + 3] = y.w;
            }
          }
          __half2 m0[kScalesPerLane], m1[kScalesPerLane];
#pragma unroll
          for (int x = 0; x < kScalesPerLane; ++x) {
            const float a0 = byte_scale(sc0[ms * 16 * kSB + x * 32 / BS]) * fk;
            const float a1 = byte_scale(sc0[ms * 16 * kSB + 8 * kSB + x * 32 / BS]) * fk;
            m0[x] = h2(pack_half2(a0, a0));
            m1[x] = h2(pack_half2(a1, a1));
          }
#pragma unroll
          for (int t = 0; t < T8; ++t) s[t][ms][0] = s[t][ms][1] = s[t][ms][2] = s[t][ms][3] = 0.f;
#pragma unroll
          for (int w = 0; w < kKW; ++w) {  // a word: 8 dims, two k-steps
            uint32_t h0[4], h1[4];
            e2m1x8_to_half(w0[w], h0);
            e2m1x8_to_half(w1[w], h1);
            const int x = w / (kKW / kScalesPerLane);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t af[4] = {u32(__hmul2(h2(h0[2 * k]), m0[x])), u32(__hmul2(h2(h1[2 * k]), m1[x])),
                                      u32(__hmul2(h2(h0[2 * k + 1]), m0[x])), u32(__hmul2(h2(h1[2 * k + 1]), m1[x]))};
#pragma unroll
              for (int t = 0; t < T8; ++t) mma_f16(s[t][ms], af, qf[t][2 * w + k][0], qf[t][2 * w + k][1]);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the keys
      bool more = __all_sync(0xffffffffu, ahead.left > 0 && !gave_up);
      if (more) fetch_keys();
      gave_up |= !quick_wait(bar_v, phase & 1, &sh_abort, &g_err_kv4attn, 47);
      more = __all_sync(0xffffffffu, more && !gave_up);
      phase ^= gave_up ? 0u : 1u;
      if (any) {
        // ---- softmax over the tile
        int low;
        const int top_v = top_scale(vs + kCodeBytes, edge || (MIXED && ref_v > common_v), low);
        const int new_v = MIXED ? max(max(ref_v, top_v), 13) : max(ref_v, top_v);
        if constexpr (MIXED) {
          common_v = max(common_v, cut ? 13 : top_v);
          // far above the sums so far, or this tile's values far below what only some rows read
          alone |= (cut && ref_v != 0 && new_v - ref_v > kSpread) || (new_v > common_v && new_v - low > kSpread);
        }
        const float fv = ref_v == new_v ? 1.f : pow2i(ref_v - new_v);
        ref_v = new_v;
        uint32_t pb[T8][MS][2];
#pragma unroll
        for (int t = 0; t < T8; ++t) {
          float mx[2] = {-INFINITY, -INFINITY};
          float f[2] = {f_row[t][0] * f_tile, f_row[t][1] * f_tile};
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (f[h] < 1e-37f) f[h] = 1e-37f;  // not 0, for masked scores (-infinity) times it
#pragma unroll
          for (int ms = 0; ms < MS; ++ms)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if (!whole) {
                const int tok = tok0 + ms * 16 + ((n & 1) ? 4 + ((n >> 1) ^ 1) : (n >> 1)) + (x >> 1) * 8;
                if (tok > pos[t][x & 1] || tok <= pos[t][x & 1] - win) s[t][ms][x] = -INFINITY;
              }
              mx[x & 1] = fmaxf(mx[x & 1], s[t][ms][x]);
            }
          float base[2], al[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 4));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 8));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 16));
            const float mn = fmaxf(m[t][h], mx[h] * f[h]);
            const float mu = mn == -INFINITY ? 0.f : mn;
            al[h] = ex2(m[t][h] - mu);
            base[h] = 15.f - mu;
            m[t][h] = mn;
            l[t][h] *= al[h];
            al[h] *= fv;
          }
          if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
            for (int i2 = 0; i2 < KO; ++i2) {
              o[t][i2][0] *= al[0];
              o[t][i2][1] *= al[1];
              o[t][i2][2] *= al[0];
              o[t][i2][3] *= al[1];
            }
          }
#pragma unroll
          for (int ms = 0; ms < MS; ++ms) {
            float e[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              e[x] = ex2(fmaf(s[t][ms][x], f[x & 1], base[x & 1]));
              l[t][x & 1] += e[x];
            }
            pb[t][ms][0] = movmatrix_trans(pack_half2(e[0], e[1]));
            pb[t][ms][1] = movmatrix_trans(pack_half2(e[2], e[3]));
          }
        }
        // ---- weighted values, transposed.  A register of A is a pair of dims
        // of one token, so the matrix' k runs over (token, parity), 8 tokens a
        // step, and two products with the weights at the even or at the odd
        // places give the even and the odd dims: twice the products, which the
        // tensor cores have room for, and no permutation of pairs
        const float fr = pow2i(140 - ref_v);
        // tokens of k = 2j and 2j + 1 of the scores' group of 8
        const uint8_t* v0 = vs + j * (D / 2) + n * kVB;
        const uint8_t* v1 = vs + (4 + (j ^ 1)) * (D / 2) + n * kVB;
        const uint8_t* z0 = vs + kCodeBytes + j * kSB + n * (D / 8) / BS;
        const uint8_t* z1 = vs + kCodeBytes + (4 + (j ^ 1)) * kSB + n * (D / 8) / BS;
#pragma unroll
        for (int ms = 0; ms < MS; ++ms)
#pragma unroll
          for (int e8 = 0; e8 < 2; ++e8) {  // 8 tokens
            uint32_t w[2][kVW];
            __half2 sc[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint8_t* c = (x ? v1 : v0) + (ms * 2 + e8) * 4 * D;
              if constexpr (kVW == 1) {
                w[x][0] = *reinterpret_cast<const uint32_t*>(c);
              } else if constexpr (kVW == 2) {
                const uint2 u = *reinterpret_cast<const uint2*>(c);
                w[x][0] = u.x, w[x][1] = u.y;
              } else {
                const uint4 u = *reinterpret_cast<const uint4*>(c);
                w[x][0] = u.x, w[x][1] = u.y, w[x][2] = u.z, w[x][3] = u.w;
              }
              const float z = byte_scale((x ? z1 : z0)[(ms * 2 + e8) * 8 * kSB]) * fr;
              sc[x] = h2(pack_half2(z, z));
            }
            uint32_t be[T8][2], bo[T8][2];
#pragma unroll
            for (int t = 0; t < T8; ++t) {
              if constexpr (kTwin) {  // rows 0 .. 3 at the even places, their copies at the odd ones
                be[t][0] = __byte_perm(pb[t][ms][e8], 0u, n < 4 ? 0x4410u : 0x1044u);
                be[t][1] = __byte_perm(pb[t][ms][e8], 0u, n < 4 ? 0x4432u : 0x3244u);
              } else {
                be[t][0] = pb[t][ms][e8] & 0xFFFFu;
                bo[t][0] = pb[t][ms][e8] << 16;
                be[t][1] = pb[t][ms][e8] >> 16;
                bo[t][1] = pb[t][ms][e8] & 0xFFFF0000u;
              }
            }
#pragma unroll
            for (int x = 0; x < kVW; ++x) {
              uint32_t ha[4], hb[4];
              e2m1x8_to_half(w[0][x], ha);
              e2m1x8_to_half(w[1][x], hb);
#pragma unroll
              for (int y = 0; y < 2; ++y) {  // dims 8x + 4y .. + 3 of the lane's
                const uint32_t af[4] = {u32(__hmul2(h2(ha[2 * y]), sc[0])), u32(__hmul2(h2(ha[2 * y + 1]), sc[0])),
                                        u32(__hmul2(h2(hb[2 * y]), sc[1])), u32(__hmul2(h2(hb[2 * y + 1]), sc[1]))};
#pragma unroll
                for (int t = 0; t < T8; ++t) {
                  if constexpr (kTwin) {
                    mma_f16(o[t][2 * x + y], af, be[t][0], be[t][1]);
                  } else {
                    mma_f16(o[t][2 * (2 * x + y)], af, be[t][0], be[t][1]);
                    mma_f16(o[t][2 * (2 * x + y) + 1], af, bo[t][0], bo[t][1]);
                  }
                }
              }
            }
          }
      }
      __syncwarp();  // every lane has read the values
      if (more) {
        fetch_values();
        skip<D, NT>(a, p, ahead, kWarps);
        locate();
      }
    }

    // ---- join the warps
    float(*ml)[2][kRows] = sh_ml[seg & 1];
#pragma unroll
    for (int t = 0; t < T8; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = l[t][h];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (n == 0 && t * 8 + 2 * j + h < kRows) {
          ml[warp][0][t * 8 + 2 * j + h] = m[t][h];
          ml[warp][1][t * 8 + 2 * j + h] = x;
        }
        l[t][h] = x;
      }
    if (MIXED && alone && lane == 0) atomicOr(&sh_alone, 1u << min(seg, 31));
    __syncthreads();
#pragma unroll
    for (int t = 0; t < T8; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = t * 8 + (kTwin ? 2 * (j & 1) : 2 * j) + h;
        float mm = ml[0][0][r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, ml[w][0][r]);
        // sums stand for value * 2^(ref_v - 127 - 13) * p 2^15
        const float f = l[t][h] == 0.f ? 0.f : ex2(m[t][h] - mm);
        const float fa = pow2i((ref_v - 155) / 2), fb = pow2i(ref_v - 155 - (ref_v - 155) / 2);
        float* dst = merge + (warp * kRows + r) * kPitch + n * (D / 8);
        if constexpr (kTwin) {
#pragma unroll
          for (int i = 0; i < KO; ++i) {  // even dims in columns 0 .. 3, odd dims in 4 .. 7
            dst[4 * i + (j >> 1)] = o[t][i][h] * f * fa * fb;
            dst[4 * i + 2 + (j >> 1)] = o[t][i][2 + h] * f * fa * fb;
          }
        } else {
#pragma unroll
          for (int i = 0; i < KO; i += 2)
            *reinterpret_cast<float4*>(dst + 2 * i) =  // o[i]: even dims, o[i + 1]: odd dims
                make_float4(o[t][i][h] * f * fa * fb, o[t][i + 1][h] * f * fa * fb, o[t][i][2 + h] * f * fa * fb,
                            o[t][i + 1][2 + h] * f * fa * fb);
        }
      }
    __syncthreads();
    const bool complete = seg_tiles == cur.w.tiles;
    float* slot = p.part + static_cast<int64_t>(2 * cta + (seg > 0)) * C::kSlot;
    constexpr int kTpr = D / 8;  // threads a row, 8 dims each
    for (int x = tid; x < kRows * kTpr; x += kThreads) {
      const int r = x / kTpr, d = (x - r * kTpr) * 8;
      if (!RNL_DCHECK(&g_err_kv4attn,
                      cta < kMaxCtas && cur.w.s.row0 + (all_rows - 1) / p.G < a.n_rows && (kvh + 1) * p.G <= p.Hq, 105))
        continue;
      if (r0 + r >= all_rows || (sh_alone >> min(seg, 31) & 1)) continue;
      float mm = -INFINITY, ll = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[w][0][r]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (ml[w][1][r] != 0.f) ll += ml[w][1][r] * ex2(ml[w][0][r] - mm);
      ll *= 1.f / 32768.f;
      float v[8] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(merge + (w * kRows + r) * kPitch + d);
        const float4 z = *reinterpret_cast<const float4*>(merge + (w * kRows + r) * kPitch + d + 4);
        v[0] += y.x, v[1] += y.y, v[2] += y.z, v[3] += y.w;
        v[4] += z.x, v[5] += z.y, v[6] += z.z, v[7] += z.w;
      }
      // scores that the steps of 15 - maximum are too coarse for: a weight may have
      // left binary16 (the sums are not finite then) or vanished
      if (d == 0 && (!(fabsf(v[0]) < INFINITY) || (fabsf(mm) >= kTopScore && mm != -INFINITY)))
        atomicOr(&sh_alone, 1u << min(seg, 31));
      if (complete) {
        store_row<D>(p, cur.w.s, kvh, r0 + r, d, v, mm, ll);
      } else {
        float4* dst = reinterpret_cast<float4*>(slot + r * D + d);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        if (d == 0) {
          slot[kRows * D + r] = mm;
          slot[kRows * D + kRows + r] = ll;
        }
      }
    }
    // the item begins here and goes on in later CTAs: this CTA's record (unit x
    // is in the last range c with units c / ctas < x + 1)
    if (tid == 0 && cur.tile == 0 && !complete) {
      const int64_t end = at + cur.w.tiles;  // the item's last tile + 1
      const int last = static_cast<int>((end * ctas - 1) / units);
      p.rec[cta] = make_int4(cur.head * cur.w.groups + cur.group, cur.b, last, seg > 0);
    }
    done += seg_tiles;
    ++seg;
    at += seg_tiles + kItemCost;
    skip<D, NT>(a, p, cur, seg_tiles);
  }
  if (gave_up) {  // keys and values of that tile, and the next one's keys if they were asked for
    drain_wait(bar_k, phase & 1);
    drain_wait(bar_v, phase & 1);
    drain_wait(bar_k, (phase & 1) ^ 1u);
  }
  __syncthreads();
  if (sh_alone != 0)
    segments_by_rows<D, NT>(a, p, sh_b, sh_w, sh_off, u0, u1, sh_alone);
  grid_dependency_wait();
}

// Joins the partial sums of the items that were cut: CTA c the one that CTA c
// of the first kernel began.  kJoin groups of threads take every kJoin-th piece,
// each with the pieces' maxima first and then their sums; the groups are added
// in order.
template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kJoin * 128)
    kv4_attn_join_kernel(const Args a, const AttnParams p) {
  using C = Cfg<D, NT>;
  constexpr int kRows = C::kRows, kTpr = D / 8, kJoin = C::kJoin;
  __shared__ float sh_m[kRows], sh_l[kJoin][kRows];
  __shared__ __align__(16) float sh_v[kJoin][kRows][D];
  grid_dependency_wait();
  const int first = blockIdx.x;
  const int4 rec = p.rec[first];
  if (rec.x < 0) return;
  Span w;
  load_span<D, NT>(a, p, rec.y, w);
  const int kvh = rec.x / w.groups, group = rec.x - kvh * w.groups;
  const int all_rows = w.s.rows * p.G, r0 = group * kRows;
  if (!RNL_DCHECK(&g_err_kv4attn, rec.z >= first && rec.z < kMaxCtas && r0 < all_rows && kvh < a.Hkv, 106)) return;
  const int tid = threadIdx.x, g = tid >> 7;
  const float* base = p.part + static_cast<int64_t>(2) * first * C::kSlot;
  auto slot = [&](int c) { return base + static_cast<int64_t>(2 * (c - first) + (c == first ? rec.w : 0)) * C::kSlot; };
  // maxima: a warp a row
  for (int r = tid >> 5; r < kRows; r += kJoin * 4) {
    float mm = -INFINITY;
    for (int c = first + (tid & 31); c <= rec.z; c += 32) mm = fmaxf(mm, slot(c)[kRows * D + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    if ((tid & 31) == 0) sh_m[r] = mm;
  }
  __syncthreads();
  for (int x = tid & 127; x < kRows * kTpr; x += 128) {
    const int r = x / kTpr, d = (x - r * kTpr) * 8;
    const float mm = sh_m[r];
    float ll = 0.f, v[8] = {};
#pragma unroll 4
    for (int c = first + g; c <= rec.z; c += kJoin) {
      const float* s = slot(c);
      const float pm = s[kRows * D + r], pl = s[kRows * D + kRows + r];
      const float4 y = *reinterpret_cast<const float4*>(s + r * D + d);
      const float4 z = *reinterpret_cast<const float4*>(s + r * D + d + 4);
      const float f = pl != 0.f ? ex2(pm - mm) : 0.f;
      ll += pl * f;
      v[0] += y.x * f, v[1] += y.y * f, v[2] += y.z * f, v[3] += y.w * f;
      v[4] += z.x * f, v[5] += z.y * f, v[6] += z.z * f, v[7] += z.w * f;
    }
    *reinterpret_cast<float4*>(&sh_v[g][r][d]) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(&sh_v[g][r][d + 4]) = make_float4(v[4], v[5], v[6], v[7]);
    if (d == 0) sh_l[g][r] = ll;
  }
  __syncthreads();
  for (int x = tid; x < kRows * kTpr; x += kJoin * 128) {
    const int r = x / kTpr, d = (x - r * kTpr) * 8;
    if (r0 + r >= all_rows) continue;
    float ll = 0.f, v[8] = {};
#pragma unroll
    for (int i = 0; i < kJoin; ++i) {
      ll += sh_l[i][r];
#pragma unroll
      for (int y = 0; y < 8; ++y) v[y] += sh_v[i][r][d + y];
    }
    store_row<D>(p, w.s, kvh, r0 + r, d, v, sh_m[r], ll);
  }
}

template <int D, int NT, int BS, bool MIXED>
rnl_status launch_split(const AttnParams& p, const Args& a, const DeviceInfo& dev, bool after_prompt, cudaStream_t s) {
  using C = Cfg<D, NT>;
  const rnl_status st = ensure_smem_attr(reinterpret_cast<const void*>(kv4_attn_kernel<D, NT, BS, MIXED>), dev.device, C::kSmem);
  if (st != RNL_OK) return st;
  const int ctas = std::min(dev.sm_count * C::kMinCtas, kMaxCtas);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = at;
  // early only behind this call's own prompt kernels: what stands before the
  // call in the stream may write what this kernel reads
  cfg.numAttrs = after_prompt ? 1 : 0;
  trace_before(s);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_attn_kernel<D, NT, BS, MIXED>, a, p);
  trace_after(s, "kv4_attn");
  if (e != cudaSuccess) return RNL_ERR_LAUNCH;
  cfg.blockDim = dim3(C::kJoin * 128);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  trace_before(s);
  e = cudaLaunchKernelEx(&cfg, kv4_attn_join_kernel<D, NT>, a, p);
  trace_after(s, "kv4_attn_join");
  return e == cudaSuccess ? RNL_OK : RNL_ERR_LAUNCH;
}

}  // namespace

namespace {
// Rows of a sequence (times G) up to which this file's kernel takes it.  It reads
// the cache once per 16 rows, the prompt kernel once per 256, but that takes
// 30 us longer to start: 8, 16 and 32 rows (G = 4) of 32 sequences of 2000 to
// 9000 tokens 154, 281 and 531 us here, 168, 175 and 179 us there.
constexpr int kFewRows = 32;
// Rows times key heads times tokens (as many as the tables can hold) up to which
// the prompt kernel is not launched at all: 16 rows of 2 sequences of up to 9000
// tokens (9.2 million) 37 us here, 60 us there; 32 rows over 12000 (12.3 million)
// 58 and 68; 32 rows of 2 sequences of 6000 (12.3 million) 64 and 56.  Lengths are on
// the device, so tables with room for a longer context count as longer sequences: 8
// rows (G = 4) of 2 sequences of 6000 tokens 32 us with tables of 6016 tokens, 38 with
// 131072, and the output's last bits then come from the other kernel.
constexpr int64_t kFewWork = 12000000;
size_t few_workspace_bytes(int64_t D) {
  const size_t slot = static_cast<size_t>(16) * (static_cast<size_t>(D) + 2) * 4;  // NT = 2
  return (kMaxCtas * (sizeof(int4) + 2 * slot) + 255) / 256 * 256;
}
// Whether some sequence may have more than kFewRows rows, and a prompt kernel (not for head_dim 256).
bool may_prompt(int64_t T, int64_t G, int64_t D) { return T * G > kFewRows && kv4_prompt_fits(D); }
}  // namespace

size_t kv4_attn_workspace_bytes(int64_t T, int64_t D, int64_t G) {
  return few_workspace_bytes(D) + (may_prompt(T, G, D) ? kv4_prompt_workspace_bytes(D) : 0);
}

rnl_status launch_kv4_attention(const Kv4AttnArgs& x, const rnl_kv4_cache& c, const rnl_kv4_seqs& q,
                                cudaStream_t s) {
  g_launched.store(true, std::memory_order_relaxed);
  DeviceInfo dev;
  const rnl_status st = current_device(&dev);
  if (st != RNL_OK) return st;
  const Args a = make_args(c, q);
  AttnParams p;
  p.q = static_cast<const __nv_bfloat16*>(x.q);
  p.q_stride = x.q_stride;
  p.out = static_cast<__nv_bfloat16*>(x.out);
  p.lse = x.lse;
  p.rec = static_cast<int4*>(x.ws);
  p.part = reinterpret_cast<float*>(p.rec + kMaxCtas);
  p.scale_log2 = x.scale * 1.4426950408889634f;
  p.Hq = static_cast<int>(x.Hq);
  p.G = p.Hq / a.Hkv;
  p.causal = x.causal;
  p.window = x.window < (int64_t{1} << 30) ? static_cast<int>(x.window) : 0;  // lengths end at 2^30
  p.few = 0x7fffffff;
  bool after = false;
  const int64_t tokens = c.n_kv_heads * (q.max_pages * c.page_size);  // below 2^46
  if (q.cu_rows != nullptr && may_prompt(q.n_rows, p.G, a.D) && q.n_rows * p.G > kFewWork / std::max<int64_t>(tokens, 1)) {
    p.few = kFewRows;
    const rnl_status pst = launch_kv4_prompt(p, a, static_cast<int>(c.block),
                                             static_cast<char*>(x.ws) + few_workspace_bytes(a.D), dev, s);
    if (pst != RNL_OK) return pst;
    after = true;
  }
  // 4, 8 or 16 rows an item: the fewest that hold the rows a sequence has on average
  // (with 8 rows an item 131072 tokens x 8 take 267 us instead of 242; with 16, 32
  // sequences of 2 rows 91 instead of 66).  The rows of prompts count in that average, though the other
  // kernel takes them: 64 single tokens beside a prompt of 2048 rows get items of 16 rows (380 us, the
  // two alone 149 and 157)
  const int64_t rows = (q.n_rows + q.n_seqs - 1) / q.n_seqs * p.G;
  const bool mixed = a.cu != nullptr && p.causal;
  auto go = [&](auto d, auto bs) {
    constexpr int D = decltype(d)::value, BS = decltype(bs)::value;
    if (mixed)
      return rows <= 4   ? launch_split<D, 0, BS, true>(p, a, dev, after, s)
             : rows <= 8 ? launch_split<D, 1, BS, true>(p, a, dev, after, s)
                         : launch_split<D, 2, BS, true>(p, a, dev, after, s);
    return rows <= 4   ? launch_split<D, 0, BS, false>(p, a, dev, after, s)
           : rows <= 8 ? launch_split<D, 1, BS, false>(p, a, dev, after, s)
                       : launch_split<D, 2, BS, false>(p, a, dev, after, s);
  };
  auto by_block = [&](auto d) {
    return c.block == 64 ? go(d, std::integral_constant<int, 64>{}) : go(d, std::integral_constant<int, 32>{});
  };
  if (a.D == 64) return by_block(std::integral_constant<int, 64>{});
  if (a.D == 128) return by_block(std::integral_constant<int, 128>{});
  return by_block(std::integral_constant<int, 256>{});
}

rnl_status read_clear_error_kv4attn(unsigned int* word) {
  if (!g_launched.load(std::memory_order_relaxed)) return RNL_OK;
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_kv4attn, sizeof v) != cudaSuccess) return RNL_ERR_LAUNCH;
  if (v != 0 && cudaMemcpyToSymbol(g_err_kv4attn, &zero, sizeof zero) != cudaSuccess)
    return RNL_ERR_LAUNCH;
  *word = v;
  return RNL_OK;
}

}  // namespace rnl
