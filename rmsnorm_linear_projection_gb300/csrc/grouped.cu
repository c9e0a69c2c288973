// grouped.cu -- products grouped by expert with ragged sizes, of bf16 or of
// MXFP8 operands (E4M3 codes with an E8M0 scale per 32 or 64 elements):
//
//   out[i] = bf16(sum_k x[rows[i], k] W[e, :, k])        rows i of expert e
//   out[i] = bf16(silu(g) u),  g = the first half of W[e]'s rows, u the second    (swiglu)
//
// on CTA pairs (tcgen05.mma.cta_group::2): a unit is 256 weight rows (128 a
// CTA, the M side) against a tile of up to 256 rows of the group (the N side,
// half of them staged by each CTA), see grouped.cuh.  The rows named by `rows` are
// gathered while they are staged (16-byte asynchronous copies by four warps),
// so that no sorted copy of x is written; rows that stand in order come as TMA boxes.
// Measured against the copies: TMA gathers of four rows, issued by elected lanes of
// the four warps: MXFP8 32000 x 4096 -> 2 x 768 over 64 experts 162-165 against 168-170
// us, bf16 32768 x 2048 -> 2 x 1408 over 32 experts 228-234 against 219-227.  (Each warp
// must then have rows in every stage: one without any can fall a phase of `empty`
// behind.)  For swiglu the weight box interleaves 16 gate rows with the 16 up rows of
// the same features, which puts both sums of a feature into one warp's lanes.
//
// Measured: 4096 x 4096 -> 4864 with one expert 83-85 us, 1.92 PFLOP/s (bound by
// the tensor pipe), gathered 87-89; MXFP8 4032 x 8192 -> 4864 94 us, 3.41 PFLOP/s,
// gathered 106 (by L2 -> SM copies: 30 KB a k-block); 32768 x 2048 -> 2 x 1408 over 32
// experts 219-233 us, 259-274 once the power limit holds; 64 rows over 34 experts of
// the same size 62-64 us (HBM, 6.2 TB/s).
//
// Roles per CTA (480 threads): warp 0 weight boxes (TMA), warp 1 MMA issue (even CTA),
// warps 2-9 epilogue, warps 10-13 gathers, warp 14 their hand-over, or the boxes of
// rows that stand in order; MXFP8 (608 threads) warps 15-18 the scales into tensor
// memory.
// Every wait is bounded (ptx.cuh).
#include <cuda_bf16.h>

#include <atomic>

#include "grouped.cuh"
#include "internal.h"

namespace rnl {
namespace {

using namespace gemm;
using namespace grouped;

__device__ unsigned int g_err_grouped;
std::atomic<bool> g_launched{false};

constexpr int kRowBytes = 128;                    // of a k-block: 64 bf16 or 128 codes
constexpr int kStep = 32;                         // the pair's products take N in steps of 32
constexpr int kGatherWarps = 4;                   // 32 of the CTA's rows each
constexpr int kRelayWarp = 2 + kEpiWarps + kGatherWarps;
constexpr int kScaleWarps = 4;                    // one a TMEM lane quarter
constexpr int64_t kSlotWords = 2 * 128 * 256;     // partial sums of one pair: [CTA][column][lane]
constexpr int kMaxPairs = kMaxPartialSlots - 1;   // the last slot holds the flags

// Scales go through shared memory four k-blocks at a time, a row's bytes of them
// (16, or 8 with 64 elements a scale) after the other: 128 weight rows, then 224
// rows of x.
constexpr int kSfBatch = 4;
constexpr int kSfRows = 11 * 32;

// MX: two accumulators of 224 columns leave 64 columns of TMEM for the scales of
// four k-blocks, two slots of an even and an odd one (of 16 columns each: weight
// rows' at +0, the group's at +8).
template <bool MX>
struct Form {
  static constexpr int kTile = MX ? 224 : 256;  // rows of a group a tile, at most
  static constexpr int kThreads = (kRelayWarp + 1 + (MX ? kScaleWarps : 0)) * 32;
  static constexpr uint32_t kStageBytes = kABytes + kTile / 2 * kRowBytes;
  static constexpr size_t kSfBytes = MX ? 2 * kSfRows * 16 : 0;
  static constexpr uint32_t kSfBase = 2 * kTile;
  static constexpr int kSfSlots = 2;
  static_assert(kStageBytes % 1024 == 0, "swizzle atoms");
  static_assert(!MX || kSfBase + kSfSlots * 32 <= 512, "TMEM columns");
};

// x as boxes of 128, 64, 32 and 16 rows (rows that stand in order)
struct XMaps {
  CUtensorMap m[4];
};

struct __align__(16) Ctrl {
  uint64_t full[kMaxStages];   // even CTA: both CTAs' loads of a stage
  uint64_t empty[kMaxStages];  // each CTA: its stage read by the pair's MMAs
  uint64_t landed[kMaxStages];  // each CTA: its gathered rows of a stage
  uint64_t tmem_full[2];       // each CTA: accumulator ready
  uint64_t tmem_empty[2];      // even CTA: both CTAs' epilogues have read it
  uint64_t sf_full[2];         // even CTA: both CTAs' scales of a slot are in TMEM
  uint64_t sf_empty[2];        // each CTA: the slot's k-blocks have been multiplied
  uint32_t tmem_base;
  int abort;
  Plan plan;
};

__host__ __device__ constexpr size_t table_bytes(int E) { return (static_cast<size_t>(E) + 1) * 8; }

struct Args {
  const uint8_t* x;
  int64_t row_bytes;    // of x and W
  const uint8_t* x_scale;
  const uint8_t* w_scale;
  int nb;               // scale bytes a row
  int sf_vec;           // bytes a load of scales: what the rows' alignment allows (a batch's 16 or 8, 4 or 1)
  const int32_t* offsets;
  const int32_t* rows;  // may be null
  int R;                // rows of x
  int M;                // rows of out
  int E, N;             // N weight rows an expert
  int num_kb;
  int stages;
  __nv_bfloat16* out;
  float* partial;
  uint64_t* flags;
  uint64_t epoch;
};

template <int BLK>
struct Sf {
  static constexpr int kRowBytes = kSfBatch * 128 / BLK;  // scales of a row and batch: 16 or 8
  static constexpr int kRowWords = kRowBytes / 4;
};

// The scale bytes of four k-blocks from kb on of one row (127 behind its last).  vec:
// bytes a load, what the rows' alignment allows: the whole batch, words, or single
// bytes put together.  From L2: the kernel before may have written the scales, which
// closes the read-only path, and plain loads, held between the barriers around them,
// took 24008 x 768 -> 4096 over 128 experts from 124 to 132 us (these 125.5).  The
// addresses come from the plan that is made behind the wait for that kernel.
template <int BLK>
__device__ __forceinline__ void load_scales(const uint8_t* p, int kb, int nb, int vec,
                                            uint32_t (&w)[Sf<BLK>::kRowWords]) {
  constexpr int kBytes = Sf<BLK>::kRowBytes, kWords = Sf<BLK>::kRowWords;
  const int b0 = kb / kSfBatch * kBytes;
  const uint8_t* q = p + b0;
  if (vec == kBytes && b0 + kBytes <= nb) {
    if constexpr (kWords == 4) {
      const uint4 u = __ldcg(reinterpret_cast<const uint4*>(q));
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
      const uint2 u = __ldcg(reinterpret_cast<const uint2*>(q));
      w[0] = u.x, w[1] = u.y;
    }
  } else if (vec >= 4) {
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      w[i] = b0 + 4 * i < nb ? __ldcg(reinterpret_cast<const uint32_t*>(q) + i) : 0x7F7F7F7Fu;
  } else {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      uint32_t v = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v |= static_cast<uint32_t>(b0 + 4 * i + j < nb ? __ldcg(q + 4 * i + j) : 127) << (8 * j);
      w[i] = v;
    }
  }
}

// What load_scales has loaded of a row, into shared memory.
template <int BLK>
__device__ __forceinline__ void put_scales(uint8_t* dst, const uint32_t (&w)[Sf<BLK>::kRowWords]) {
  if constexpr (BLK == 32)
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}

// The scale words of two k-blocks of a row (its bytes in shared memory at p): a byte
// for each 32-element block of the hardware, a 64-element scale given to it twice.
template <int BLK>
__device__ __forceinline__ void take_scales(const uint8_t* p, uint32_t& even, uint32_t& odd) {
  if constexpr (BLK == 32) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    even = u.x;
    odd = u.y;
  } else {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    even = __byte_perm(u, 0, 0x1100);
    odd = __byte_perm(u, 0, 0x3322);
  }
}

// BLK: 0 for bf16, 32 or 64 for MXFP8 operands with that many elements a scale.
template <bool SWIGLU, int BLK>
__global__ void __launch_bounds__(Form<BLK != 0>::kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ XMaps maps_x, const Args a) {
  constexpr bool MX = BLK != 0;
  using F = Form<MX>;
  constexpr int kTile = F::kTile;
  constexpr uint32_t kStageBytes = F::kStageBytes;
  constexpr int kBKElems = MX ? kRowBytes : kRowBytes / 2;
  constexpr int kFeatCta = SWIGLU ? 64 : 128;  // output features a CTA
  constexpr uint32_t kTmemCols = 512;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_addr);
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + a.stages * kStageBytes);
  uint32_t* sf_smem = reinterpret_cast<uint32_t*>(ctrl + 1);  // two batches of scales
  int* off = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(sf_smem) + F::kSfBytes);
  int* pre = off + a.E + 1;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // uniform to the compiler
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1;
  const int num_pairs = gridDim.x >> 1;
  const int N_out = SWIGLU ? a.N / 2 : a.N;
  const int num_f = (N_out + 2 * kFeatCta - 1) / (2 * kFeatCta);
  // rows that stand in order come as TMA boxes (900 rows x 32 experts, 1408 -> 2048 in
  // bf16: 111 against 117 us by the gathering warps; MXFP8 4032 x 8192 -> 4864 94
  // against 106)
  const bool gather = a.rows != nullptr;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(smem_u32(&ctrl->full[s]), gather ? 3 : 1);  // the boxes' bytes, and each CTA's gathered rows
      mbar_init(smem_u32(&ctrl->landed[s]), kGatherWarps * 32);
      mbar_init(smem_u32(&ctrl->empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&ctrl->tmem_full[b]), 1);
      mbar_init(smem_u32(&ctrl->tmem_empty[b]), 2 * kEpiWarps);
    }
    for (int b = 0; b < F::kSfSlots; ++b) {
      mbar_init(smem_u32(&ctrl->sf_full[b]), 2 * kScaleWarps);
      mbar_init(smem_u32(&ctrl->sf_empty[b]), 1);
    }
    ctrl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&ctrl->tmem_base), kTmemCols);
    tmem_relinquish_pair();
  }
  grid_launch_dependents();
  grid_dependency_wait();
  build_groups(a.offsets, a.E, a.M, num_f, kTile, off, pre, &g_err_grouped, 213);
  const Groups groups{off, pre, a.E, num_f};
  if (warp == 0) make_plan<kTile, kStep>(ctrl->plan, groups, num_pairs, a.num_kb, pair, lane);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = ctrl->tmem_base;
  volatile int* abort = &ctrl->abort;
  Walk<kTile, kStep> walk(ctrl->plan, groups, lane);

  if (warp == 0) {
    // ------------------------------------------------------- weight producer
    if (lane == 0) tma_prefetch_map(&map_w);
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int it = 0; it < walk.n && ok; ++it) {
      const Item w = walk.at(it);
      const int f0 = (w.t.f * 2 + static_cast<int>(rank)) * kFeatCta;
      const uint32_t bytes = 2 * kABytes + (gather ? 0u : static_cast<uint32_t>(w.t.n) * kRowBytes);  // of both CTAs
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        ok = mbar_wait(smem_u32(&ctrl->empty[stage]), phase ^ 1u, abort, &g_err_grouped, 205) &&
             RNL_DCHECK(&g_err_grouped, stage < static_cast<uint32_t>(a.stages), 206);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t sa = base + stage * kStageBytes;
        const uint32_t full_local = smem_u32(&ctrl->full[stage]);
        const uint32_t full_even = mapa_shared(full_local, 0);
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(full_local, bytes);
          if constexpr (SWIGLU)
            tma_load_5d_pair(sa, &map_w, full_even, kb * kBKElems, 0, 0, f0 / 16, w.t.e);
          else
            tma_load_2d_pair(sa, &map_w, full_even, kb * kBKElems, w.t.e * a.N + f0);
        }
        __syncwarp();
        if (++stage == static_cast<uint32_t>(a.stages)) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == kRelayWarp && !gather) {
    // -------------------------------------------------------- row producer
    // rows that stand in order: as boxes of 128 to 16 rows.  (A warp of its own, and an
    // elected lane of it: from lane 0 of the weight's warp MXFP8 4032 x 8192 -> 4864 took
    // 122 us, from lane 0 of this one 109)
    if (lane == 0) tma_prefetch_map(&maps_x.m[0]);
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int it = 0; it < walk.n && ok; ++it) {
      const Item w = walk.at(it);
      const int half = w.t.n / 2;
      const int x_row = w.t.row0 + static_cast<int>(rank) * half;
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        ok = __all_sync(0xffffffffu,
                        mbar_wait(smem_u32(&ctrl->empty[stage]), phase ^ 1u, abort, &g_err_grouped, 215));
        if (!ok) break;
        const uint32_t dst = base + stage * kStageBytes + kABytes;
        const uint32_t full_even = mapa_shared(smem_u32(&ctrl->full[stage]), 0);
        if (elect_one()) {
          int at = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (half & (128 >> b)) {
              tma_load_2d_pair(dst + at * kRowBytes, &maps_x.m[b], full_even, kb * kBKElems, x_row + at);
              at += 128 >> b;
            }
        }
        __syncwarp();
        if (++stage == static_cast<uint32_t>(a.stages)) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp == kRelayWarp) {
    // --------------------------------------------------------------- relay
    // hands a stage's rows to the tensor cores.  Not by the warps that copy:
    // their fence would wait for every copy that they have in flight
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int it = 0; it < walk.n && ok; ++it) {
      const Item w = walk.at(it);
      if (lane == 0) {
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!mbar_wait(smem_u32(&ctrl->landed[stage]), phase, abort, &g_err_grouped, 202)) {
            ok = false;
            break;
          }
          fence_proxy_async_shared();
          const uint32_t full_local = smem_u32(&ctrl->full[stage]);
          if (rank == 0)
            mbar_arrive(full_local);
          else
            mbar_arrive_remote(mapa_shared(full_local, 0));
          if (++stage == static_cast<uint32_t>(a.stages)) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
  } else if (MX && warp > kRelayWarp) {
    // ------------------------------------------------------- scale writers
    // four k-blocks at a time: the 128 threads load the scales of the CTA's weight
    // rows and of all the tile's rows (three rows a thread) and put them into shared
    // memory; each warp then writes the words of two k-blocks into its lane quarter
    // of a TMEM slot, once what the slot held has been multiplied.  A chain of
    // 0.19 us a k-block (one word at a time through shared memory 0.27), against 0.25
    // that the products take
    if constexpr (MX) {
      const int quarter = warp & 3;
      const int me = (warp - kRelayWarp - 1) * 32 + lane;
      const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
      uint32_t slot = 0, phase = 0;
      bool ok = true;
      // Scales are loaded two batches ahead, across items (one batch ahead, a batch
      // took as long as its loads, 1.1 us), and the rows of the group are looked up an
      // item ahead.  What is being loaded: batch `kb` of item `it`, rows me (weight),
      // me and me + 128 (group).
      int it = 0, kb = 0, next_row[2];
      const uint8_t* p[3];
      Item w, next;
      auto look_up = [&]() {  // the next item and its rows
        next = walk.at(it + 1 < walk.n ? it + 1 : it);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = next.t.row0 + min(me + 128 * h, next.t.valid - 1);
          next_row[h] = a.rows != nullptr ? a.rows[i] : i;
        }
      };
      auto enter = [&]() {  // makes the next item the one in hand
        w = next;
        kb = w.kb0 & ~(kSfBatch - 1);
        const int f0 = (w.t.f * 2 + static_cast<int>(rank)) * kFeatCta;
        // rows that are none take another's scale, their products are not stored
        int n;
        if (SWIGLU)  // TMEM lane 32 q + 16 h + i: feature 16 q + i, gate (h = 0) or up
          n = min(f0 + (me >> 5) * 16 + (me & 15), N_out - 1) + ((me & 16) ? N_out : 0);
        else
          n = min(f0 + me, a.N - 1);
        p[0] = a.w_scale + (static_cast<int64_t>(w.t.e) * a.N + n) * a.nb;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = next_row[h];  // (the gathers report one that is out of range)
          p[1 + h] = a.x_scale + static_cast<int64_t>(r >= 0 && r < a.R ? r : 0) * a.nb;
        }
        look_up();
      };
      // a batch: its scales, its first k-block and the range of them that is multiplied
      struct Batch {
        uint32_t v[3][Sf<BLK>::kRowWords];
        int kb, lo, hi;  // hi 0: none
      };
      auto load = [&](Batch& b) {
        b.hi = 0;
        if (it >= walk.n) return;
#pragma unroll
        for (int h = 0; h < 3; ++h) load_scales<BLK>(p[h], kb, a.nb, a.sf_vec, b.v[h]);
        b.kb = kb;
        b.lo = w.kb0;
        b.hi = w.kb1;
        kb += kSfBatch;
        if (kb >= w.kb1 && ++it < walk.n) enter();
      };
      constexpr int kRowScale = Sf<BLK>::kRowBytes;
      auto write = [&](Batch& b, uint8_t* sf) {
        put_scales<BLK>(sf + me * kRowScale, b.v[0]);
        put_scales<BLK>(sf + (128 + me) * kRowScale, b.v[1]);
        if (me < 96) put_scales<BLK>(sf + (256 + me) * kRowScale, b.v[2]);
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const int first = b.kb, lo = b.lo, hi = b.hi;
        load(b);
#pragma unroll
        for (int k = 0; k < kSfBatch; k += 2) {  // a slot: two k-blocks
          // (a warp that gives up on a slot still takes part in the barriers)
          if (!ok || first + k + 2 <= lo || first + k >= hi) continue;
          uint32_t even[16], odd[16];  // columns: weight rows' words at 0, the group's at 8
          const uint8_t* q = sf + lane * kRowScale + k * (kRowScale / kSfBatch);
#pragma unroll
          for (int j = 0; j < 11; ++j)
            take_scales<BLK>(q + j * 32 * kRowScale, even[j < 4 ? j : j + 4], odd[j < 4 ? j : j + 4]);
#pragma unroll
          for (int j = 4; j < 8; ++j) even[j] = odd[j] = 0u;
          even[15] = odd[15] = 0u;
          const bool got = mbar_wait(smem_u32(&ctrl->sf_empty[slot]), phase ^ 1u, abort, &g_err_grouped, 200);
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            continue;
          }
          tc_fence_after();
          const uint32_t col = tmem_base + lane_addr + F::kSfBase + slot * 32;
          tmem_st_16cols(col, even);
          tmem_st_16cols(col + 16, odd);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            const uint32_t bar = smem_u32(&ctrl->sf_full[slot]);
            if (rank == 0)
              mbar_arrive(bar);
            else
              mbar_arrive_remote(mapa_shared(bar, 0));
          }
          if (++slot == F::kSfSlots) {
            slot = 0;
            phase ^= 1u;
          }
        }
      };
      if (walk.n > 0) {
        it = -1;
        look_up();
        it = 0;
        enter();
        Batch b0, b1;
        load(b0);
        load(b1);
        while (b0.hi > 0) {
          write(b0, reinterpret_cast<uint8_t*>(sf_smem));
          if (b1.hi == 0) break;
          write(b1, reinterpret_cast<uint8_t*>(sf_smem) + kSfRows * 16);
        }
      }
    }
  } else if (warp >= 2 + kEpiWarps) {
    // ------------------------------------------------------------- gathers
    // each warp brings 32 of the CTA's rows, 16 bytes a lane and copy, to where a
    // TMA load with the 128-byte swizzle would put them
    const int gw = warp - (2 + kEpiWarps);
    const int sub = lane >> 3, chunk = lane & 7;
    uint32_t stage = 0, phase = 0;
    bool ok = gather;
    Item w, next;
    int row[8];  // of the next item
    auto look_up = [&](const Item& i) {
      const int first = static_cast<int>(rank) * (i.t.n / 2) + gw * 32 + sub;
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // rows behind the tile's last one repeat it (their columns are not stored)
        row[j] = a.rows[i.t.row0 + min(first + 4 * j, i.t.valid - 1)];
      }
    };
    if (ok && walk.n > 0) {
      next = walk.at(0);
      look_up(next);
    }
    for (int it = 0; it < walk.n && ok; ++it) {
      w = next;
      const int half = w.t.n / 2;
      const uint8_t* src[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (row[i] < 0 || row[i] >= a.R) {
          atomicCAS(&g_err_grouped, 0u, kErrArg | (204u << 8));
          row[i] = 0;
        }
        src[i] = a.x + row[i] * a.row_bytes + chunk * 16;
      }
      if (it + 1 < walk.n) {
        next = walk.at(it + 1);
        look_up(next);
      }
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        const bool got = mbar_wait(smem_u32(&ctrl->empty[stage]), phase ^ 1u, abort, &g_err_grouped, 212);
        if (!__all_sync(0xffffffffu, got && RNL_DCHECK(&g_err_grouped, half <= kTile / 2, 203))) {
          ok = false;
          break;
        }
        const uint32_t dst = base + stage * kStageBytes + kABytes + (gw * 32 + sub) * 128;
        const int k0 = kb * kRowBytes;
        const uint32_t bytes = k0 + chunk * 16 < a.row_bytes ? 16u : 0u;
        const int from = bytes ? k0 : -chunk * 16;  // an address inside the row where nothing is read
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (gw * 32 + 4 * i < half)  // (row & 7) = sub + 4 (i & 1)
            cp_async_16(dst + i * 512 + ((chunk ^ (sub + 4 * (i & 1))) << 4), src[i] + from, bytes);
        cp_async_arrive(smem_u32(&ctrl->landed[stage]));
        if (++stage == static_cast<uint32_t>(a.stages)) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    cp_async_wait_all();  // nothing in flight when the warp leaves
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue
    if (rank == 0) {
      uint32_t stage = 0, phase = 0, slot = 0, sf_phase = 0;
      bool ok = true;
      Item next = walk.at(0);
      for (int it = 0; it < walk.n && ok; ++it) {
        const Item w = next;
        const uint32_t buf = it & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&ctrl->tmem_empty[buf]), ((it >> 1) & 1) ^ 1u, abort,
                                               &g_err_grouped, 207));
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + buf * kTile;
        const uint32_t idesc = MX ? idesc_mxf8(256, w.t.n) : idesc_bf16(256, w.t.n);
        for (int kb = w.kb0; kb < w.kb1 && ok; ++kb) {
          // (MX: a slot of scales holds an even and the next odd k-block)
          const bool sf_new = MX && ((kb & 1) == 0 || kb == w.kb0);
          ok = mbar_wait(smem_u32(&ctrl->full[stage]), phase, abort, &g_err_grouped, 208) &&
               (!sf_new || mbar_wait(smem_u32(&ctrl->sf_full[slot]), sf_phase, abort, &g_err_grouped, 201));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sa = base + stage * kStageBytes;
          const uint64_t adesc = desc_kmajor_sw128(sa);
          const uint64_t bdesc = desc_kmajor_sw128(sa + kABytes);
          const uint32_t sf = tmem_base + F::kSfBase + slot * 32 + (kb & 1) * 16;
          const bool sf_done = MX && ((kb & 1) != 0 || kb + 1 == w.kb1);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // 32 bytes of a row each
              const uint32_t add = (kb > w.kb0 || k > 0) ? 1u : 0u;
              if constexpr (MX)
                umma_mxf8_pair(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc_mxf8_id(idesc, k), sf, sf + 8, add);
              else
                umma_bf16_pair(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, add);
            }
            umma_commit_pair(smem_u32(&ctrl->empty[stage]), 0x3);
            if (sf_done) umma_commit_pair(smem_u32(&ctrl->sf_empty[slot]), 0x3);
            if (kb + 1 == w.kb1) umma_commit_pair(smem_u32(&ctrl->tmem_full[buf]), 0x3);
          }
          __syncwarp();
          if (kb == w.kb0 && it + 1 < walk.n) next = walk.at(it + 1);  // while the products run
          if (sf_done && ++slot == F::kSfSlots) {
            slot = 0;
            sf_phase ^= 1u;
          }
          if (++stage == static_cast<uint32_t>(a.stages)) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int ew = warp - 2;
    const int quarter = warp & 3;  // TMEM lanes this warp may access
    const int half = ew >> 2;      // takes every other 32-column group
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t empty_even[2] = {mapa_shared(smem_u32(&ctrl->tmem_empty[0]), 0),
                                    mapa_shared(smem_u32(&ctrl->tmem_empty[1]), 0)};
    const int64_t lane_off = static_cast<int64_t>(rank) * 128 * 256 + quarter * 32 + lane;
    int it = 0;
    for (; it < walk.n; ++it) {
      const Item w = walk.at(it);
      const Tile& t = w.t;
      const uint32_t buf = it & 1;
      bool got = mbar_wait(smem_u32(&ctrl->tmem_full[buf]), (it >> 1) & 1, abort, &g_err_grouped, 209);
      if (w.kind == kFinish)  // a flag a lane
        for (int q = w.first + lane; q < pair && got; q += 32)
          got = flag_wait(a.flags + (static_cast<int64_t>(q) * 2 + rank) * kEpiWarps + ew, a.epoch, abort,
                          &g_err_grouped, 210);
      if (!__all_sync(0xffffffffu, got)) break;
      __syncwarp();  // what a lane acquired is every lane's
      tc_fence_after();
      const int f0 = (t.f * 2 + static_cast<int>(rank)) * kFeatCta;
      const int feat = SWIGLU ? f0 + quarter * 16 + (lane & 15) : f0 + quarter * 32 + lane;
      for (int c = half * 32; c < t.n; c += 64) {
        uint32_t r[32];
        tmem_ld_32cols(tmem_base + lane_addr + buf * kTile + c, r);
        tmem_ld_wait();
        if (!RNL_DCHECK(&g_err_grouped, c + 32 <= kTile && t.row0 + t.valid <= a.M && pair < kMaxPairs, 211)) continue;
        if (w.kind == kPartial) {
          float* dst = a.partial + pair * kSlotWords + lane_off + static_cast<int64_t>(c) * 128;
#pragma unroll
          for (int j = 0; j < 32; ++j) dst[j * 128] = __uint_as_float(r[j]);
          continue;
        }
        if (w.first < pair) {  // the lower workers' parts, in their order; half a part's loads ahead
          const float* src = a.partial + w.first * kSlotWords + lane_off + static_cast<int64_t>(c) * 128;
          float lo[16], hi[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) lo[j] = __ldcg(src + j * 128);
          for (int q = w.first; q < pair; ++q, src += kSlotWords) {
#pragma unroll
            for (int j = 0; j < 16; ++j) hi[j] = __ldcg(src + (16 + j) * 128);
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + lo[j]);
            if (q + 1 < pair) {
#pragma unroll
              for (int j = 0; j < 16; ++j) lo[j] = __ldcg(src + kSlotWords + j * 128);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) r[16 + j] = __float_as_uint(__uint_as_float(r[16 + j]) + hi[j]);
          }
        }
        if constexpr (SWIGLU)
          store_cols_swiglu(a.out, N_out, t.row0, t.valid, c, feat, lane, r);
        else
          store_cols(a.out, N_out, t.row0, t.valid, c, feat, lane, r);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0)
          mbar_arrive(smem_u32(&ctrl->tmem_empty[buf]));
        else
          mbar_arrive_remote(empty_even[buf]);  // (what it orders are reads of TMEM)
      }
      // a flag is consumed by one warp, which sets it back, so that a replayed
      // graph waits for its own
      for (int q = w.first + lane; q < pair; q += 32) a.flags[(static_cast<int64_t>(q) * 2 + rank) * kEpiWarps + ew] = 0;
      if (w.kind == kPartial) {
        __threadfence();
        __syncwarp();
        if (lane == 0)
          join_visit(a.flags + (static_cast<int64_t>(pair) * 2 + rank) * kEpiWarps + ew, a.epoch, a.epoch);
      }
    }
    if (it < walk.n)  // a wait has run out
      give_up_joins<kTile, kStep>(ctrl->plan, groups, it, lane, a.flags + rank * kEpiWarps + ew, 2 * kEpiWarps, a.epoch);
  }

  // a CTA that gave up on a wait lets the copies and products in flight end
  if (*abort) {
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 100000ull) __nanosleep(1000);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// CTA pairs that are resident at once (all of the grid is).
template <bool SWIGLU, int BLK>
int resident_pairs(const DeviceInfo& dev, size_t smem) {
  static std::atomic<int> cached[64];
  const int c = cached[dev.device].load(std::memory_order_relaxed);
  if (c > 0) return c;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (dev.sm_count / 2), 1, 1);
  cfg.blockDim = dim3(Form<BLK != 0>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, grouped_kernel<SWIGLU, BLK>, &cfg) != cudaSuccess) n = 0;
  cudaGetLastError();
  if (n <= 0 || n > dev.sm_count / 2) n = dev.sm_count / 2;
  if (n > kMaxPairs) n = kMaxPairs;
  cached[dev.device].store(n, std::memory_order_relaxed);
  return n;
}

template <bool SWIGLU, int BLK>
rnl_status launch(const GroupedArgs& g, const DeviceInfo& dev, cudaStream_t s) {
  constexpr bool MX = BLK != 0;
  using F = Form<MX>;
  auto kern = grouped_kernel<SWIGLU, BLK>;
  const size_t fixed = 1024 + sizeof(Ctrl) + F::kSfBytes + table_bytes(static_cast<int>(g.E));
  const size_t fit = (kSmemLimit - fixed) / F::kStageBytes;
  const int stages = static_cast<int>(fit < static_cast<size_t>(kMaxStages) ? fit : kMaxStages);
  const size_t smem = fixed + stages * F::kStageBytes;
  if (ensure_smem_attr(reinterpret_cast<const void*>(kern), dev.device, kSmemLimit) != RNL_OK) return RNL_ERR_LAUNCH;
  CUtensorMap mw;
  const uint64_t N = g.N, K = g.K, row = MX ? K : 2 * K;
  constexpr uint32_t kBox = MX ? kRowBytes : kRowBytes / 2;
  const CUtensorMapDataType dt = MX ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  rnl_status st;
  if (SWIGLU) {
    // [expert][16 features][gate / up][feature][k]: 64 features' gate and up rows in groups of 16
    const uint64_t dims[5] = {K, 16, 2, N / 32, static_cast<uint64_t>(g.E)};
    const uint64_t strides[4] = {row, N / 2 * row, 16 * row, N * row};
    const uint32_t box[5] = {kBox, 16, 2, 4, 1};
    st = make_map_5d(&mw, dt, g.w, dims, strides, box);
  } else {
    st = make_map_2d(&mw, dt, g.w, K, g.E * N, row, kBox, 128);
  }
  if (st != RNL_OK) return st;
  XMaps mx = {};  // (gathered rows take no boxes)
  for (int b = 0; b < 4 && g.rows == nullptr; ++b) {
    st = make_map_2d(&mx.m[b], dt, g.x, K, g.R, row, kBox, 128 >> b);
    if (st != RNL_OK) return st;
  }
  Args a;
  a.x = static_cast<const uint8_t*>(g.x);
  a.row_bytes = static_cast<int64_t>(row);
  a.x_scale = g.x_scale;
  a.w_scale = g.w_scale;
  a.nb = MX ? static_cast<int>(g.K / g.block) : 0;
  a.sf_vec = 1;
  if constexpr (MX) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(g.x_scale) | reinterpret_cast<uintptr_t>(g.w_scale) |
                           static_cast<uintptr_t>(a.nb);
    a.sf_vec = bits % Sf<BLK>::kRowBytes == 0 ? Sf<BLK>::kRowBytes : (bits % 4 == 0 ? 4 : 1);
  }
  a.offsets = g.offsets;
  a.rows = g.rows;
  a.R = static_cast<int>(g.R);
  a.M = static_cast<int>(g.M);
  a.E = static_cast<int>(g.E);
  a.N = static_cast<int>(g.N);
  a.num_kb = static_cast<int>((row + kRowBytes - 1) / kRowBytes);
  a.stages = stages;
  a.out = static_cast<__nv_bfloat16*>(g.out);
  a.partial = static_cast<float*>(g.ws);
  a.flags = reinterpret_cast<uint64_t*>(a.partial + kMaxPairs * kSlotWords);
  a.epoch = next_flag_epoch();
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * static_cast<unsigned>(resident_pairs<SWIGLU, BLK>(dev, smem)), 1, 1);
  cfg.blockDim = dim3(F::kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  trace_before(s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mw, mx, a);
  trace_after(s, MX ? (SWIGLU ? "grouped_mxfp8_swiglu" : "grouped_mxfp8")
                    : (SWIGLU ? "grouped_bf16_swiglu" : "grouped_bf16"));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return RNL_ERR_LAUNCH;
  }
  return RNL_OK;
}

}  // namespace

rnl_status launch_grouped(const GroupedArgs& g, cudaStream_t s) {
  if (g.M == 0) return RNL_OK;
  DeviceInfo dev;
  const rnl_status st = current_device(&dev);
  if (st != RNL_OK) return st;
  g_launched.store(true, std::memory_order_relaxed);
  if (g.block == 0) return g.swiglu ? launch<true, 0>(g, dev, s) : launch<false, 0>(g, dev, s);
  if (g.block == 32) return g.swiglu ? launch<true, 32>(g, dev, s) : launch<false, 32>(g, dev, s);
  return g.swiglu ? launch<true, 64>(g, dev, s) : launch<false, 64>(g, dev, s);
}

rnl_status read_clear_error_grouped(unsigned int* word) {
  if (!g_launched.load(std::memory_order_relaxed)) return RNL_OK;
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_err_grouped, sizeof v) != cudaSuccess) return RNL_ERR_LAUNCH;
  if (v != 0 && cudaMemcpyToSymbol(g_err_grouped, &zero, sizeof zero) != cudaSuccess) return RNL_ERR_LAUNCH;
  *word = v;
  return RNL_OK;
}

}  // namespace rnl
