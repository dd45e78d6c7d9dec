// Tensor-core attention of a step (tcgen05): all rows of the batch over the
// shared prefix, and the new rows of longer sequences over their own keys.
//
// Over the prefix every row of the batch sees the same keys, so for one KV
// head the rows of all sequences and the heads of the group form one matrix
// of packed rows (token-major: row = token * g + head): Q K^T and P V are
// plain products of 128-row query tiles.  A sequence whose own packed rows
// exceed the streaming kernel's 16 is cut the same way over its own keys, with
// a causal limit per row.  A unit is a query tile of one KV head; its 128-key
// tiles are steps of the line that rbkv_step.h cuts evenly over one CTA per
// SM, so every CTA walks the same number of steps whatever the shapes.
//
// The streaming kernel's memory traffic runs beside this kernel's tensor work
// on the same SM, so this one keeps to 129 KB of shared memory and half of the
// registers.  Roles:
//  - warp 4 (TMA): streams 128-key K and V tiles through a 4-stage ring of
//    32 KB (128-byte swizzle), in the order K0 K1 V0 K2 V1 K3 ...; lane i
//    copies box i of a tile (one block, or 128 keys of a larger one);
//  - warp 5 (MMA): one elected lane issues S = Q K^T (M=128, N=128 keys,
//    K=128; Q from tensor memory) into one of two score buffers and
//    O += P V (P from tensor memory), in the order QK(0) QK(1), then per key
//    tile j: PV(j) QK(j+2).  The next tile's scores are so computed under the
//    softmax of the current one;
//  - warps 0-3 (softmax): thread i owns packed row i = TMEM lane i.  It writes
//    its row of Q into tensor memory (two Q buffers: the next unit's is
//    written while the current one's last products run), keeps a running max
//    that is raised only when the row max grows by more than 2^8 (the
//    accumulator in tensor memory is then rescaled in place), writes P as bf16
//    pairs over the score columns it has read, and at the end of a segment
//    stores the normalised partial output and its log-sum-exp (or O, when
//    nothing is to be joined).
// Tensor memory (512 columns x 128 lanes): scores 0 [0,128), scores 1
// [128,256), O [256,384), Q 0 [384,448), Q 1 [448,512).  Registers move from
// the second warpgroup to the first (setmaxnreg).
// Every wait is bounded; on timeout the kernel records RBKV_ERR_TIMEOUT, lets
// its copies and MMAs drain (bounded), frees its tensor memory and returns.
#include <algorithm>
#include <atomic>

#include "rbkv_step.h"
#include "rbkv_ptx.cuh"
#include "rbkv_tcgen05.cuh"

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace rbkv {

namespace {

using namespace tc;

constexpr int kRows = kStepTileRows;        // 128 query rows (MMA M)
constexpr int kKeys = kStepTileKeys;        // 128 keys per KV tile (MMA N of QK^T)
constexpr int kStages = 4;                  // ring stages, each one K or one V tile
constexpr int kHalf = kKeys * 128;          // 16 KB: 128 rows x 64 head dims
constexpr int kTileBytes = 2 * kHalf;       // 32 KB: 128 rows x 128 head dims
constexpr int kProducerWarp = 4;
constexpr int kMmaWarp = 5;
// Two warpgroups: the softmax warps, and one with the TMA and MMA warps (its
// other two warps idle).  Launched at kLaunchRegs a thread, the second gives
// back down to kIssueRegs and the first takes kSoftmaxRegs: the shares add up
// to the launch's total (a larger claim would wait forever), and the launch's
// total leaves half of an SM's registers to a streaming CTA.
constexpr int kThreads = 256;
constexpr int kLaunchRegs = 128;
constexpr int kIssueRegs = 48;
constexpr int kSoftmaxRegs = 208;
static_assert(128 * kIssueRegs + 128 * kSoftmaxRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch's registers");
constexpr int kTmemCols = 512;
constexpr int kOCol = 256;
constexpr int kQCol = 384;                  // two buffers of 64 columns
constexpr long long kWaitLimit = 4000000000LL;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;   // log2 units

// Each barrier is waited on in order of its phases and can never run two
// phases ahead of a waiter (the parity of a wait is then unambiguous).
struct Bars {
  uint64_t q_full[2];             // Q of a unit in tensor memory, by buffer
  uint64_t kv_full[kStages];      // a K or V tile landed (TMA)
  uint64_t kv_empty[kStages];     // the MMAs are done with the stage
  uint64_t s_full[2];             // QK^T of a key tile done, by score buffer
  uint64_t p_full[2];             // its P written (and V tail rows zeroed)
  uint64_t o_done[2];             // its PV done
  uint64_t o_free;                // a unit's O read: the next unit may overwrite it
  uint64_t drain;                 // every MMA the CTA issued done
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(kStages * kTileBytes + (int)sizeof(Bars) <= kStepTileSmem,
              "shared-memory layout overflows its allocation");

// Ring index, from the unit's first, of K_j and V_j of a segment of n tiles.
__device__ __forceinline__ uint32_t ring_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ uint32_t ring_v(int j, int n) {
  return j + 1 < n ? 2 * j + 2 : 2 * n - 1;
}

// One segment of a unit as every role sees it.
struct Item {
  const int32_t* table;
  int kv_head;
  int row, n_tok;  // first row and tokens of the query tile
  int pos;         // last key its first token sees (the prefix: every token)
  int kb, ke;      // key range of the segment
  int n;           // its key tiles
  bool prefix, head, whole;
};

// Walks a CTA's part [x, end) of the line.
struct Walk {
  int64_t x, end;
  int unit;              // tiled sequence
};

__device__ __forceinline__ bool next_item(Walk& w, const DevStep& ds, const ShapeInfo& s,
                                          const StepPlan& plan, const StepWork& work, int tpt,
                                          Item& it) {
  while (w.x < w.end) {
    int n;                 // the unit's key tiles
    int64_t unit0;         // its place on the line
    int keys;              // and its keys
    if (w.x < work.tile_prefix) {
      n = work.prefix_tile_steps;
      const int64_t unit = step_div(w.x, n + kStepTileUnit);
      unit0 = unit * (n + kStepTileUnit);
      it.kv_head = (int)step_div(unit, work.prefix_rows);
      const int tile = (int)(unit - (int64_t)it.kv_head * work.prefix_rows);
      it.prefix = true;
      it.table = ds.prefix_table;
      it.row = tile * tpt;
      it.n_tok = min(tpt, work.rows - it.row);
      it.pos = ds.prefix_len - 1;
      keys = ds.prefix_len;
    } else {
      StepSeq e = plan.tiled[w.unit];
      while (w.x - work.tile_prefix >= (int64_t)s.H_kv * ((int64_t)e.cum + e.tiles))
        e = plan.tiled[++w.unit];
      const int seen = e.ctx - e.n_new;
      const int64_t base = work.tile_prefix + (int64_t)s.H_kv * e.cum;
      it.kv_head = (int)step_div(w.x - base, e.tiles);
      unit0 = base + (int64_t)it.kv_head * e.tiles;
      int tile = 0;
      n = step_key_tiles(seen, e.n_new, tpt, 0);
      while (w.x - unit0 >= n + kStepTileUnit) {
        unit0 += n + kStepTileUnit;
        n = step_key_tiles(seen, e.n_new, tpt, ++tile);
      }
      it.prefix = false;
      it.table = ds.block_table + (int64_t)e.seq * ds.max_blocks;
      it.row = e.row + tile * tpt;
      it.n_tok = min(tpt, e.n_new - tile * tpt);
      it.pos = seen + tile * tpt;
      keys = it.pos + it.n_tok;
    }
    // the unit's tiles [first, last) of this segment
    const int64_t from = w.x - unit0 - kStepTileUnit, to = w.end - unit0 - kStepTileUnit;
    const int first = (int)(from < 0 ? 0 : from);
    const int last = (int)(to < 0 ? 0 : to < n ? to : n);
    w.x = unit0 + n + kStepTileUnit;
    if (first >= last) continue;
    it.head = first == 0;
    it.whole = it.head && last == n;
    it.kb = first * kKeys;
    it.ke = (int)min((int64_t)keys, (int64_t)last * kKeys);
    it.n = last - first;
    return true;
  }
  return false;
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

__global__ void __launch_bounds__(kThreads, 2)
    step_tile_kernel(const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, DevStep ds, ShapeInfo shp,
                     StepWorkspace ws, const __nv_bfloat16* __restrict__ q,
                     __nv_bfloat16* __restrict__ o, int first) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (first) ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  const StepPlan plan = step_plan(ds.plan, ds.num_seqs, ds.max_tokens);
  const StepWork work = step_work(ds, shp, plan);
  const int64_t ctas = min((int64_t)gridDim.x, work.tile_total);
  if ((ptx::smem_u32(smem_raw) & 1023) || blockIdx.x >= ctas) {
    // (the swizzled operand layouts need a 1024-byte aligned base)
    if (threadIdx.x == 0 && blockIdx.x < ctas) atomicCAS(ds.status, 0, kDevBounds);
    ptx::pdl_wait_previous();   // the grid's completion still covers its predecessor
    return;
  }
  uint8_t* kv_s = smem_raw;                      // [kStages][kTileBytes]
  Bars* bars = reinterpret_cast<Bars*>(kv_s + kStages * kTileBytes);
  volatile int* abort_flag = &bars->abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int B = shp.B, g = shp.g, tpt = step_tile_tokens(g);

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&bars->q_full[b], 4 * 32);
      ptx::mbar_init(&bars->s_full[b], 1);
      ptx::mbar_init(&bars->p_full[b], 4 * 32);
      ptx::mbar_init(&bars->o_done[b], 1);
    }
    ptx::mbar_init(&bars->o_free, 4 * 32);
    ptx::mbar_init(&bars->drain, 1);
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&bars->kv_full[s], 1);
      ptx::mbar_init(&bars->kv_empty[s], 1);
    }
    bars->abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  Walk walk;
  walk.x = step_cut(blockIdx.x, work.tile_total, ctas);
  walk.end = step_cut(blockIdx.x + 1, work.tile_total, ctas);
  walk.unit = 0;
  if (walk.x >= work.tile_prefix) {
    // the tiled sequence that holds this CTA's first step
    const int64_t v = step_div(walk.x - work.tile_prefix, shp.H_kv);
    int hi = plan.header[kPlanTiled] - 1;
    while (walk.unit < hi) {
      const int mid = (walk.unit + hi + 1) >> 1;
      if (plan.tiled[mid].cum <= v) walk.unit = mid;
      else hi = mid - 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // Every role walks the same segments in the same order.  Ring indices, score
  // buffers and barrier phases carry over from segment to segment: `gi` is the
  // ring index of a segment's K_0, `tc0` the number of its first key tile.
  if (warp >= 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == kProducerWarp) {
      // ---------------------------------------------------------- TMA producer
      // Lane i copies box i of a tile; a box whose block id is out of range is
      // skipped (and reported).  Ids are loaded three tiles ahead.
      const int box_rows = B < kKeys ? B : kKeys, boxes = kKeys / box_rows;
      Item it;
      uint32_t gi = 0;
      bool stop = false;
      while (!stop && next_item(walk, ds, shp, plan, work, tpt, it)) {
        auto look_up = [&](int j) -> int {
          const int key = it.kb + j * kKeys + lane * box_rows;
          return lane < boxes && j < it.n && key < it.ke ? it.table[key / B] : -2;
        };
        // one K or V tile: j is the tile, id this lane's box of it (-2: none)
        auto copy = [&](const CUtensorMap* map, int j, int id, uint32_t index) {
          const int st = index % kStages;
          bool go = !*abort_flag;
          if (go && index >= (uint32_t)kStages)
            go = ptx::mbar_wait(&bars->kv_empty[st], ((index / kStages) - 1) & 1, kWaitLimit);
          if (!__all_sync(0xffffffffu, go)) {
            if (lane == 0) {
              ptx::report_wait(ds.status, kDevTimeout, 72, (int)index);
              *abort_flag = 1;
            }
            stop = true;
            return;
          }
          const bool ok = id != -2 && (uint32_t)id < (uint32_t)ds.num_blocks;
          if (id != -2 && !ok) atomicCAS(ds.status, 0, kDevBounds);
          const int n = __popc(__ballot_sync(0xffffffffu, ok));
          if (lane == 0)
            ptx::mbar_arrive_expect_tx(&bars->kv_full[st], (uint32_t)(n * box_rows * 256));
          __syncwarp();
          if (ok) {
            const int key = it.kb + j * kKeys + lane * box_rows;
            const int row = (id * shp.H_kv + it.kv_head) * B + key % B;
            uint8_t* dst = kv_s + st * kTileBytes + lane * box_rows * 128;
            ptx::tma_load_2d(dst, map, 0, row, &bars->kv_full[st]);
            ptx::tma_load_2d(dst + kHalf, map, 64, row, &bars->kv_full[st]);
          }
          __syncwarp();
        };
        int id0 = look_up(0), id1 = look_up(1), id2 = look_up(2);
        copy(&tmap_k, 0, id0, gi);
        if (!stop && it.n > 1) copy(&tmap_k, 1, id1, gi + 1);
        for (int j = 0; !stop && j < it.n; ++j) {
          const int id3 = look_up(j + 3);
          copy(&tmap_v, j, id0, gi + ring_v(j, it.n));
          if (!stop && j + 2 < it.n) copy(&tmap_k, j + 2, id2, gi + ring_k(j + 2));
          id0 = id1;
          id1 = id2;
          id2 = id3;
        }
        if (!stop) gi += 2 * it.n;
      }
      // every copy must land before the CTA may exit: the softmax warps waited
      // for each tile of a finished walk; after an abort, wait for the stages
      if (stop)
        for (int st = 0; st < kStages; ++st)
          for (uint32_t ph = 0; ph < 2; ++ph)
            ptx::mbar_wait(&bars->kv_full[st], ph, kWaitLimit / 64);
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- MMA issuer
      // The whole warp walks the loop and waits, so that every operand of an
      // MMA is a warp-uniform value; one elected lane issues.
      const bool leader = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      constexpr uint32_t idesc_s = instr_desc(kRows, kKeys, 0);
      constexpr uint32_t idesc_o = instr_desc(kRows, 128, 1);
      // descriptor words of ring stage 0 as K (K-major) and as V (MN-major, the
      // two 64-column halves kHalf apart)
      const uint32_t hi = desc_hi(1024);
      const uint32_t k_lo = desc_lo(ptx::smem_u32(kv_s), 16);
      const uint32_t v_lo = desc_lo(ptx::smem_u32(kv_s), kHalf);
      static_assert(kKeys == 128 && kHalf == 16384, "the K = 128 issue blocks assume these");
      // S = Q K^T into score buffer t & 1 (whose P the PV of tile t - 2 read:
      // MMAs of one thread run in order)
      auto issue_qk = [&](uint32_t t, uint32_t index, uint32_t qbuf) {
        const uint32_t st = index % kStages;
        const uint32_t kt = __shfl_sync(0xffffffffu, k_lo + ((st * kTileBytes) >> 4), 0);
        if (leader) {
          tc_mma_ts_kmajor_k128(tm + (t & 1) * kKeys, tm + kQCol + qbuf * 64, kt, hi, idesc_s);
          tc_commit(&bars->s_full[t & 1]);
          tc_commit(&bars->kv_empty[st]);
        }
        __syncwarp();
      };
      // O += P V
      auto issue_pv = [&](uint32_t t, uint32_t index, bool acc) {
        const uint32_t st = index % kStages;
        const uint32_t vt = __shfl_sync(0xffffffffu, v_lo + ((st * kTileBytes) >> 4), 0);
        if (leader) {
          tc_mma_ts_k128(tm + kOCol, tm + (t & 1) * kKeys, vt, hi, idesc_o, acc);
          tc_commit(&bars->o_done[t & 1]);
          tc_commit(&bars->kv_empty[st]);
        }
        __syncwarp();
      };
      bool ok = true;
      int site = 0, at = 0;
      // After a wait on a barrier that other threads' tensor-memory accesses
      // complete (Q or P written, O read) the MMAs that follow are ordered
      // after those accesses with a tcgen05 fence.
      auto wait_bar = [&](uint64_t* bar, uint32_t parity, int where, int index) {
        const bool got = ptx::mbar_wait(bar, parity, kWaitLimit) && !*abort_flag;
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          site = where;
          at = index;
          return false;
        }
        tc_fence_after();
        return true;
      };
      Item it;
      uint32_t gi = 0, tc0 = 0;
      for (uint32_t k = 0; ok && next_item(walk, ds, shp, plan, work, tpt, it); ++k) {
        if (!wait_bar(&bars->q_full[k & 1], (k >> 1) & 1, 73, (int)k)) break;
        for (int j = 0; ok && j < 2 && j < it.n; ++j) {
          const uint32_t index = gi + ring_k(j);
          if (!wait_bar(&bars->kv_full[index % kStages], (index / kStages) & 1, 74, (int)index))
            break;
          issue_qk(tc0 + j, index, k & 1);
        }
        // then per key tile j: PV(j) QK(j+2) once its softmax has written P.
        // The softmax threads have also seen V_j and K_j+2 land before they
        // report P: a wait of the issuing thread costs 200 to 450 cycles while
        // its products are queued
        for (int j = 0; ok && j < it.n; ++j) {
          const uint32_t t = tc0 + j;
          if (!wait_bar(&bars->p_full[t & 1], (t >> 1) & 1, 75, (int)t)) break;
          // the previous unit's O must have been read
          if (j == 0 && k > 0 && !wait_bar(&bars->o_free, (k - 1) & 1, 76, (int)k)) break;
          issue_pv(t, gi + ring_v(j, it.n), j > 0);
          if (j + 2 < it.n) issue_qk(t + 2, gi + ring_k(j + 2), k & 1);
        }
        gi += 2 * it.n;
        tc0 += it.n;
      }
      if (!ok && lane == 0) {
        ptx::report_wait(ds.status, kDevTimeout, site, at);
        *abort_flag = 1;
      }
      // every MMA issued must finish before tensor memory is released
      if (leader) tc_commit(&bars->drain);
      __syncwarp();
      ptx::mbar_wait(&bars->drain, 0, kWaitLimit);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------------------ softmax warps
    const int row = threadIdx.x;                      // 0..127 = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    const float qk_scale = shp.scale * kLog2e;
    const int tok = row / g, hh = row - tok * g;      // its token in the tile, and head
    // this thread's query row -> tensor memory, buffer b; rows past the tile's
    // end are zero
    auto write_q = [&](const Item& u, uint32_t b) {
      float qv[64];
      uint4* q4 = reinterpret_cast<uint4*>(qv);
      if (tok < u.n_tok) {
        const uint4* src = reinterpret_cast<const uint4*>(
            q + ((int64_t)(u.row + tok) * shp.H_q + u.kv_head * g + hh) * 128);
#pragma unroll
        for (int i = 0; i < 16; ++i) q4[i] = src[i];
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) q4[i] = make_uint4(0, 0, 0, 0);
      }
      tmem_st32(lane_base + kQCol + b * 64, qv);
      tmem_st32(lane_base + kQCol + b * 64 + 32, qv + 32);
      tmem_wait_st();
      tc_fence_before();
      ptx::mbar_arrive(&bars->q_full[b]);
    };
    uint32_t gi = 0, tc0 = 0;
    bool ok = true;
    int site = 0, at = 0;
    Item it, nx;
    bool more = next_item(walk, ds, shp, plan, work, tpt, it);
    if (more) write_q(it, 0);
    for (uint32_t k = 0; more && ok; ++k) {
      // the last key this row sees
      const int pos = it.prefix ? it.pos : it.pos + tok;
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < it.n; ++j) {
        const uint32_t t = tc0 + j;
        // tcgen05.ld/st are warp-collective: every decision below is warp-uniform
        const bool got = ptx::mbar_wait(&bars->s_full[t & 1], (t >> 1) & 1, kWaitLimit);
        if (!__all_sync(0xffffffffu, got) || __any_sync(0xffffffffu, *abort_flag != 0)) {
          ok = false;
          site = 81;
          at = (int)t;
          break;
        }
        tc_fence_after();
        const uint32_t s_col = lane_base + (t & 1) * kKeys;   // S of the tile; then its P
        const int key0 = it.kb + j * kKeys;
        // this row sees the tile's first `lim` keys: those <= its position and
        // before the unit's end (a prefix of the key tile, possibly empty or all)
        const int lim = min(pos + 1, it.ke) - key0;
        const bool full = __all_sync(0xffffffffu, lim >= kKeys);
        // the whole row of scores in one round trip (four loads, one wait)
        float sc[128];
        tmem_ld32(s_col, sc);
        tmem_ld32(s_col + 32, sc + 32);
        tmem_ld32(s_col + 64, sc + 64);
        tmem_ld32(s_col + 96, sc + 96);
        tmem_wait_ld();
        if (!full) {
#pragma unroll
          for (int c = 0; c < 128; ++c) sc[c] = c < lim ? sc[c] : -INFINITY;
        }
        // row max: eight independent partial maxima over columns u, u+8, ...,
        // u+120, each built from three-input maxima (half the instructions)
        float mx8[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          float a = ptx::fmax3(sc[u], sc[u + 8], sc[u + 16]);
#pragma unroll
          for (int i = 0; i < 6; ++i) a = ptx::fmax3(a, sc[u + 24 + 16 * i], sc[u + 32 + 16 * i]);
          mx8[u] = fmaxf(a, sc[u + 120]);
        }
        const float mraw = ptx::fmax3(ptx::fmax3(mx8[0], mx8[1], mx8[2]),
                                      ptx::fmax3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
        // the scale is positive, so the row max scales with it
        const float mt = mraw * qk_scale;
        float corr = 1.f;
        const bool raise = mt > m_ref + kRescaleThreshold;
        if (raise) {
          corr = ptx::ex2(m_ref - mt);
          m_ref = mt;
        }
        // rescaling O needs every earlier PV of this unit finished (only when a
        // row's max rose)
        if (j > 0 && __any_sync(0xffffffffu, raise)) {
          const bool done =
              ptx::mbar_wait(&bars->o_done[(t - 1) & 1], ((t - 1) >> 1) & 1, kWaitLimit);
          if (!__all_sync(0xffffffffu, done)) {
            ok = false;
            site = 83;
            at = (int)t;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) {
            float ov[32];
            tmem_ld32(lane_base + kOCol + c4 * 32, ov);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) ov[c] *= corr;
            tmem_st32(lane_base + kOCol + c4 * 32, ov);
          }
          tmem_wait_st();
        }
        // a row with no key so far keeps m_ref = -inf: its p are 0
        const float nbase = m_ref == -INFINITY ? 0.f : -m_ref;
        // P as bf16 pairs over the first 64 S columns (already read): the PV
        // operand's type, each weight off by at most 2^-8 of itself; their sum
        // stays fp32.  Scaling and sum run as packed pairs (one instruction for
        // two columns): the softmax is bound by instruction issue and the
        // exponentials.
        float ps8[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) ps8[u] = 0.f;
#pragma unroll
        for (int qt = 0; qt < 4; ++qt) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            float x0, x1;
            ptx::fma2(x0, x1, sc[qt * 32 + c], sc[qt * 32 + c + 1], qk_scale, qk_scale, nbase,
                      nbase);
            const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
            const int a = (c >> 1) & 3;
            ptx::add2(ps8[2 * a], ps8[2 * a + 1], p0, p1);
            pk[c / 2] = ptx::pack_bf16x2(p0, p1);
          }
          tmem_st16(s_col + qt * 16, pk);
        }
        tmem_wait_st();
        const float ps =
            ((ps8[0] + ps8[1]) + (ps8[2] + ps8[3])) + ((ps8[4] + ps8[5]) + (ps8[6] + ps8[7]));
        l = l * corr + ps;
        // V_j and K_j+2 have landed (the issuing thread relies on it)
        const uint32_t gv = gi + ring_v(j, it.n), gk = gi + ring_k(j + 2);
        bool landed = ptx::mbar_wait(&bars->kv_full[gv % kStages], (gv / kStages) & 1, kWaitLimit);
        if (landed && j + 2 < it.n)
          landed = ptx::mbar_wait(&bars->kv_full[gk % kStages], (gk / kStages) & 1, kWaitLimit);
        if (!__all_sync(0xffffffffu, landed)) {
          ok = false;
          site = 82;
          at = (int)gv;
          break;
        }
        if (j == it.n - 1 && (it.ke % kKeys) != 0) {
          // keys past the unit's end may be anything (unwritten cache slots, and
          // 0 * NaN is NaN): their V rows are zeroed
          uint8_t* vt = kv_s + (gv % kStages) * kTileBytes;
          const int valid = it.ke - key0;
          for (int e = row; e < (kKeys - valid) * 16; e += kRows) {
            const int key = valid + e / 16, c = e % 16;
            *reinterpret_cast<uint4*>(vt + (c >> 3) * kHalf + key * 128 + ((c & 7) << 4)) =
                make_uint4(0, 0, 0, 0);
          }
          // the PV MMAs read these rows through the async proxy
          ptx::fence_proxy_async_smem();
        }
        tc_fence_before();
        ptx::mbar_arrive(&bars->p_full[t & 1]);
      }
      if (!ok) break;
      // the next unit's queries, while this one's last products run
      more = next_item(walk, ds, shp, plan, work, tpt, nx);
      if (more) write_q(nx, (k + 1) & 1);
      const uint32_t tl = tc0 + it.n - 1;
      const bool fin = ptx::mbar_wait(&bars->o_done[tl & 1], (tl >> 1) & 1, kWaitLimit);
      if (!__all_sync(0xffffffffu, fin)) {
        ok = false;
        site = 84;
        at = (int)tl;
        break;
      }
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const bool store = tok < it.n_tok;
      // O itself when nothing is to be joined, the unit's rows of the
      // workspace, or this CTA's spill rows
      const bool partial = !it.whole || ds.prefix_len > 0;
      const int64_t slot = it.head ? (int64_t)(it.row + tok) * shp.H_q + it.kv_head * g + hh
                                   : (int64_t)blockIdx.x * kRows + row;
      __nv_bfloat16* orow = o + slot * 128;
      float* prow = (it.head ? (it.prefix ? ws.pre_o : ws.own_o) : ws.tile_o) + slot * 128;
      float* plse = it.head ? (it.prefix ? ws.pre_lse : ws.own_lse) : ws.tile_lse;
#pragma unroll
      for (int c4 = 0; c4 < 4; ++c4) {
        float ov[32];
        tmem_ld32(lane_base + kOCol + c4 * 32, ov);
        tmem_wait_ld();
        if (store && !partial) {
#pragma unroll
          for (int c8 = 0; c8 < 4; ++c8) {
            uint4 v;
            v.x = ptx::pack_bf16x2(ov[c8 * 8 + 0] * inv, ov[c8 * 8 + 1] * inv);
            v.y = ptx::pack_bf16x2(ov[c8 * 8 + 2] * inv, ov[c8 * 8 + 3] * inv);
            v.z = ptx::pack_bf16x2(ov[c8 * 8 + 4] * inv, ov[c8 * 8 + 5] * inv);
            v.w = ptx::pack_bf16x2(ov[c8 * 8 + 6] * inv, ov[c8 * 8 + 7] * inv);
            *reinterpret_cast<uint4*>(orow + c4 * 32 + c8 * 8) = v;
          }
        } else if (store) {
#pragma unroll
          for (int c8 = 0; c8 < 8; ++c8)
            *reinterpret_cast<float4*>(prow + c4 * 32 + c8 * 4) =
                make_float4(ov[c8 * 4 + 0] * inv, ov[c8 * 4 + 1] * inv, ov[c8 * 4 + 2] * inv,
                            ov[c8 * 4 + 3] * inv);
        }
      }
      if (store && partial) plse[slot] = l > 0.f ? m_ref + log2f(l) : -INFINITY;
      // O has been read: the next unit's first PV may overwrite it
      tc_fence_before();
      ptx::mbar_arrive(&bars->o_free);
      gi += 2 * it.n;
      tc0 += it.n;
      it = nx;
    }
    if (!ok) {
      ptx::report_wait(ds.status, kDevTimeout, site, at);
      *abort_flag = 1;
    }
  }

  // all roles done (every wait above is bounded): release tensor memory
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (!first) ptx::pdl_wait_previous();
}

}  // namespace

cudaError_t launch_step_tile(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w,
                             const void* q, const void* k_cache, const void* v_cache, void* o,
                             bool first, cudaStream_t st) {
  const int64_t rows = (int64_t)ds.num_blocks * s.H_kv * s.B;
  const int box_rows = s.B < kKeys ? s.B : kKeys;
  CUtensorMap tk, tv;
  cudaError_t e = make_cache_tmap(&tk, k_cache, rows, s.D, box_rows);
  if (e == cudaSuccess) e = make_cache_tmap(&tv, v_cache, rows, s.D, box_rows);
  if (e != cudaSuccess) return e;
  // once per device: the shared-memory limit, and whether the build's register
  // count is the one that the split above divides (a smaller pool would leave
  // the softmax warps waiting for registers)
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load() & bit)) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, step_tile_kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(step_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kStepTileSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(step_tile_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)w.tile_grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kStepTileSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, step_tile_kernel, tk, tv, ds, s, w, (const __nv_bfloat16*)q,
                            (__nv_bfloat16*)o, first ? 1 : 0);
}

}  // namespace rbkv
