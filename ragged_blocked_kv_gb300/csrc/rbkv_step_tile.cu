// Tensor-core attention of a step (tcgen05): all rows of the batch over the
// shared prefix, and the new rows of longer sequences over their own keys.
//
// Over the prefix every row of the batch sees the same keys, so for one KV
// head the rows of all sequences and the heads of the group form one matrix
// of packed rows (token-major: row = token * g + head): Q K^T and P V are
// plain products of 128-row tiles, and the prefix's K and V are read once for
// 256 rows.  A sequence whose own packed rows exceed the streaming kernel's 16
// is cut the same way over its own keys, with a causal limit per row.
//
// A unit is a pair of 128-row query tiles (A, B) of one KV head; its 128-key
// tiles are steps of the line that rbkv_step.h cuts evenly over one CTA per
// SM, so every CTA walks the same number of steps whatever the shapes.  Roles:
//  - warp 8 (TMA): loads the unit's query tiles into shared memory (a box of
//    g heads x 128/g tokens) and streams 128-key K and V tiles, in the order
//    K0 V0 K1 V1 ..., through a 5-stage ring of 32 KB stages (128-byte
//    swizzle), looking block ids up through the block list;
//  - warp 9 (MMA): one thread issues, per query tile X, S_X = Q_X K^T
//    (M=128, N=128 keys, K=128; Q from shared memory) into tensor memory and
//    O_X += P_X V (M=128, N=128 head dims, K=128 keys; P from tensor memory),
//    in the order QK_A(0) QK_B(0), then for each key tile j: PV_A(j)
//    QK_A(j+1) PV_B(j) QK_B(j+1): one tile's softmax runs while the tensor
//    pipe works on the other tile;
//  - warps 0-3 / 4-7 (softmax of tile A / B): thread i owns packed row i =
//    TMEM lane i; it keeps a running max that is raised only when the row max
//    grows by more than 2^8 (the accumulator in tensor memory is then rescaled
//    in place), writes P as bf16 pairs over the score columns it has read, and
//    at the end of a segment stores the normalised partial output and its
//    log-sum-exp (or O, when nothing is to be joined).
// Tensor memory (512 columns x 128 lanes): S/P of A [0,128), O of A
// [128,256), S/P of B [256,384), O of B [384,512).  Shared memory: Q of A and
// B (32 KB each) and the ring (160 KB), about 225 KB: one CTA per SM.
// Every wait is bounded; on timeout the kernel records RBKV_ERR_TIMEOUT, lets
// its copies and MMAs drain (bounded), frees its tensor memory and returns.
#include <algorithm>
#include <atomic>
#include <mutex>

#include "rbkv_step.h"
#include "rbkv_ptx.cuh"
#include "rbkv_tcgen05.cuh"

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace rbkv {

namespace {

using namespace tc;

constexpr int kRows = kStepTileRows;       // 128 query rows (MMA M)
constexpr int kKeys = kStepTileKeys;       // 128 keys per KV tile (MMA N of QK^T)
constexpr int kStages = 5;                  // ring stages, each one K or one V tile
constexpr int kHalf = kKeys * 128;          // 16 KB: 128 rows x 64 head dims
constexpr int kTileBytes = 2 * kHalf;       // 32 KB: 128 rows x 128 head dims
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
// three warpgroups: two softmax warpgroups and one with the TMA and MMA
// warps (its other two warps idle), so that registers can move between
// warpgroups:
// launched at kLaunchRegs a thread, the third warpgroup gives back down to
// kIssueRegs and the softmax warpgroups take kSoftmaxRegs.  The shares add up
// to the launch's total exactly (a larger claim would wait forever).
constexpr int kThreads = 12 * 32;
constexpr int kLaunchRegs = 168;
constexpr int kIssueRegs = 88;
constexpr int kSoftmaxRegs = 208;
static_assert(128 * kIssueRegs + 256 * kSoftmaxRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch's registers");
constexpr int kTmemCols = 512;
constexpr int kTileCols = 256;              // tensor-memory columns of one query tile
constexpr int kOCol = 128;                  // O after S/P inside a tile's columns
constexpr int kSmemBytes = 2 * kTileBytes + kStages * kTileBytes + 1024;
constexpr long long kWaitLimit = 4000000000LL;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;   // log2 units

// Each barrier is waited on in order of its phases and can never run two
// phases ahead of a waiter (the parity of a wait is then unambiguous).
struct Bars {
  uint64_t q_full[2];    // query tile X landed (TMA)
  uint64_t q_empty[2];   // the last QK^T of an item read query tile X
  uint64_t kv_full[kStages];      // a K or V tile landed (TMA)
  uint64_t kv_empty[kStages];     // the MMAs are done with the stage
  uint64_t s_full[2];    // QK^T of tile X done: S_X readable
  uint64_t p_full[2];    // softmax of tile X done: P_X written (and V tail rows zeroed)
  uint64_t o_done[2];    // PV of tile X done
  uint64_t drain;        // every MMA the CTA issued done (before tensor memory is freed)
  uint64_t o_free[2];    // epilogue of tile X read O_X: the next item may overwrite it
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(2 * kTileBytes + kStages * kTileBytes + (int)sizeof(Bars) <= kSmemBytes,
              "shared-memory layout overflows its allocation");

// One segment of a unit as every role sees it.
struct Item {
  const int32_t* table;
  int kv_head;
  int row[2];      // first row of each query tile
  int n_tok[2];    // its tokens (0: no such tile)
  int n[2];        // key tiles of each query tile in this segment
  int pos;         // keys seen by tile A's first token, less one (a prefix: P - 1)
  int kb, ke;      // key range of the segment
  int nmax;        // its key tiles
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
    int n, k = 0;          // the unit's key tiles
    int64_t unit0;         // its place on the line
    StepSeq e;
    if (w.x < work.tile_prefix) {
      n = work.prefix_tile_steps;
      const int64_t unit = w.x / (n + kStepTileUnit);
      unit0 = unit * (n + kStepTileUnit);
      it.kv_head = (int)(unit / work.prefix_pairs);
      const int T = plan.header[kPlanRows];
      const int rp = (int)(unit - (int64_t)it.kv_head * work.prefix_pairs);
      it.prefix = true;
      it.table = ds.prefix_table;
      it.row[0] = rp * 2 * tpt;
      it.n_tok[0] = min(tpt, T - it.row[0]);
      it.n_tok[1] = max(0, min(tpt, T - it.row[0] - tpt));
      it.pos = ds.prefix_len - 1;
    } else {
      e = plan.tiled[w.unit];
      while (w.x - work.tile_prefix >= (int64_t)s.H_kv * ((int64_t)e.cum + e.tiles))
        e = plan.tiled[++w.unit];
      const int seen = e.ctx - e.n_new;
      const int64_t base = work.tile_prefix + (int64_t)s.H_kv * e.cum;
      it.kv_head = (int)((w.x - base) / e.tiles);
      unit0 = base + (int64_t)it.kv_head * e.tiles;
      n = step_pair_tiles(seen, e.n_new, 2 * tpt, 0);
      while (w.x - unit0 >= n + kStepTileUnit) {
        unit0 += n + kStepTileUnit;
        n = step_pair_tiles(seen, e.n_new, 2 * tpt, ++k);
      }
      const int off = k * 2 * tpt;
      it.prefix = false;
      it.table = ds.block_table + (int64_t)e.seq * ds.max_blocks;
      it.row[0] = e.row + off;
      it.n_tok[0] = min(tpt, e.n_new - off);
      it.n_tok[1] = max(0, min(tpt, e.n_new - off - tpt));
      it.pos = seen + off;
    }
    // the unit's tiles [first, last) of this segment
    const int64_t from = w.x - unit0 - kStepTileUnit, to = w.end - unit0 - kStepTileUnit;
    const int first = (int)(from < 0 ? 0 : from);
    const int last = (int)(to < 0 ? 0 : to < n ? to : n);
    w.x = unit0 + n + kStepTileUnit;
    if (first >= last) continue;
    // (the prefix: pos is its last key for every row; else A's rows see the
    // keys up to pos + their index, B's from there on)
    const int keys_a = it.prefix ? it.pos + 1 : it.pos + it.n_tok[0];
    const int keys = it.prefix ? it.pos + 1 : keys_a + it.n_tok[1];
    it.head = first == 0;
    it.whole = it.head && last == n;
    it.row[1] = it.row[0] + tpt;
    it.kb = first * kKeys;
    it.ke = (int)min((int64_t)keys, (int64_t)last * kKeys);
    it.nmax = last - first;
    it.n[0] = max(0, min(last, (int)(((int64_t)keys_a + kKeys - 1) / kKeys)) - first);
    it.n[1] = it.n_tok[1] > 0 ? it.nmax : 0;
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

// The box of a query tile's half: 64 head dims x g heads x 128/g tokens, its
// packed rows in order (tokens past max_tokens read as zero).
__device__ __forceinline__ void load_q_box(void* dst, const CUtensorMap* m, int d, int head,
                                           int token, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(d), "r"(head), "r"(token), "r"(ptx::smem_u32(bar))
      : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    step_tile_kernel(const __grid_constant__ CUtensorMap tmap_q,
                     const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, DevStep ds, ShapeInfo shp,
                     StepWorkspace ws, __nv_bfloat16* __restrict__ o, int first) {
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
  uint8_t* q_s = smem_raw;                       // [2][kTileBytes]
  uint8_t* kv_s = smem_raw + 2 * kTileBytes;     // [kStages][kTileBytes]
  Bars* bars = reinterpret_cast<Bars*>(kv_s + kStages * kTileBytes);
  volatile int* abort_flag = &bars->abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int B = shp.B, g = shp.g, tpt = step_tile_tokens(g);
  const int q_bytes = tpt * g * 256;             // a query tile's rows, 256 B each
  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      ptx::mbar_init(&bars->q_full[x], 1);
      ptx::mbar_init(&bars->q_empty[x], 1);
      ptx::mbar_init(&bars->s_full[x], 1);
      ptx::mbar_init(&bars->p_full[x], 4 * 32);
      ptx::mbar_init(&bars->o_done[x], 1);
      if (x == 0) ptx::mbar_init(&bars->drain, 1);
      ptx::mbar_init(&bars->o_free[x], 4 * 32);
    }
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
    const int64_t v = (walk.x - work.tile_prefix) / shp.H_kv;
    int hi = plan.header[kPlanTiled] - 1;
    while (walk.unit < hi) {
      const int mid = (walk.unit + hi + 1) >> 1;
      if (plan.tiled[mid].cum <= v) walk.unit = mid;
      else hi = mid - 1;
    }
  }
  Item it;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // Every role walks the same items in the same order.  The ring index `gi`
  // numbers this CTA's K and V tiles across items (K_j of an item at 2j, V_j
  // at 2j + 1 from the item's start), so stages and phases carry over.
  if (warp >= 8) {
  // the TMA, MMA and V warps' warpgroup gives registers to the softmax warpgroups
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      ptx::tma_prefetch_desc(&tmap_q);
      ptx::tma_prefetch_desc(&tmap_k);
      ptx::tma_prefetch_desc(&tmap_v);
      const int box_rows = B < kKeys ? B : kKeys;
      uint32_t gi = 0, qi[2] = {0, 0};
      bool stop = false;
      for (int k = 0; !stop && next_item(walk, ds, shp, plan, work, tpt, it); ++k) {
        #pragma unroll
        for (int x = 0; x < 2 && !stop; ++x) {
          if (it.n[x] == 0) continue;
          if (qi[x] > 0 &&
              !ptx::mbar_wait(&bars->q_empty[x], (qi[x] - 1) & 1, kWaitLimit)) {
            ptx::report_wait(ds.status, kDevTimeout, 41, k);
            *abort_flag = 1;
            stop = true;
            break;
          }
          uint8_t* dst = q_s + x * kTileBytes;
          ptx::mbar_arrive_expect_tx(&bars->q_full[x], q_bytes);
          load_q_box(dst, &tmap_q, 0, it.kv_head * g, it.row[x], &bars->q_full[x]);
          load_q_box(dst + kHalf, &tmap_q, 64, it.kv_head * g, it.row[x], &bars->q_full[x]);
          ++qi[x];
        }
        const int32_t* table = it.table;
        for (int j = 0; j < it.nmax && !stop; ++j) {
          // the boxes of key tile j: box i holds keys key0 + i * box_rows ..; a
          // box whose block id is out of range is skipped (and reported).  Rows
          // are recomputed where needed rather than kept in an array (a
          // runtime-indexed array would live in local memory)
          const int key0 = it.kb + j * kKeys;
          const int nsub = (min(it.ke - key0, kKeys) + box_rows - 1) / box_rows;
          auto box_row = [&](int i) -> int {
            const int key = key0 + i * box_rows;
            const int32_t blk = table[key / B];
            if (blk < 0 || blk >= ds.num_blocks) return -1;
            return (blk * shp.H_kv + it.kv_head) * B + (key % B);
          };
          int loads = 0;
          for (int i = 0; i < nsub; ++i) {
            if (box_row(i) >= 0)
              ++loads;
            else
              atomicCAS(ds.status, 0, kDevBounds);
          }
          for (int kv = 0; kv < 2; ++kv, ++gi) {
            const int s = gi % kStages;
            if (*abort_flag) {
              stop = true;
              break;
            }
            if (gi >= (uint32_t)kStages &&
                !ptx::mbar_wait(&bars->kv_empty[s], ((gi / kStages) - 1) & 1, kWaitLimit)) {
              ptx::report_wait(ds.status, kDevTimeout, 42, (int)gi);
              *abort_flag = 1;
              stop = true;
              break;
            }
            const CUtensorMap* map = kv ? &tmap_v : &tmap_k;
            uint8_t* dst = kv_s + s * kTileBytes;
            ptx::mbar_arrive_expect_tx(&bars->kv_full[s], (uint32_t)(loads * box_rows * 128 * 2));
            for (int i = 0; i < nsub; ++i) {
              const int row = box_row(i);
              if (row < 0) continue;
              const int off = i * box_rows * 128;
              ptx::tma_load_2d(dst + off, map, 0, row, &bars->kv_full[s]);
              ptx::tma_load_2d(dst + kHalf + off, map, 64, row, &bars->kv_full[s]);
            }
          }
        }
      }
      // every copy must land before the CTA may exit
      for (uint32_t t = gi > (uint32_t)kStages ? gi - kStages : 0; t < gi; ++t)
        ptx::mbar_wait(&bars->kv_full[t % kStages], (t / kStages) & 1, kWaitLimit);
      #pragma unroll
      for (int x = 0; x < 2; ++x)
        if (qi[x] > 0) ptx::mbar_wait(&bars->q_full[x], (qi[x] - 1) & 1, kWaitLimit);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the loop and waits, so that every operand of an MMA is
    // a warp-uniform value; one elected lane issues.
    {
      const bool leader = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      constexpr uint32_t idesc_s = instr_desc(kRows, kKeys, 0);
      constexpr uint32_t idesc_o = instr_desc(kRows, 128, 1);
      // descriptor words: the high word is common to every operand; the low
      // words of the Q tiles and of ring stage 0 (as K, K-major, and as V,
      // MN-major with the two 64-column halves kHalf apart) are offset per MMA
      const uint32_t hi = desc_hi(1024);
      const uint32_t q_lo = desc_lo(ptx::smem_u32(q_s), 16);
      const uint32_t k_lo = desc_lo(ptx::smem_u32(kv_s), 16);
      const uint32_t v_lo = desc_lo(ptx::smem_u32(kv_s), kHalf);
      // S_X = Q_X K^T into tile X's S columns (after the previous PV of tile X
      // read P_X over the same columns: MMAs of one thread run in order)
      auto issue_qk = [&](int x, uint32_t gk, bool last) {
        const uint32_t qt = q_lo + ((x * kTileBytes) >> 4);
        const uint32_t kt =
            __shfl_sync(0xffffffffu, k_lo + (((gk % kStages) * kTileBytes) >> 4), 0);
        const uint32_t d = tm + x * kTileCols;
        // head dims 16kk .. 16kk+15 in step kk: the half kk/4 of Q and K, 32-byte step kk%4
        if (leader) {
          tc_mma_ss_k128(d, qt, kt, hi, idesc_s, false);
          tc_commit(&bars->s_full[x]);
          if (last) tc_commit(&bars->q_empty[x]);
        }
        __syncwarp();
      };
      // O_X += P_X V
      auto issue_pv = [&](int x, uint32_t gv, bool acc) {
        const uint32_t vt =
            __shfl_sync(0xffffffffu, v_lo + (((gv % kStages) * kTileBytes) >> 4), 0);
        const uint32_t pt = tm + x * kTileCols;
        // keys 16kk .. 16kk+15 in step kk: P columns 8kk.., V rows 16kk.. (MN-major)
        static_assert(kKeys == 128 && kHalf == 16384, "the K = 128 issue blocks assume these");
        if (leader) {
          tc_mma_ts_k128(pt + kOCol, pt, vt, hi, idesc_o, acc);
          tc_commit(&bars->o_done[x]);
        }
        __syncwarp();
      };
      bool ok = true;
      int site = 0, at = 0;
      uint32_t gi = 0, qi[2] = {0, 0}, c[2] = {0, 0}, oi[2] = {0, 0};
      // After a wait on a barrier that other threads' tensor-memory accesses
      // complete (P written, O read) the MMAs that follow are ordered after
      // those accesses with a tcgen05 fence.  Tiles that the TMA loaded need
      // none: the barrier's transaction count already covers the copy.
      auto wait_bar = [&](uint64_t* bar, uint32_t parity, int where, int index,
                          bool tmem_sync) {
        const bool got = ptx::mbar_wait(bar, parity, kWaitLimit) && !*abort_flag;
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          site = where;
          at = index;
          return false;
        }
        if (tmem_sync) tc_fence_after();
        return true;
      };
      for (int k = 0; ok && next_item(walk, ds, shp, plan, work, tpt, it); ++k) {
        const uint32_t base = gi;
        gi += 2 * it.nmax;
        #pragma unroll
        for (int x = 0; x < 2 && ok; ++x) {
          if (it.n[x] == 0) continue;
          if (wait_bar(&bars->q_full[x], qi[x] & 1, 43, k, false)) ++qi[x];
        }
        // K_0: the first QK^T of both tiles
        if (!ok || !wait_bar(&bars->kv_full[base % kStages], (base / kStages) & 1, 44, (int)base, false))
          break;
        #pragma unroll
        for (int x = 0; x < 2; ++x)
          if (it.n[x] > 0) issue_qk(x, base, it.n[x] == 1);
        if (leader) tc_commit(&bars->kv_empty[base % kStages]);
        // then per key tile j: PV_A(j) QK_A(j+1) PV_B(j) QK_B(j+1), each tile's
        // products as soon as its softmax has written P.  The softmax threads
        // have also seen V_j and K_j+1 land before they report P: a wait of the
        // issuing thread costs 200 to 450 cycles while its products are queued
        for (int j = 0; ok && j < it.nmax; ++j) {
          const uint32_t gv = base + 2 * j + 1, gk = gv + 1;
          #pragma unroll
          for (int x = 0; ok && x < 2; ++x) {
            if (j >= it.n[x]) continue;
            if (!wait_bar(&bars->p_full[x], c[x] & 1, 46, (int)c[x], true)) break;
            if (j == 0 && oi[x] > 0 &&   // the previous item's epilogue must have read O_X
                !wait_bar(&bars->o_free[x], (oi[x] - 1) & 1, 47, (int)oi[x], true))
              break;
            issue_pv(x, gv, j > 0);
            ++c[x];
            if (j + 1 < it.n[x]) issue_qk(x, gk, j + 2 == it.n[x]);
          }
          if (!ok) break;
          // a stage is released once every product that reads it was issued
          if (leader) tc_commit(&bars->kv_empty[gv % kStages]);
          if (j + 1 < it.nmax && leader) tc_commit(&bars->kv_empty[gk % kStages]);
        }
        #pragma unroll
        for (int x = 0; x < 2; ++x)
          if (it.n[x] > 0) ++oi[x];
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
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------------------ softmax warps
    const int x = warp >> 2;                          // query tile of this warpgroup
    const int row = threadIdx.x & 127;                // 0..127 = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + x * kTileCols;
    const float qk_scale = shp.scale * kLog2e;
    uint32_t cnt = 0, gbase = 0;
    bool ok = true;
    int site = 0, at = 0;
    const int tok = row / g, hh = row - tok * g;      // its token in the tile, and head
    while (ok && next_item(walk, ds, shp, plan, work, tpt, it)) {
      // this warpgroup's tile, selected without indexing by x (a runtime value)
      const int nx = x ? it.n[1] : it.n[0];
      if (nx == 0) {
        gbase += 2 * it.nmax;
        continue;
      }
      const int kb = it.kb;
      const int ke = it.ke;
      // the last key this row sees
      const int pos = it.prefix ? it.pos : it.pos + x * tpt + tok;
      const uint32_t g_item = gbase;                  // ring index of the item's K_0
      gbase += 2 * it.nmax;
      // keys past the item's end in its last key tile may be anything (unwritten
      // cache slots, and 0 * NaN is NaN): they are zeroed in V, before any PV
      // reads that tile, by A's warpgroup when A reads it (the issuer runs A's
      // PV first), else by B's
      const bool zeroer = (x == 0) ? (nx == it.nmax) : (it.n[0] != it.nmax);
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < nx; ++j) {
        const uint32_t t = cnt + j;
        // tcgen05.ld/st are warp-collective: every decision below is warp-uniform
        const bool got = ptx::mbar_wait(&bars->s_full[x], t & 1, kWaitLimit);
        if (!__all_sync(0xffffffffu, got) || __any_sync(0xffffffffu, *abort_flag != 0)) {
          ok = false;
          site = 51;
          at = (int)t;
          break;
        }
        tc_fence_after();
        const uint32_t s_col = lane_base;               // S of key tile j; then its P
        const int key0 = kb + j * kKeys;
        // this row sees the tile's first `lim` keys: those <= its position and
        // before its tile's end (a prefix of the key tile, possibly empty or all)
        const int lim = min(pos + 1, ke) - key0;
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
        // rescaling O needs every earlier PV of this item finished (only when
        // a row's max rose)
        if (j > 0 && __any_sync(0xffffffffu, raise)) {
          const bool done = ptx::mbar_wait(&bars->o_done[x], (t - 1) & 1, kWaitLimit);
          if (!__all_sync(0xffffffffu, done)) {
            ok = false;
            site = 53;
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
        // a row with no key in this piece so far keeps m_ref = -inf: its p are 0
        const float nbase = m_ref == -INFINITY ? 0.f : -m_ref;
        // P as bf16 pairs over the first 64 S columns (already read), 64 keys
        // (32 columns) per store.  The scaling and the row sum run as packed
        // pairs (one instruction for two columns): the softmax is bound by
        // instruction issue and the exponentials, and it runs while the
        // tensor pipe works on the other query tile.
        float ps8[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) ps8[u] = 0.f;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float pk[32];
          uint32_t* pk32 = reinterpret_cast<uint32_t*>(pk);
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            float x0, x1;
            ptx::fma2(x0, x1, sc[hf * 64 + c], sc[hf * 64 + c + 1], qk_scale, qk_scale, nbase,
                      nbase);
            const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
            const int a = (c >> 1) & 3;
            ptx::add2(ps8[2 * a], ps8[2 * a + 1], p0, p1);
            pk32[c / 2] = ptx::pack_bf16x2(p0, p1);
          }
          tmem_st32(s_col + hf * 32, pk);
        }
        tmem_wait_st();
        const float ps =
            ((ps8[0] + ps8[1]) + (ps8[2] + ps8[3])) + ((ps8[4] + ps8[5]) + (ps8[6] + ps8[7]));
        l = l * corr + ps;
        // V_j and K_j+1 have landed (the issuing thread relies on it)
        const uint32_t gv = g_item + 2 * j + 1;     // ring index of V_j
        bool landed = ptx::mbar_wait(&bars->kv_full[gv % kStages], (gv / kStages) & 1, kWaitLimit);
        if (landed && j + 1 < it.nmax)
          landed = ptx::mbar_wait(&bars->kv_full[(gv + 1) % kStages], ((gv + 1) / kStages) & 1,
                                  kWaitLimit);
        if (!__all_sync(0xffffffffu, landed)) {
          ok = false;
          site = 52;
          at = (int)gv;
          break;
        }
        if (zeroer && j == it.nmax - 1 && (it.ke % kKeys) != 0) {
          const int s = gv % kStages;
          uint8_t* vt = kv_s + s * kTileBytes;
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
        ptx::mbar_arrive(&bars->p_full[x]);
      }
      if (!ok) break;
      const uint32_t tl = cnt + nx - 1;
      cnt += nx;
      const bool fin = ptx::mbar_wait(&bars->o_done[x], tl & 1, kWaitLimit);
      if (!__all_sync(0xffffffffu, fin)) {
        ok = false;
        site = 54;
        at = (int)tl;
        break;
      }
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const int row0 = x ? it.row[1] : it.row[0];
      const bool store = tok < (x ? it.n_tok[1] : it.n_tok[0]);
      // O itself when nothing is to be joined, the unit's rows of the
      // workspace, or this CTA's spill rows
      const bool partial = !it.whole || ds.prefix_len > 0;
      const int64_t slot = it.head
                               ? (int64_t)(row0 + tok) * shp.H_q + it.kv_head * g + hh
                               : ((int64_t)blockIdx.x * 2 + x) * kRows + row;
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
      // O_X has been read: the next item's first PV may overwrite it
      tc_fence_before();
      ptx::mbar_arrive(&bars->o_free[x]);
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
  CUtensorMap tq, tk, tv;
  cudaError_t e = make_q_tmap(&tq, q, ds.max_tokens, s);
  if (e == cudaSuccess) e = make_cache_tmap(&tk, k_cache, rows, s.D, box_rows);
  if (e == cudaSuccess) e = make_cache_tmap(&tv, v_cache, rows, s.D, box_rows);
  if (e != cudaSuccess) return e;
  // the shared-memory limit is raised once per device
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load() & bit)) {
    e = cudaFuncSetAttribute(step_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(step_tile_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)w.tile_grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, step_tile_kernel, tq, tk, tv, ds, s, w, (__nv_bfloat16*)o,
                            first ? 1 : 0);
}

}  // namespace rbkv
