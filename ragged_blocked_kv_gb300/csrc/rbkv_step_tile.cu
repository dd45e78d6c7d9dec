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
//  - warps 4 and 7 (TMA): stream the 128-key tiles of K and of V through a
//    4-stage ring of 32 KB (128-byte swizzle), in the order K0 K1 V0 K2 V1 K3
//    ..., one box per block (or 128 keys of a larger one) and half of the head
//    dim; the lanes hold the block ids, one elected lane copies.  (A copy costs
//    its thread about 200 cycles: one warp for both could not keep up with a
//    step of 1600);
//  - warp 5 (MMA): one elected lane issues S = Q K^T (M=128, N=128 keys,
//    K=128; Q from tensor memory) into one of two score buffers and
//    O += P V (P from tensor memory), in the order QK(0) QK(1), then per key
//    tile j: PV(j) QK(j+2).  The next tile's scores are so computed under the
//    softmax of the current one;
//  - warp 6 walks the line and publishes the segments to the other roles (one
//    copy of that code: the kernel starts with cold instruction caches, and a
//    second copy cost a segment 4000 cycles); and it reports, with the softmax
//    threads, that a tile's products may be issued: it has seen V_j and K_j+2
//    land, so that the issuing thread has one wait per step (a wait costs it
//    200 to 450 cycles while its products are queued) and the softmax threads
//    none for the ring;
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
//
// Bound by two chains of a key tile of nearly the same length, 1900 cycles: the
// softmax (see S 280 or more, read it 220, maximum 270, exponentials and P 980)
// and the ring (K_j+2 takes the stage that QK(j) releases: 330 until its
// producer wakes, 850 for its four copies, 650 until they land); the two
// products take 1180 of the tensor pipe.  Besides, 7000 cycles to start and 4500
// to 8000 per unit.  Alone, 512 rows of 32 heads behind 4096 keys (34 GFLOP) take 33.5 us,
// 1.03 PFLOP/s and 54% of the library's best product; 64 rows of 64 heads
// behind 15999 keys 38 us.  (Tensor pipe 39% active; issue 31%.)
//
// Drafted tokens (rbkv_step_attention_draft) are the same kernel with another mask:
// a row sees a run of keys from the first and, behind it, those of its ancestors
// (rbkv_step.h).  Only a unit's last tile or two hold such keys; their scores are
// hidden in tensor memory in front of the softmax, which stays as it is.  Two query
// tiles of one sequence may be walked side by side (StepLanes).  Of a unit's 8000
// cycles beside its key tiles (1500 each), as stamped behind 1100 keys, the queries
// take 2800 (3300 in 16-byte loads), the results 2500, the hidden scores 1300; a
// call's first 18000 cycles are cold caches.
//
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
constexpr int kKeyWarp = 4, kValueWarp = 7;
constexpr int kMmaWarp = 5;
constexpr int kWalkWarp = 6;
constexpr int kSegments = 8, kAhead = 3;    // published segments, and how far ahead
// Two warpgroups: the softmax warps, and one with the other roles.  Launched at
// kLaunchRegs a thread, the second gives back down to kIssueRegs and the first
// takes kSoftmaxRegs: the shares add up to the launch's total (a larger claim
// would wait forever), and the launch's total leaves half of an SM's registers
// to a streaming CTA.
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

// One segment of a unit, as published (n = 0: there are no more).
struct __align__(16) Segment {
  const int32_t* table;
  int kv_head;
  int row, n_tok;  // first row and tokens of the query tile
  int pos;         // last key its first token sees (the prefix: every token)
  int kb, ke;      // key range of the segment
  int n;           // its key tiles
  int flags;
  int cuts;        // at a unit's head: CTAs that begin inside the unit behind it
  int tree;        // drafted tokens: keys in front of the tree; -1: rows see runs of keys
};
static_assert(sizeof(Segment) == 48, "Segment is 12 int32");
enum { kPrefix = 1, kHead = 2, kWhole = 4 };

// Drafted tokens: the values of tile j of a segment, landed at vt, that no row or
// not every row sees, for the products: zeros behind the unit's last key (unwritten
// cache slots may hold anything, and 0 * NaN is NaN) and in place of those that are
// not finite and that some rows do not see, with a mark in `found` (the epilogue
// looks them up).  The walking warp does so under the tile's softmax: done
// by the softmax threads it took a unit's last tile 2000 cycles longer.
__device__ __forceinline__ void clean_values(const Segment& it, int j, uint8_t* vt,
                                             volatile uint32_t* found, uint32_t mark) {
  const int lane = threadIdx.x & 31, key0 = it.kb + j * kKeys;
  const int all_see = it.tree >= 0 ? it.tree : it.pos + 1;
  const bool ragged = all_see < it.ke && key0 + kKeys > all_see;
  if (!ragged && (j < it.n - 1 || it.ke % kKeys == 0)) return;
  const int valid = min(it.ke - key0, kKeys), from = ragged ? max(all_see - key0, 0) : valid;
  // a lane: 16 bytes of every other row
  uint8_t* mine = vt + ((lane >> 3) & 1) * kHalf + ((lane & 7) << 4);
  const int odd = lane >> 4;
#pragma unroll 8
  for (int r = valid + odd; r < kKeys; r += 2)
    *reinterpret_cast<uint4*>(mine + r * 128) = make_uint4(0, 0, 0, 0);
  // (0 x, summed, is 0 where all of them are finite and NaN elsewhere)
  __nv_bfloat162 sum = __float2bfloat162_rn(0.f), zero = sum;
#pragma unroll 8
  for (int r = from + odd; r < valid; r += 2) {
    const uint4 w = *reinterpret_cast<const uint4*>(mine + r * 128);
    sum = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.x), zero, sum);
    sum = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.y), zero, sum);
    sum = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.z), zero, sum);
    sum = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.w), zero, sum);
  }
  if (__low2float(sum) != 0.f || __high2float(sum) != 0.f) {
    for (int r = from + odd; r < valid; r += 2)
      zero_nonfinite(reinterpret_cast<uint4*>(mine + r * 128));
    *found = mark;
  }
  // the PV MMAs read these rows through the async proxy
  ptx::fence_proxy_async_smem();
  __syncwarp();
}

// Drafted tokens: the road of the step (see StepLanes), and a CTA's walk over its
// lane of its pair's part: single units' steps [x, end), then pairs' places [px, pend).
struct Road {
  int64_t single, half, total, pairs;      // steps of single units, their places, all; CTA pairs
  __device__ __forceinline__ int64_t cut(int64_t i) const { return step_cut(i, total, pairs); }
  // where the single units' steps of CTA c begin
  __device__ __forceinline__ int64_t begin(int c) const {
    const int64_t u = min(cut(c >> 1), half);
    return c & 1 ? u + min(cut((c >> 1) + 1), half) : 2 * u;
  }
};
struct LaneWalk {
  int64_t x, end, px, pend;
  int unit;                  // tiled sequence, and its entries
  int pair_unit;             // where the pairs' part begins (-1: it has been entered)
  StepLanes lanes;
  StepSeq seq;
};

// What a lane's walk needs, in shared memory, where one thread walks.  (In registers
// it spilled what the warp needs for reporting landed tiles.)
struct Lane {
  DevStep ds;
  ShapeInfo s;
  StepWork work;
  Road road;
  LaneWalk walk;
};

// Each barrier is waited on in order of its phases and can never run two
// phases ahead of a waiter (the parity of a wait is then unambiguous).
struct Bars {
  uint64_t q_full[2];             // Q of a unit in tensor memory, by buffer
  uint64_t kv_full[kStages];      // a K or V tile landed (TMA)
  uint64_t kv_empty[kStages];     // the MMAs are done with the stage
  uint64_t s_full[2];             // QK^T of a key tile done, by score buffer
  uint64_t p_full[2];             // its P written, V tail rows zeroed, V_j and K_j+2 landed
  uint64_t o_done[2];             // its PV done
  uint64_t o_free;                // a unit's O read: the next unit may overwrite it
  uint64_t drain;                 // every MMA the CTA issued done
  uint64_t published[kSegments];  // a segment is in its slot
  Segment segments[kSegments];
  uint32_t tmem_base;
  int abort_flag;
  Lane lane;                      // drafted tokens
  // a block id outside the pool has been met (set before its K tile lands)
  volatile int missing;
  // k + 1 of the last segment k that held non-finite values of keys which some
  // of its rows see, by k & 1 (every softmax warp has stored segment k before
  // any of them reports a P of k + 1, hence before segment k + 2 has scores)
  // (drafted tokens: by k % kSegments, the walking warp finds them)
  volatile uint32_t nonfinite[kSegments];
};
static_assert(kStages * kTileBytes + (int)sizeof(Bars) <= kStepTileSmem,
              "shared-memory layout overflows its allocation");

// Ring index, from the segment's first, of K_j and V_j of a segment of n tiles.
// The products read the stages in just this order (QK(0) QK(1) PV(0) QK(2) ...),
// so stages are released in index order; each producer warp's indices are at
// most four apart, so when it waits for the release of index i - 4, that of
// i - 8 is over and the parity of its wait is unambiguous.
__device__ __forceinline__ uint32_t ring_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ uint32_t ring_v(int j, int n) {
  return j + 1 < n ? 2 * j + 2 : 2 * n - 1;
}

// The last of n entries whose place is at or before v: 32 places tested at a time by
// the warp (in front of the first segment every round trip counts; against halving,
// in a graph: 64 trees of 32 tokens 185.7 and 184.7 us, a mixed batch of 98 sequences
// 206.2 and 204.3, one tree 49.0 either way).
template <class F>
__device__ __forceinline__ int last_at(int n, int64_t v, F cum) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const bool le = lane * step < n && cum(lo + lane * step) <= v;
    const int k = max(31 - __clz(__ballot_sync(0xffffffffu, le)), 0);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// Walks a CTA's part [x, end) of the line.
struct Walk {
  int64_t x, end;
  int unit;              // tiled sequence
};

template <bool kDraft>
__device__ __forceinline__ bool next_segment(Walk& w, const DevStep& ds, const ShapeInfo& s,
                                             const StepPlan& plan, const StepWork& work,
                                             int64_t ctas, int tpt, Segment& it) {
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
      it.flags = kPrefix;
      it.table = ds.prefix_table;
      it.row = tile * tpt;
      it.n_tok = min(tpt, work.rows - it.row);
      it.pos = ds.prefix_len - 1;
      if (kDraft) it.tree = -1;
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
      it.flags = 0;
      it.table = ds.block_table + (int64_t)e.seq * ds.max_blocks;
      it.row = e.row + tile * tpt;
      it.n_tok = min(tpt, e.n_new - tile * tpt);
      it.pos = seen + tile * tpt;
      if (kDraft) it.tree = e.n_new <= kStepTreeTokens ? seen : -1;
      keys = it.pos + it.n_tok;
    }
    // the unit's tiles [first, last) of this segment
    const int64_t from = w.x - unit0 - kStepTileUnit, to = w.end - unit0 - kStepTileUnit;
    const int first = (int)(from < 0 ? 0 : from);
    const int last = (int)(to < 0 ? 0 : to < n ? to : n);
    w.x = unit0 + n + kStepTileUnit;
    if (first >= last) continue;
    it.flags |= (first == 0 ? kHead : 0) | (first == 0 && last == n ? kWhole : 0);
    it.kb = first * kKeys;
    it.ke = (int)min((int64_t)keys, (int64_t)last * kKeys);
    it.n = last - first;
    it.cuts = 0;
    // (CTA c begins at floor(c total / ctas): the first at or behind p is
    // ceil(p ctas / total))
    if (first == 0 && last < n)
      it.cuts = (int)step_div(w.x * ctas + work.tile_total - 1, work.tile_total) -
                ((int)blockIdx.x + 1);
    return true;
  }
  it.n = 0;
  return false;
}

__device__ __forceinline__ Road draft_road(const DevStep& ds, const ShapeInfo& s,
                                           const StepWork& work) {
  const StepLanes all = ds.work[0];
  Road r;
  r.single = work.tile_prefix + (int64_t)s.H_kv * all.single_len;
  r.half = (r.single + 1) / 2;
  r.total = r.half + (int64_t)s.H_kv * all.pair_len;
  r.pairs = min((int64_t)gridDim.x / 2, r.total);
  return r;
}

__device__ __forceinline__ void enter_unit(LaneWalk& w, const DevStep& ds, const StepPlan& plan,
                                           int unit) {
  w.unit = unit;
  w.lanes = ds.work[1 + unit];
  w.seq = plan.tiled[unit];
}

// (by a warp)
__device__ __forceinline__ void start_lane(Lane* lane, const DevStep& ds, const ShapeInfo& s,
                                           const StepPlan& plan, const StepWork& work) {
  const Road road = draft_road(ds, s, work);
  const int c = (int)blockIdx.x, n = plan.header[kPlanTiled];
  LaneWalk w;
  w.x = road.begin(c);
  w.end = min(road.begin(c + 1), road.single);
  w.px = max(road.cut(c >> 1), road.half) - road.half;
  w.pend = max(road.cut((c >> 1) + 1), road.half) - road.half;
  w.unit = -1;
  w.pair_unit = 0;
  const StepLanes* lanes = ds.work + 1;
  if (w.px < w.pend)
    w.pair_unit =
        last_at(n, step_div(w.px, s.H_kv), [&](int i) { return lanes[i].pair_cum; });
  if (w.end > max(w.x, work.tile_prefix))
    enter_unit(w, ds, plan,
               last_at(n, step_div(max(w.x - work.tile_prefix, (int64_t)0), s.H_kv),
                       [&](int i) { return lanes[i].single_cum; }));
  if ((threadIdx.x & 31) == 0) {
    lane->ds = ds;
    lane->s = s;
    lane->work = work;
    lane->road = road;
    lane->walk = w;
  }
  __syncwarp();
}

__device__ __forceinline__ bool next_segment(Lane* lane, Segment* to) {
  LaneWalk& w = lane->walk;
  const DevStep& ds = lane->ds;
  const ShapeInfo& s = lane->s;
  const StepWork& work = lane->work;
  const Road& road = lane->road;
  const StepPlan plan = step_plan(ds.plan, ds.num_seqs, ds.max_tokens);
  const int tpt = step_tile_tokens(s.g);
  Segment& it = *to;
  // a query tile of a tiled sequence; returns its key tiles
  auto own_tile = [&](int tile) -> int {
    const StepSeq& e = w.seq;
    const int seen = e.ctx - e.n_new;
    it.flags = 0;
    it.table = ds.block_table + (int64_t)e.seq * ds.max_blocks;
    it.row = e.row + tile * tpt;
    it.n_tok = min(tpt, e.n_new - tile * tpt);
    it.pos = seen + tile * tpt;
    it.tree = e.n_new <= kStepTreeTokens ? seen : -1;
    it.ke = it.pos + it.n_tok;
    return step_key_tiles(seen, e.n_new, tpt, tile);
  };
  // its key tiles [first, last) of n for this segment
  auto publish = [&](int first, int last, int n) {
    it.flags |= (first == 0 ? kHead : 0) | (first == 0 && last == n ? kWhole : 0);
    it.kb = first * kKeys;
    it.ke = (int)min((int64_t)it.ke, (int64_t)last * kKeys);
    it.n = last - first;
    it.cuts = 0;
  };
  auto clamp = [](int64_t v, int n) { return (int)(v < 0 ? 0 : v < n ? v : n); };
  while (w.x < w.end) {
    int n;
    int64_t unit0;
    if (w.x < work.tile_prefix) {
      n = work.prefix_tile_steps;
      const int64_t unit = step_div(w.x, n + kStepTileUnit);
      unit0 = unit * (n + kStepTileUnit);
      it.kv_head = (int)step_div(unit, work.prefix_rows);
      const int tile = (int)(unit - (int64_t)it.kv_head * work.prefix_rows);
      it.flags = kPrefix;
      it.table = ds.prefix_table;
      it.row = tile * tpt;
      it.n_tok = min(tpt, work.rows - it.row);
      it.pos = ds.prefix_len - 1;
      it.tree = -1;
      it.ke = ds.prefix_len;
    } else {
      const int64_t v = w.x - work.tile_prefix;
      while (v >= (int64_t)s.H_kv * ((int64_t)w.lanes.single_cum + w.lanes.single_len))
        enter_unit(w, ds, plan, w.unit + 1);
      const int64_t base = (int64_t)s.H_kv * w.lanes.single_cum;
      it.kv_head = (int)step_div(v - base, w.lanes.single_len);
      unit0 = work.tile_prefix + base + (int64_t)it.kv_head * w.lanes.single_len;
      const int seen = w.seq.ctx - w.seq.n_new;
      int tile = 2 * step_pairs(seen, w.seq.n_new, tpt);
      n = step_key_tiles(seen, w.seq.n_new, tpt, tile);
      while (w.x - unit0 >= n + kStepTileUnit) {
        unit0 += n + kStepTileUnit;
        n = step_key_tiles(seen, w.seq.n_new, tpt, ++tile);
      }
      own_tile(tile);
    }
    const int64_t key0 = unit0 + kStepTileUnit;
    const int first = clamp(w.x - key0, n), last = clamp(w.end - key0, n);
    w.x = key0 + n;
    if (first >= last) continue;
    publish(first, last, n);
    if (first == 0 && last < n) {
      // CTAs that begin in front of the unit's end: the first that does not
      int lo = (int)blockIdx.x + 1, hi = 2 * (int)road.pairs;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (road.begin(mid) >= w.x) hi = mid;
        else lo = mid + 1;
      }
      it.cuts = lo - ((int)blockIdx.x + 1);
    }
    return true;
  }
  while (w.px < w.pend) {
    if (w.pair_unit >= 0) {
      enter_unit(w, ds, plan, w.pair_unit);
      w.pair_unit = -1;
    }
    while (w.px >= (int64_t)s.H_kv * ((int64_t)w.lanes.pair_cum + w.lanes.pair_len))
      enter_unit(w, ds, plan, w.unit + 1);
    const int64_t base = (int64_t)s.H_kv * w.lanes.pair_cum;
    it.kv_head = (int)step_div(w.px - base, w.lanes.pair_len);
    int64_t unit0 = base + (int64_t)it.kv_head * w.lanes.pair_len;
    const int seen = w.seq.ctx - w.seq.n_new;
    int pair = 0, both = step_key_tiles(seen, w.seq.n_new, tpt, 1);
    while (w.px - unit0 >= both + kStepTileUnit) {
      unit0 += both + kStepTileUnit;
      both = step_key_tiles(seen, w.seq.n_new, tpt, 2 * ++pair + 1);
    }
    // (the first tile of a pair may have fewer keys: its lane is empty behind them)
    const int n = own_tile(2 * pair + ((int)blockIdx.x & 1));
    const int64_t key0 = unit0 + kStepTileUnit;
    const int first = clamp(w.px - key0, n), last = clamp(w.pend - key0, n);
    w.px = key0 + both;
    if (first >= last) continue;
    publish(first, last, n);
    // pairs that begin in front of this tile's end
    if (first == 0 && last < n)
      it.cuts = ((int)step_div((key0 + n + road.half) * road.pairs + road.total - 1, road.total) -
                 (((int)blockIdx.x >> 1) + 1)) | kSpillsApart;
    return true;
  }
  it.n = 0;
  return false;
}

// Wait for a phase of a barrier; false when it gave up or another role did.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity,
                                           volatile int* abort_flag) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (*abort_flag || clock64() - t0 > kWaitLimit) return false;
  }
  return true;
}

__device__ __forceinline__ void load8(float* v, const void* p) {
  uint32_t r[8];
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "l"(p)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// A row's 32 floats as 256-bit stores (whole sectors per lane).
__device__ __forceinline__ void store8(float* p, const float* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])),
               "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
               "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
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

// A block id outside the pool has been met.  (Not inlined: in the producers' loop
// these few instructions cost a percent of the kernel.)
__device__ __noinline__ void note_missing(Bars* bars, int32_t* status) {
  atomicCAS(status, 0, kDevBounds);
  bars->missing = 1;
}

// Scores -inf, in tensor memory, for the keys of a tile that have no block.
// (Not inlined, and called from the branch of a wait that gave up: elsewhere in
// the softmax loop these few instructions, which never run otherwise, made a step
// of 512 rows behind 4096 keys take 134 to 137 us instead of 127; so, 128.)
__device__ __noinline__ void hide_keys(uint32_t s_col, const int32_t* table, int key0, int ke,
                                       int B, int num_blocks) {
  const int lane = threadIdx.x & 31, key = key0 + lane * 8;   // blocks are of 8 keys or more
  const bool none =
      lane < kKeys / 8 && key < ke && (uint32_t)table[key / B] >= (uint32_t)num_blocks;
  for (uint32_t m = __ballot_sync(0xffffffffu, none); m; m &= m - 1)
    tmem_fill8(s_col + 8 * (__ffs(m) - 1), -INFINITY);
  tmem_wait_st();
}

// Scores -inf, in tensor memory, of what a drafted row does not see: it sees the
// tile's first `lim` keys and those whose bits its ancestors' set has (null: none),
// bit `by` being the tile's first key.  (In tensor memory and not inlined: as a mask
// over the softmax's registers it spilled 540 bytes, and only a unit's last tile or
// two need it.)
__device__ __noinline__ void hide_others(uint32_t s_col, const uint4* set, int by, int lim) {
  uint32_t own[4];
  draft_window(set ? *set : make_uint4(0, 0, 0, 0), by, own);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int run = lim - 32 * x;
    if (by + 32 * x + 32 <= 0) continue;      // (in front of the tree: every row sees these)
    const uint32_t sees = own[x] | (run <= 0 ? 0u : run >= 32 ? ~0u : (1u << run) - 1u);
    float v[32];
    tmem_ld32(s_col + 32 * x, v);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = sees >> c & 1u ? v[c] : -INFINITY;
    tmem_st32(s_col + 32 * x, v);
  }
  tmem_wait_st();
}

// kDraft: drafted tokens; kLanes: with a road of lanes.
template <bool kDraft, bool kLanes>
__global__ void __launch_bounds__(kThreads, 2)
    step_tile_kernel(const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, DevStep ds, ShapeInfo shp,
                     StepWorkspace ws, const __nv_bfloat16* __restrict__ q,
                     const __nv_bfloat16* __restrict__ v_cache, __nv_bfloat16* __restrict__ o) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  const StepPlan plan = step_plan(ds.plan, ds.num_seqs, ds.max_tokens);
  const StepWork work = step_work(ds, shp, plan);
  const int64_t ctas = !step_matches<kDraft>(ds, shp, plan) ? 0
                       : kLanes ? 2 * draft_road(ds, shp, work).pairs
                                : min((int64_t)gridDim.x, work.tile_total);
  if (blockIdx.x >= ctas) return;
  if (ptx::smem_u32(smem_raw) & 1023) {
    // (the swizzled operand layouts need a 1024-byte aligned base)
    if (threadIdx.x == 0) atomicCAS(ds.status, 0, kDevBounds);
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
      ptx::mbar_init(&bars->p_full[b], 4 * 32 + 1);
      ptx::mbar_init(&bars->o_done[b], 1);
    }
    ptx::mbar_init(&bars->o_free, 4 * 32);
    ptx::mbar_init(&bars->drain, 1);
    for (int i = 0; i < kSegments; ++i) ptx::mbar_init(&bars->published[i], 1);
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&bars->kv_full[s], 1);
      ptx::mbar_init(&bars->kv_empty[s], 1);
    }
    bars->abort_flag = bars->missing = 0;
    for (int i = 0; i < kSegments; ++i) bars->nonfinite[i] = 0;
    ptx::fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // The k-th segment of this CTA; false when there is none (or the wait for it
  // gave up).
  auto segment = [&](uint32_t k, Segment& it) -> bool {
    const bool got =
        wait_phase(&bars->published[k % kSegments], (k / kSegments) & 1, abort_flag);
    if (!__all_sync(0xffffffffu, got)) return false;
    it = bars->segments[k % kSegments];
    return it.n > 0;
  };

  // Every role takes the same segments in the same order.  Ring indices, score
  // buffers and barrier phases carry over from segment to segment: `gi` is the
  // ring index of a segment's K_0, `tc0` the number of its first key tile.
  if (warp >= 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == kKeyWarp || warp == kValueWarp) {
      // --------------------------------------------------------- TMA producers
      // Lane i holds the block id of box i of a tile; -2: no such box; -1: an id
      // outside the pool, which is reported.  (Id -1 makes rows in front of the
      // cache: the copy fills the box with zeros, and the softmax threads take
      // its scores for -inf.)  Ids are loaded a tile ahead, the next segment's
      // while the last tile of the current one is copied.
      const bool leader = elect_one();
      const bool is_k = warp == kKeyWarp;
      const CUtensorMap* map = is_k ? &tmap_k : &tmap_v;
      const int box_rows = B < kKeys ? B : kKeys, boxes = kKeys / box_rows;
      auto look_up = [&](const Segment& u, int j) -> int {
        const int key = u.kb + j * kKeys + lane * box_rows;
        if (lane >= boxes || key >= u.ke) return -2;
        const int blk = u.table[key / B];
        return (uint32_t)blk < (uint32_t)ds.num_blocks ? blk : -1;
      };
      Segment it, nx;
      uint32_t gi = 0, k = 0;
      bool ok = true;
      bool more = segment(0, it);
      int id = more ? look_up(it, 0) : -2;
      while (more && ok) {
        for (int j = 0; ok && j < it.n; ++j) {
          if (__any_sync(0xffffffffu, id == -1)) note_missing(bars, ds.status);
          __syncwarp();
          int id_next = -2;
          if (j + 1 < it.n) {
            id_next = look_up(it, j + 1);
          } else {
            more = segment(++k, nx);
            if (more) id_next = look_up(nx, 0);
          }
          const uint32_t index = gi + (is_k ? ring_k(j) : ring_v(j, it.n));
          const int st = index % kStages;
          if (index >= (uint32_t)kStages)
            ok = wait_phase(&bars->kv_empty[st], ((index / kStages) - 1) & 1, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) {
            if (leader) {
              ptx::report_wait(ds.status, kDevTimeout, is_k ? 72 : 71, (int)index);
              *abort_flag = 1;
            }
            break;
          }
          const uint32_t mask = __ballot_sync(0xffffffffu, id != -2);
          if (leader)
            ptx::mbar_arrive_expect_tx(&bars->kv_full[st],
                                       (uint32_t)(__popc(mask) * box_rows * 256));
          // (a box begins a block, but for blocks of more than 128 keys)
          const int in_block = B > kKeys ? (it.kb + j * kKeys) % B : 0;
          uint8_t* dst = kv_s + st * kTileBytes;
          for (int i = 0; i < boxes; ++i) {
            const int row =
                (__shfl_sync(0xffffffffu, id, i) * shp.H_kv + it.kv_head) * B + in_block;
            if (leader && (mask >> i & 1)) {
              ptx::tma_load_2d(dst + i * box_rows * 128, map, 0, row, &bars->kv_full[st]);
              ptx::tma_load_2d(dst + kHalf + i * box_rows * 128, map, 64, row,
                               &bars->kv_full[st]);
            }
          }
          __syncwarp();
          id = id_next;
        }
        gi += 2 * it.n;
        it = nx;
      }
      // every copy must land before the CTA may exit: a finished walk's tiles
      // were all used; after an abort, wait for both phases of every stage
      if (!ok)
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
        const bool got = wait_phase(bar, parity, abort_flag);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          site = where;
          at = index;
          return false;
        }
        tc_fence_after();
        return true;
      };
      Segment it;
      uint32_t gi = 0, tc0 = 0;
      for (uint32_t k = 0; ok && segment(k, it); ++k) {
        if (!wait_bar(&bars->q_full[k & 1], (k >> 1) & 1, 73, (int)k)) break;
        for (int j = 0; ok && j < 2 && j < it.n; ++j) {
          const uint32_t index = gi + ring_k(j);
          if (!wait_bar(&bars->kv_full[index % kStages], (index / kStages) & 1, 74, (int)index))
            break;
          issue_qk(tc0 + j, index, k & 1);
        }
        // then per key tile j: PV(j) QK(j+2) once its softmax has written P and
        // V_j and K_j+2 have landed (both of which p_full reports)
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
    } else if (warp == kWalkWarp) {
      // ------------------------------------------- the walk, and landed tiles
      Walk walk;
      if constexpr (kLanes) start_lane(&bars->lane, ds, shp, plan, work);
      walk.x = step_cut(blockIdx.x, work.tile_total, ctas);
      walk.end = step_cut(blockIdx.x + 1, work.tile_total, ctas);
      walk.unit = 0;
      if (!kLanes && walk.x >= work.tile_prefix) {
        // the tiled sequence that holds this CTA's first step
        const int64_t v = step_div(walk.x - work.tile_prefix, shp.H_kv);
        int hi = plan.header[kPlanTiled] - 1;
        if constexpr (kDraft)
          walk.unit = hi = last_at(hi + 1, v, [&](int i) { return plan.tiled[i].cum; });
        while (walk.unit < hi) {
          const int mid = (walk.unit + hi + 1) >> 1;
          if (plan.tiled[mid].cum <= v) walk.unit = mid;
          else hi = mid - 1;
        }
      }
      // A slot is written again eight segments later; when a segment's first
      // tile is handled here the softmax warps have left all but the two
      // segments before it, so kAhead + 2 slots are in use at most.
      static_assert(kAhead + 3 <= kSegments, "segment ring");
      uint32_t n_pub = 0;
      bool last = false;
      auto publish = [&] {
        if (last) return;
        Segment& slot = bars->segments[n_pub % kSegments];
        if constexpr (kLanes) {
          int more = 0;
          if (lane == 0) more = next_segment(&bars->lane, &slot);
          last = __shfl_sync(0xffffffffu, more, 0) == 0;
        } else {
          Segment u;
          last = !next_segment<kDraft>(walk, ds, shp, plan, work, ctas, tpt, u);
          if (lane == 0) slot = u;
        }
        if (lane == 0) ptx::mbar_arrive(&bars->published[n_pub % kSegments]);
        ++n_pub;
      };
      uint32_t gi = 0, t = 0;
      bool ok = true;
      for (uint32_t k = 0; ok; ++k) {
        while (n_pub <= k + kAhead && !last) publish();
        Segment it;
        if (!segment(k, it)) break;
        for (int j = 0; ok && j < it.n; ++j, ++t) {
          const uint32_t gv = gi + ring_v(j, it.n), gk = gi + ring_k(j + 2);
          // Once S_j is there, K_j and every tile of smaller ring index but V_j-1
          // have landed, so the stages of V_j and K_j+2 are in the phase before
          // the one that is waited for, or in it; and they stay there until P_j is
          // reported.
          ok = wait_phase(&bars->s_full[t & 1], (t >> 1) & 1, abort_flag);
          ok = ok && wait_phase(&bars->kv_full[gv % kStages], (gv / kStages) & 1, abort_flag);
          if constexpr (kDraft) {
            ok = __all_sync(0xffffffffu, ok);
            if (ok)
              clean_values(it, j, kv_s + (gv % kStages) * kTileBytes,
                           &bars->nonfinite[k % kSegments], k + 1);
          }
          if (ok && j + 2 < it.n)
            ok = wait_phase(&bars->kv_full[gk % kStages], (gk / kStages) & 1, abort_flag);
          // (not before the barrier's last phase is over: it would count for that)
          if (ok && t >= 2) ok = wait_phase(&bars->p_full[t & 1], ((t - 2) >> 1) & 1, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (ok && lane == 0) ptx::mbar_arrive(&bars->p_full[t & 1]);
          if (!ok && lane == 0) {
            ptx::report_wait(ds.status, kDevTimeout, 77, (int)t);
            *abort_flag = 1;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        gi += 2 * it.n;
      }
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
    auto write_q = [&](const Segment& u, uint32_t b) {
      float qv[64];
      uint4* q4 = reinterpret_cast<uint4*>(qv);
      if (tok < u.n_tok) {
        const uint4* src = reinterpret_cast<const uint4*>(
            q + ((int64_t)(u.row + tok) * shp.H_q + u.kv_head * g + hh) * 128);
        if (kDraft && ((uintptr_t)q & 31) == 0) {
          // (whole sectors per lane: 16-byte loads of a row each took 3300 cycles)
#pragma unroll
          for (int i = 0; i < 8; ++i) load8(qv + 8 * i, src + 2 * i);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) q4[i] = src[i];
        }
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
    // drafted tokens: this row's place (looked up with its queries)
    auto place_of = [&](const Segment& u) {
      return kDraft && u.tree >= 0 && tok < u.n_tok ? ds.place[u.row + tok] : 0;
    };
    // With lanes, the softmax runs once over whatever tensor memory holds before the
    // first segment is there: its instructions are in the caches then (one tree of 64
    // behind 32768 keys 54.5 to 52.7 us, 64 behind 2200 183.5 to 180.3; on the line a
    // mixed batch lost 3 us by it).
    Segment it = {};
    int place = 0;
    bool more = true;
    if constexpr (kLanes) {
      it.n = 1;
      it.tree = -1;
    } else {
      more = segment(0, it);
      if (more) {
        place = place_of(it);
        write_q(it, 0);
      }
    }
    for (int k = kLanes ? -1 : 0; more && ok; ++k) {
      const bool dry = kLanes && k < 0;
      // the last key this row sees
      int pos = it.flags & kPrefix ? it.pos : it.pos + tok;
      int all_see = it.pos + 1;              // keys that every row sees
      if constexpr (kDraft) {
        if (it.tree >= 0) {
          all_see = it.tree;
          if (tok < it.n_tok && place != it.pos + tok)
            pos = it.tree - 1;               // and then its ancestors
        }
      }
      float m_ref = -INFINITY, l = 0.f;
      for (int j = 0; j < it.n; ++j) {
        const uint32_t t = tc0 + j;
        // tcgen05.ld/st are warp-collective: every decision below is warp-uniform
        const bool got = dry || wait_phase(&bars->s_full[t & 1], (t >> 1) & 1, abort_flag);
        const uint32_t s_col = lane_base + (t & 1) * kKeys;   // S of the tile; then its P
        const int key0 = it.kb + j * kKeys;
        // (a block id outside the pool is noted before its K tile lands)
        if (!__all_sync(0xffffffffu, got && !bars->missing)) {
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            site = 81;
            at = (int)t;
            break;
          }
          tc_fence_after();
          hide_keys(s_col, it.table, key0, it.ke, B, ds.num_blocks);
        }
        tc_fence_after();
        // this row sees the tile's first `lim` keys: those <= its position and
        // before the unit's end (a prefix of the key tile, possibly empty or all)
        int lim = min(pos + 1, it.ke) - key0;
        if (kDraft && it.tree >= 0 && key0 + kKeys > it.tree) {
          hide_others(s_col, pos < it.tree ? ds.ancestors + it.row + tok : nullptr,
                      key0 - it.tree, lim);
          lim = kKeys;
        }
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
        const bool ragged = all_see < it.ke && key0 + kKeys > all_see;
        if (!kDraft && (ragged || (j == it.n - 1 && (it.ke % kKeys) != 0))) {
          // keys past the unit's end may be anything (unwritten cache slots, and
          // 0 * NaN is NaN): their V rows are zeroed.  So are non-finite values
          // of keys that some rows do not see; the epilogue looks them up.
          const uint32_t gv = gi + ring_v(j, it.n);
          const bool landed =
              wait_phase(&bars->kv_full[gv % kStages], (gv / kStages) & 1, abort_flag);
          if (!__all_sync(0xffffffffu, landed)) {
            ok = false;
            site = 82;
            at = (int)gv;
            break;
          }
          uint8_t* vt = kv_s + (gv % kStages) * kTileBytes;
          const int valid = min(it.ke - key0, kKeys);
          for (int e = row; e < (kKeys - valid) * 16; e += kRows) {
            const int key = valid + e / 16, c = e % 16;
            *reinterpret_cast<uint4*>(vt + (c >> 3) * kHalf + key * 128 + ((c & 7) << 4)) =
                make_uint4(0, 0, 0, 0);
          }
          const int from = ragged ? max(all_see - key0, 0) : valid;
          bool found = false;
          for (int e = row; e < (valid - from) * 16; e += kRows) {
            const int key = from + e / 16, c = e % 16;
            found |= zero_nonfinite(reinterpret_cast<uint4*>(vt + (c >> 3) * kHalf + key * 128 +
                                                             ((c & 7) << 4)));
          }
          if (found) bars->nonfinite[k & 1] = k + 1;
          // the PV MMAs read these rows through the async proxy
          ptx::fence_proxy_async_smem();
        }
        tc_fence_before();
        if (!dry) ptx::mbar_arrive(&bars->p_full[t & 1]);
      }
      if (!ok) break;
      // the next unit's queries, while this one's last products run
      Segment nx;
      more = segment(k + 1, nx);
      if (more) {
        place = place_of(nx);
        write_q(nx, (k + 1) & 1);
      }
      if (dry) {
        it = nx;
        continue;
      }
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
      const bool head = it.flags & kHead, pre = it.flags & kPrefix;
      const bool partial = !(it.flags & kWhole) || ds.prefix_len > 0;
      const int64_t slot = head ? (int64_t)(it.row + tok) * shp.H_q + it.kv_head * g + hh
                                : (int64_t)blockIdx.x * kRows + row;
      __nv_bfloat16* orow = o + slot * 128;
      if (head && row == 0)
        (pre ? ws.pre_cut : ws.own_cut)[(int64_t)it.row * shp.H_kv + it.kv_head] =
            Spills{(int32_t)blockIdx.x + (kDraft && (it.cuts & kSpillsApart) ? 2 : 1), it.cuts};
      float* prow = (head ? (pre ? ws.pre_o : ws.own_o) : ws.tile_o) + slot * 128;
      float* plse = head ? (pre ? ws.pre_lse : ws.own_lse) : ws.tile_lse;
      float ov[128];
#pragma unroll
      for (int c4 = 0; c4 < 4; ++c4) tmem_ld32(lane_base + kOCol + c4 * 32, ov + c4 * 32);
      tmem_wait_ld();
      // O has been read: the next unit's first PV may overwrite it
      tc_fence_before();
      ptx::mbar_arrive(&bars->o_free);
#pragma unroll
      for (int c = 0; c < 128; ++c) ov[c] *= inv;
      if (bars->nonfinite[kDraft ? k % kSegments : k & 1] == (uint32_t)k + 1) {
        // (written before the last P was reported, so before its product)
        const int end = kDraft && it.tree >= 0 ? it.ke : min(it.ke, pos + 1);
        for (int key = max(it.kb, all_see); key < end; ++key) {
          if (kDraft && key > pos &&
              (pos >= it.tree || !draft_bit(ds.ancestors[it.row + tok], key - it.tree)))
            continue;
          const int blk = it.table[key / B];
          if ((uint32_t)blk >= (uint32_t)ds.num_blocks) continue;
          const uint4* src = reinterpret_cast<const uint4*>(
              v_cache + (((int64_t)blk * shp.H_kv + it.kv_head) * B + key % B) * 128);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint4 x = src[c];
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t bad = w[i] & nonfinite2(w[i]);
              ov[8 * c + 2 * i] += __uint_as_float(bad << 16);
              ov[8 * c + 2 * i + 1] += __uint_as_float(bad & 0xffff0000u);
            }
          }
        }
      }
      if (store && !partial) {
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
          uint4 v;
          v.x = ptx::pack_bf16x2(ov[c + 0], ov[c + 1]);
          v.y = ptx::pack_bf16x2(ov[c + 2], ov[c + 3]);
          v.z = ptx::pack_bf16x2(ov[c + 4], ov[c + 5]);
          v.w = ptx::pack_bf16x2(ov[c + 6], ov[c + 7]);
          *reinterpret_cast<uint4*>(orow + c) = v;
        }
      } else if (store) {
#pragma unroll
        for (int c = 0; c < 128; c += 8) store8(prow + c, ov + c);
        plse[slot] = l > 0.f ? m_ref + log2f(l) : -INFINITY;
      }
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
}

}  // namespace

namespace {
template <bool kDraft, bool kLanes>
cudaError_t launch(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w, const void* q,
                   const void* k_cache, const void* v_cache, void* o, cudaStream_t st) {
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
    e = cudaFuncGetAttributes(&fa, step_tile_kernel<kDraft, kLanes>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(step_tile_kernel<kDraft, kLanes>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kStepTileSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(step_tile_kernel<kDraft, kLanes>,
                               cudaFuncAttributePreferredSharedMemoryCarveout,
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
  return cudaLaunchKernelEx(&cfg, step_tile_kernel<kDraft, kLanes>, tk, tv, ds, s, w,
                            (const __nv_bfloat16*)q, (const __nv_bfloat16*)v_cache,
                            (__nv_bfloat16*)o);
}
}  // namespace

cudaError_t launch_step_tile(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w,
                             const void* q, const void* k_cache, const void* v_cache, void* o,
                             cudaStream_t st) {
  // Pairs of query tiles pay where a sequence has more than one and keys enough for
  // the second one's to be read from HBM again (64 trees of 64 tokens, groups of 4:
  // 221 us without, 187 with, behind 2200 keys, 134 and 129 behind 1100); the walk of
  // the lanes costs the others (behind 300, 84.5 and 88.5; trees of one tile behind
  // up to 8192, 190 and 197), and what the tables can hold is all the host knows: keys
  // of a sequence, and its rows on average.
  const bool lanes = ds.place && (int64_t)ds.max_tokens * s.g > (int64_t)kRows * ds.num_seqs &&
                     (int64_t)ds.max_blocks * s.B >= 2 * kStepPairTiles * kKeys;
  auto fn = !ds.place ? launch<false, false> : lanes ? launch<true, true> : launch<true, false>;
  return fn(ds, s, w, q, k_cache, v_cache, o, st);
}

}  // namespace rbkv
