// Streaming attention of a step: units of at most 16 packed query rows (a
// sequence's new tokens x the heads of one KV group) over the sequence's own
// keys; every cached K/V byte is read once, so HBM bounds it.
//
// The units' 64-key tiles lie on one line that is cut evenly over the CTAs
// (rbkv_step.h): two CTAs per SM, each with
//  - a producer warp that streams K and V tiles through the block table with
//    TMA (128-byte swizzle) into a 3-stage ring of 32 KB stages;
//  - four consumer warps that share every tile, 16 keys each: S = Q K^T with
//    m16n8k16 MMAs (the rows padded to 16; the contraction is tiny, so they
//    only lift the bound that CUDA cores would set), an online softmax in
//    registers, O += P V; at the end of a segment their (max, sum, O) are
//    merged through shared memory, half of the head dim at a time (16 KB of
//    scratch beside the ring leaves room for two CTAs per SM).
// Every wait is bounded; on timeout the kernel records RBKV_ERR_TIMEOUT and
// returns.
#include <algorithm>
#include <atomic>

#include "rbkv_step.h"
#include "rbkv_ptx.cuh"

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace rbkv {

namespace {

constexpr int kStages = 3;
constexpr int kConsumers = 4;
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kKeys = kStepStreamKeys;
constexpr int kGroup = 16 * 256;              // 16 keys of K or V, head_dim 128
constexpr int kTile = kKeys * 256;            // K or V tile
constexpr int kStage = 2 * kTile;             // K + V
constexpr int kRows = kStepPackedRows;
constexpr int kScratch = kConsumers * kRows * 64 * 4;   // [warp][row][64] fp32
constexpr int kMl = kConsumers * kRows * 2 * 4;         // (max, sum) per warp and row
constexpr int kSegments = 4;            // published segments; more than kStages
static_assert(kSegments > kStages && (2 * kStages + kSegments) % 2 == 0, "segment ring");
constexpr int kSmemBytes =
    kStages * kStage + kScratch + kMl + (2 * kStages + kSegments) * 8 + kSegments * 32 + 16;
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
constexpr long long kWaitLimit = 4000000000LL;   // ~2 s of SM clock
constexpr float kLog2e = 1.4426950408889634f;

// Byte offset, inside one K or V tile, of the 16-byte chunk holding elements
// d..d+7 (d % 8 == 0) of key row `key`: groups of 16 keys, each as two halves
// of the head dim, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_off(int key, int d) {
  const int chunk = (d & 63) >> 3;
  return (key >> 4) * kGroup + (d >> 6) * (kGroup / 2) + (key & 15) * 128 +
         ((chunk ^ (key & 7)) << 4);
}

// One segment of a unit, as the producer publishes it to the consumers.
struct __align__(16) Segment {
  int row, n_tok;        // first row and tokens of the unit
  int kv_head;
  int tile, tiles;       // first key tile, and number of them (0: no more segments)
  int keys;              // keys of the unit's last row
  int diag;              // keys of its first row (the prefix: every row sees all)
  int flags;
};
static_assert(sizeof(Segment) == 32, "Segment is 8 int32");
enum { kPrefix = 1, kHead = 2, kWhole = 4 };

struct Shared {
  uint8_t* stages;
  float* scratch;
  float* ml;
  uint64_t* full;
  uint64_t* empty;
  uint64_t* published;
  Segment* segments;
  volatile int* abort_flag;
};

__device__ __forceinline__ Shared carve(uint8_t* raw) {
  Shared s;
  s.stages = raw;
  s.scratch = reinterpret_cast<float*>(raw + kStages * kStage);
  s.ml = s.scratch + kScratch / 4;
  s.full = reinterpret_cast<uint64_t*>(s.ml + kMl / 4);
  s.empty = s.full + kStages;
  s.published = s.empty + kStages;
  s.segments = reinterpret_cast<Segment*>(s.published + kSegments);
  s.abort_flag = reinterpret_cast<volatile int*>(s.segments + kSegments);
  return s;
}

// The producer's walk over its CTA's part [x, end) of the line.  Units follow
// one another without a division: the next KV head, then the next sequence,
// whose entry is loaded one sequence ahead.
struct Walk {
  int64_t end, unit0;    // end of the part; the unit's place on the line
  int unit, kv_head;
  StepSeq cur, next;
  const int32_t* table;

  __device__ __forceinline__ void enter(const DevStep& ds, const ShapeInfo& s,
                                        const StepPlan& plan, const StepWork& work) {
    if (unit < plan.header[kPlanStreamed]) {
      next = plan.streamed[min(unit + 1, ds.num_seqs - 1)];
      unit0 = (int64_t)s.H_kv * cur.cum + (int64_t)kv_head * (cur.tiles + kStepStreamUnit);
      table = ds.block_table + (int64_t)cur.seq * ds.max_blocks;
    } else {
      cur.row = 0;
      cur.n_new = plan.header[kPlanRows];
      cur.ctx = ds.prefix_len;
      cur.tiles = work.prefix_stream_tiles;
      unit0 = work.stream_own + (int64_t)kv_head * (cur.tiles + kStepStreamUnit);
      table = ds.prefix_table;
    }
  }

  // (every lane of the warp calls it: the search tests 32 places at a time)
  __device__ __forceinline__ void start(int64_t x, const DevStep& ds, const ShapeInfo& s,
                                        const StepPlan& plan, const StepWork& work, int lane) {
    int64_t base = work.stream_own;
    unit = plan.header[kPlanStreamed];
    int len = work.prefix_stream_tiles + kStepStreamUnit;
    if (x < work.stream_own) {
      // the last sequence at or before x
      const int32_t v = (int32_t)(x / s.H_kv);
      int lo = 0, left = unit;
      while (left > 1) {
        const int step = (left + 31) >> 5;
        const bool le = lane * step < left && plan.streamed[lo + lane * step].cum <= v;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));   // lane 0 always holds
        lo += k * step;
        left = min(step, left - k * step);
      }
      unit = lo;
      cur = plan.streamed[unit];
      base = (int64_t)s.H_kv * cur.cum;
      len = cur.tiles + kStepStreamUnit;
    }
    kv_head = (int)(x - base) / len;    // (a sequence's line fits 32 bits with its heads)
    enter(ds, s, plan, work);
  }

  // The segment of the unit in [x, end), and on to the next unit; false when
  // the part has no tile of it.
  __device__ __forceinline__ bool segment(int64_t x, Segment& g, const int32_t*& ids,
                                          const DevStep& ds, const ShapeInfo& s,
                                          const StepPlan& plan, const StepWork& work,
                                          int64_t& x_next) {
    const bool prefix = unit >= plan.header[kPlanStreamed];
    const int n = cur.tiles;
    g.row = cur.row;
    g.n_tok = cur.n_new;
    g.kv_head = kv_head;
    g.keys = cur.ctx;
    g.diag = prefix ? cur.ctx : cur.ctx - cur.n_new + 1;
    ids = table;
    const int64_t from = x - unit0 - kStepStreamUnit, to = end - unit0 - kStepStreamUnit;
    const int last = (int)(to < 0 ? 0 : to < n ? to : n);
    g.tile = (int)(from < 0 ? 0 : from);
    g.tiles = last - g.tile;
    g.flags = (prefix ? kPrefix : 0) | (g.tile == 0 ? kHead : 0) |
              (g.tile == 0 && last == n ? kWhole : 0);
    x_next = unit0 + n + kStepStreamUnit;
    if (x_next < end) {
      if (++kv_head == s.H_kv) {
        kv_head = 0;
        ++unit;
        cur = next;
      }
      enter(ds, s, plan, work);
    }
    return g.tiles > 0;
  }
};

// The caches as tensor maps: boxes of 64 keys or a block, and of 16 keys.
struct Maps {
  CUtensorMap k, v, k_one, v_one;
};

__global__ void __launch_bounds__(kThreads, 2)
    step_stream_kernel(const __grid_constant__ Maps maps, DevStep ds, ShapeInfo shp,
                       StepWorkspace ws, const __nv_bfloat16* __restrict__ q,
                       __nv_bfloat16* __restrict__ o, int first) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (first) ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  Shared sm = carve(smem_raw);
  volatile int& abort_flag = *sm.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = shp.g, B = shp.B, H_kv = shp.H_kv;
  const StepPlan plan = step_plan(ds.plan, ds.num_seqs, ds.max_tokens);
  const StepWork work = step_work(ds, shp, plan);
  const int64_t ctas = min((int64_t)gridDim.x, work.stream_total);
  if ((ptx::smem_u32(smem_raw) & 1023) || blockIdx.x >= ctas) {
    // (the swizzled tile layout needs a 1024-byte aligned base)
    if (threadIdx.x == 0 && blockIdx.x < ctas) atomicCAS(ds.status, 0, kDevBounds);
    ptx::pdl_wait_previous();   // the grid's completion still covers its predecessor
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&sm.full[s], 1);
      ptx::mbar_init(&sm.empty[s], kConsumers);
    }
    for (int s = 0; s < kSegments; ++s) ptx::mbar_init(&sm.published[s], 1);
    abort_flag = 0;
    ptx::fence_barrier_init();
  }
  __syncthreads();

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    Walk walk;
    walk.end = step_cut(blockIdx.x + 1, work.stream_total, ctas);
    int64_t x = step_cut(blockIdx.x, work.stream_total, ctas);
    walk.start(x, ds, shp, plan, work, lane);
    if (lane == 0) {
      const int box_rows = B < kKeys ? B : kKeys;
      Segment it, nx;
      const int32_t *ids, *nx_ids;
      auto next = [&](Segment& g, const int32_t*& p) {
        while (x < walk.end) {
          int64_t to;
          const bool some = walk.segment(x, g, p, ds, shp, plan, work, to);
          x = to;
          if (some) return;
        }
        g.tiles = 0;
      };
      // block ids of a tile's boxes (none past the unit's last key), loaded
      // one tile ahead so that their latency hides behind the ring's waits
      int32_t blk[kKeys / 8];
      auto look = [&](const Segment& g, const int32_t* p, int j) {
        const int k0 = (g.tile + j) * kKeys;
#pragma unroll
        for (int i = 0; i < kKeys / 8; ++i)
          if (i * box_rows < kKeys && k0 + i * box_rows < g.keys)
            blk[i] = p[(k0 + i * box_rows) / B];
      };
      uint32_t idx = 0, seg = 0;
      bool stop = false;
      next(it, ids);
      if (it.tiles) look(it, ids, 0);
      for (;; ++seg) {
        // (a slot of the segment ring is free again once a tile three before
        // the next one was released: kSegments > kStages)
        sm.segments[seg % kSegments] = it;
        ptx::mbar_arrive(&sm.published[seg % kSegments]);
        if (it.tiles == 0 || stop) break;
        next(nx, nx_ids);
        for (int j = 0; j < it.tiles; ++j, ++idx) {
          const int s = idx % kStages;
          if (abort_flag ||
              (idx >= (uint32_t)kStages &&
               !ptx::mbar_wait(&sm.empty[s], ((idx / kStages) - 1) & 1, kWaitLimit))) {
            ptx::report_wait(ds.status, kDevTimeout, 61, (int)idx);
            abort_flag = 1;
            stop = true;
            break;
          }
          const int k0 = (it.tile + j) * kKeys;
          uint8_t* kdst = sm.stages + s * kStage;
          uint8_t* vdst = kdst + kTile;
          // boxes of box_rows keys; of a box that the unit's keys end in, only
          // the 16-key groups that hold some (whole boxes would read 32 keys
          // too many per unit on average: a tenth of the traffic at 256 keys)
          uint32_t keys = 0;
#pragma unroll
          for (int i = 0; i < kKeys / 8; ++i) {
            const int left = it.keys - k0 - i * box_rows;
            if (i * box_rows < kKeys && left > 0) {
              if (blk[i] < 0 || blk[i] >= ds.num_blocks)
                atomicCAS(ds.status, 0, kDevBounds);
              else
                keys += left >= box_rows ? box_rows : min(box_rows, (left + 15) & ~15);
            }
          }
          ptx::mbar_arrive_expect_tx(&sm.full[s], keys * 512);
#pragma unroll
          for (int i = 0; i < kKeys / 8; ++i) {
            const int left = it.keys - k0 - i * box_rows;
            if (i * box_rows < kKeys && left > 0 && blk[i] >= 0 && blk[i] < ds.num_blocks) {
              const int row = (blk[i] * H_kv + it.kv_head) * B + ((k0 + i * box_rows) % B);
              if (box_rows < 16) {
                // 8-key blocks: half a group per copy
                const int off = (i >> 1) * kGroup + (i & 1) * 8 * 128;
                ptx::tma_load_2d(kdst + off, &maps.k, 0, row, &sm.full[s]);
                ptx::tma_load_2d(kdst + off + kGroup / 2, &maps.k, 64, row, &sm.full[s]);
                ptx::tma_load_2d(vdst + off, &maps.v, 0, row, &sm.full[s]);
                ptx::tma_load_2d(vdst + off + kGroup / 2, &maps.v, 64, row, &sm.full[s]);
              } else if (left > box_rows - 16) {
                ptx::tma_load_4d(kdst + i * box_rows * 256, &maps.k, row >> 4, &sm.full[s]);
                ptx::tma_load_4d(vdst + i * box_rows * 256, &maps.v, row >> 4, &sm.full[s]);
              } else {
                for (int f = 0; f < left; f += 16) {
                  const int at = (i * box_rows + f) * 256;
                  ptx::tma_load_4d(kdst + at, &maps.k_one, (row + f) >> 4, &sm.full[s]);
                  ptx::tma_load_4d(vdst + at, &maps.v_one, (row + f) >> 4, &sm.full[s]);
                }
              }
            }
          }
          if (j + 1 < it.tiles) look(it, ids, j + 1);
          else if (nx.tiles) look(nx, nx_ids, 0);
        }
        if (stop) break;
        it = nx;
        ids = nx_ids;
      }
      // let every load this CTA issued land before the CTA can exit
      for (uint32_t t = idx > (uint32_t)kStages ? idx - kStages : 0; t < idx; ++t)
        ptx::mbar_wait(&sm.full[t % kStages], (t / kStages) & 1, kWaitLimit);
    }
    ptx::pdl_wait_previous();
    return;
  }

  // -------------------------------------------------------------- consumers
  const float qk_scale = shp.scale * kLog2e;
  const int r0 = lane >> 2, r1 = r0 + 8;      // fragment rows: token r / g, head r % g
  const int t0 = r0 / g, t1 = r1 / g;
  const int cq = (lane & 3) * 2;              // fragment column pair
  const uint32_t stages_u32 = ptx::smem_u32(sm.stages);
  uint32_t tile_base = 0;

  // the unit's query rows as m16n8k16 A fragments; rows past its end are zero
  auto load_q = [&](const Segment& u, uint32_t(&dst)[8][4]) {
    const bool live0 = t0 < u.n_tok, live1 = t1 < u.n_tok;
    const uint32_t* q0 = reinterpret_cast<const uint32_t*>(
        q + ((int64_t)(u.row + t0) * shp.H_q + u.kv_head * g + r0 % g) * 128);
    const uint32_t* q1 = reinterpret_cast<const uint32_t*>(
        q + ((int64_t)(u.row + t1) * shp.H_q + u.kv_head * g + r1 % g) * 128);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const int c = (kk * 16 + cq) >> 1;
      dst[kk][0] = live0 ? __ldg(q0 + c) : 0u;
      dst[kk][1] = live1 ? __ldg(q1 + c) : 0u;
      dst[kk][2] = live0 ? __ldg(q0 + c + 4) : 0u;
      dst[kk][3] = live1 ? __ldg(q1 + c + 4) : 0u;
    }
  };
  uint32_t qa[8][4];
  // the next published segment; one without tiles ends the walk
  uint32_t seg = 0;
  auto take = [&](Segment& u) -> bool {
    if (!ptx::mbar_wait(&sm.published[seg % kSegments], (seg / kSegments) & 1, kWaitLimit)) {
      if (lane == 0) {
        ptx::report_wait(ds.status, kDevTimeout, 63, (int)seg);
        abort_flag = 1;
      }
      u.tiles = 0;
    } else {
      u = sm.segments[seg % kSegments];
    }
    ++seg;
    return __all_sync(0xffffffffu, u.tiles > 0);
  };
  Segment it;
  bool more = take(it);
  if (ptx::named_bar_or(1, kConsumers * 32, abort_flag != 0)) more = false;
  if (more) load_q(it, qa);

  while (more) {
    const int nt = it.tiles;
    const int nrg = it.n_tok * g;
    const int lim0 = min(it.keys, it.diag + t0), lim1 = min(it.keys, it.diag + t1);
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float acc_o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc_o[i][0] = acc_o[i][1] = acc_o[i][2] = acc_o[i][3] = 0.f;

    // every warp takes 16 keys (rows 16*warp .. 16*warp+15) of every tile, so
    // each warp consumes the stages strictly in order
    const int wk = warp * 16;
    for (int j = 0; j < nt && !abort_flag; ++j) {
      const uint32_t idx = tile_base + j;
      const int s = idx % kStages;
      if (!ptx::mbar_wait(&sm.full[s], (idx / kStages) & 1, kWaitLimit)) {
        // give up on this unit; the merge barriers below are still met by
        // every consumer warp, then all of them leave together
        if (lane == 0) {
          ptx::report_wait(ds.status, kDevTimeout, 62, (int)idx);
          abort_flag = 1;
        }
        __syncwarp();
        break;
      }
      const int k0 = (it.tile + j) * kKeys;
      const int valid = min(kKeys, it.keys - k0) - wk;   // valid keys of this warp's 16
      const uint32_t kt = stages_u32 + s * kStage;
      const uint32_t vt = kt + kTile;
      if (valid < 16) {
        // rows past the unit's last key may hold anything (unwritten cache
        // slots, stale tiles): zero this warp's such V rows so 0 * V stays 0
        uint8_t* vrow = sm.stages + s * kStage + kTile + warp * kGroup;
        const int from = valid < 0 ? 0 : valid;
        for (int e = lane; e < (16 - from) * 16; e += 32) {
          const int key = from + e / 16, c = e % 16;
          *reinterpret_cast<uint4*>(vrow + (c >> 3) * (kGroup / 2) + key * 128 +
                                    ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      if (valid > 0) {
        // S = Q K^T over this warp's 16 keys: 2 n-tiles of 8 keys
        float sc[2][4];
        sc[0][0] = sc[0][1] = sc[0][2] = sc[0][3] = 0.f;
        sc[1][0] = sc[1][1] = sc[1][2] = sc[1][3] = 0.f;
        const int mi = lane >> 3;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const int key = wk + (mi >> 1) * 8 + (lane & 7);
          const int d = kk * 16 + (mi & 1) * 8;
          uint32_t b0, b1, b2, b3;
          ptx::ldsm_x4(kt + tile_off(key, d), b0, b1, b2, b3);
          ptx::mma_bf16_16816(sc[0], qa[kk], b0, b1);
          ptx::mma_bf16_16816(sc[1], qa[kk], b2, b3);
        }
        // scale, mask keys past each row's limit, online softmax (rows r0 and r1)
        const int valid0 = min(kKeys, lim0 - k0) - wk, valid1 = min(kKeys, lim1 - k0) - wk;
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int key = n * 8 + cq;
          sc[n][0] = key < valid0 ? sc[n][0] * qk_scale : -INFINITY;
          sc[n][1] = key + 1 < valid0 ? sc[n][1] * qk_scale : -INFINITY;
          sc[n][2] = key < valid1 ? sc[n][2] * qk_scale : -INFINITY;
          sc[n][3] = key + 1 < valid1 ? sc[n][3] * qk_scale : -INFINITY;
          mx0 = fmaxf(mx0, fmaxf(sc[n][0], sc[n][1]));
          mx1 = fmaxf(mx1, fmaxf(sc[n][2], sc[n][3]));
        }
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
        const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
        // a row with no visible key so far keeps max -inf: its terms are 0
        const float b0 = mn0 == -INFINITY ? 0.f : mn0, b1 = mn1 == -INFINITY ? 0.f : mn1;
        const float c0 = ptx::ex2(m0 - b0), c1 = ptx::ex2(m1 - b1);
        m0 = mn0;
        m1 = mn1;
        const float p00 = ptx::ex2(sc[0][0] - b0), p01 = ptx::ex2(sc[0][1] - b0);
        const float p02 = ptx::ex2(sc[0][2] - b1), p03 = ptx::ex2(sc[0][3] - b1);
        const float p10 = ptx::ex2(sc[1][0] - b0), p11 = ptx::ex2(sc[1][1] - b0);
        const float p12 = ptx::ex2(sc[1][2] - b1), p13 = ptx::ex2(sc[1][3] - b1);
        l0 = l0 * c0 + (p00 + p01 + p10 + p11);
        l1 = l1 * c1 + (p02 + p03 + p12 + p13);
        // the weights enter the value product as bf16 (its operand type): each
        // off by at most 2^-8 of itself; their sum above stays fp32
        uint32_t pa[4];
        pa[0] = ptx::pack_bf16x2(p00, p01);
        pa[1] = ptx::pack_bf16x2(p02, p03);
        pa[2] = ptx::pack_bf16x2(p10, p11);
        pa[3] = ptx::pack_bf16x2(p12, p13);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          acc_o[i][0] *= c0;
          acc_o[i][1] *= c0;
          acc_o[i][2] *= c1;
          acc_o[i][3] *= c1;
        }
        // O += P V over the 16 keys: 16 n-tiles of 8 head-dim columns
#pragma unroll
        for (int dp2 = 0; dp2 < 8; ++dp2) {
          const int key = wk + (mi & 1) * 8 + (lane & 7);
          const int d = dp2 * 16 + (mi >> 1) * 8;
          uint32_t v0, v1, v2, v3;
          ptx::ldsm_x4_t(vt + tile_off(key, d), v0, v1, v2, v3);
          ptx::mma_bf16_16816(acc_o[2 * dp2], pa, v0, v1);
          ptx::mma_bf16_16816(acc_o[2 * dp2 + 1], pa, v2, v3);
        }
      }
      __syncwarp();
      if (lane == 0) {
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&sm.empty[s]);
      }
    }
    tile_base += nt;

    // the next segment and its queries, loaded while this one is merged
    const Segment cur = it;
    more = !abort_flag && take(it);
    uint32_t qn[8][4];
    if (more) load_q(it, qn);

    // ---- merge the four warps' states and write the segment's result -------
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if ((lane & 3) == 0) {
      sm.ml[(warp * kRows + r0) * 2 + 0] = m0;
      sm.ml[(warp * kRows + r0) * 2 + 1] = l0;
      sm.ml[(warp * kRows + r1) * 2 + 0] = m1;
      sm.ml[(warp * kRows + r1) * 2 + 1] = l1;
    }
    ptx::named_bar_sync(1, kConsumers * 32);
    float M0 = -INFINITY, M1 = -INFINITY, L0 = 0.f, L1 = 0.f;
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) {
      M0 = fmaxf(M0, sm.ml[(w * kRows + r0) * 2]);
      M1 = fmaxf(M1, sm.ml[(w * kRows + r1) * 2]);
    }
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) {
      const float mw0 = sm.ml[(w * kRows + r0) * 2], mw1 = sm.ml[(w * kRows + r1) * 2];
      if (mw0 != -INFINITY) L0 += ptx::ex2(mw0 - M0) * sm.ml[(w * kRows + r0) * 2 + 1];
      if (mw1 != -INFINITY) L1 += ptx::ex2(mw1 - M1) * sm.ml[(w * kRows + r1) * 2 + 1];
    }
    const float f0 = (m0 == -INFINITY || L0 == 0.f) ? 0.f : ptx::ex2(m0 - M0) / L0;
    const float f1 = (m1 == -INFINITY || L1 == 0.f) ? 0.f : ptx::ex2(m1 - M1) / L1;
    // where row r of the segment goes: O itself when nothing is to be joined,
    // the unit's rows of the workspace, or this CTA's spill rows
    const bool head = cur.flags & kHead, pre = cur.flags & kPrefix;
    const bool direct = (cur.flags & kWhole) && ds.prefix_len == 0;
    float* part = head ? (pre ? ws.pre_o : ws.own_o) : ws.stream_o;
    float* lse = head ? (pre ? ws.pre_lse : ws.own_lse) : ws.stream_lse;
    auto place = [&](int r) -> int64_t {
      return head ? (int64_t)(cur.row + r / g) * shp.H_q + cur.kv_head * g + r % g
                  : (int64_t)blockIdx.x * kRows + r;
    };
    const int t = threadIdx.x;   // 0..127
    float* scr = sm.scratch + warp * kRows * 64;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      // each warp stores its rescaled O, 64 columns (8-column groups permuted
      // by the row, for the banks); then all four are summed per element
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int a = hf * 8 + i;
        if (r0 < nrg)
          *reinterpret_cast<float2*>(scr + r0 * 64 + ((i ^ (r0 & 7)) << 3) + cq) =
              make_float2(acc_o[a][0] * f0, acc_o[a][1] * f0);
        if (r1 < nrg)
          *reinterpret_cast<float2*>(scr + r1 * 64 + ((i ^ (r1 & 7)) << 3) + cq) =
              make_float2(acc_o[a][2] * f1, acc_o[a][3] * f1);
      }
      ptx::named_bar_sync(1, kConsumers * 32);
      for (int e = t; e < nrg * 16; e += kConsumers * 32) {
        const int r = e >> 4, c4 = (e & 15) * 4;
        const int at = r * 64 + (((c4 >> 3) ^ (r & 7)) << 3) + (c4 & 7);
        float4 a = *reinterpret_cast<const float4*>(sm.scratch + at);
#pragma unroll
        for (int w = 1; w < kConsumers; ++w) {
          const float4 b = *reinterpret_cast<const float4*>(sm.scratch + w * kRows * 64 + at);
          a.x += b.x;
          a.y += b.y;
          a.z += b.z;
          a.w += b.w;
        }
        const int64_t to = place(r) * 128 + hf * 64 + c4;
        if (direct) {
          uint2 packed;
          packed.x = ptx::pack_bf16x2(a.x, a.y);
          packed.y = ptx::pack_bf16x2(a.z, a.w);
          *reinterpret_cast<uint2*>(o + to) = packed;
        } else {
          *reinterpret_cast<float4*>(part + to) = a;
        }
      }
      if (hf == 0) ptx::named_bar_sync(1, kConsumers * 32);
    }
    if (!direct && warp == 0 && (lane & 3) == 0) {
      if (r0 < nrg) lse[place(r0)] = L0 > 0.f ? M0 + log2f(L0) : -INFINITY;
      if (r1 < nrg) lse[place(r1)] = L1 > 0.f ? M1 + log2f(L1) : -INFINITY;
    }
    // all consumer warps leave together if anyone gave up
    if (ptx::named_bar_or(1, kConsumers * 32, abort_flag != 0)) break;
    if (more) {
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
#pragma unroll
        for (int x = 0; x < 4; ++x) qa[kk][x] = qn[kk][x];
    }
  }
  ptx::pdl_wait_previous();
}

// ---------------------------------------------------------------------------
// The join: one warp per (row, query head), four columns per lane.
// ---------------------------------------------------------------------------
// O = sum_i 2^(L_i - M) O_i / sum_i 2^(L_i - M) over the row's partial
// outputs: its own part and the prefix's, each with the spills of the CTAs
// whose cuts fall inside its unit.  The cuts are a formula; a block works out
// those of its row and KV heads once, one thread each, and its warps then
// join the heads: lane i weighs source i, all lanes add four columns of each.
// Bound by the partials' traffic (from L2, they were just written).
constexpr int kJoinWarps = 4;
constexpr int kJoinHeads = 8;     // query heads of a block

// Spills of a unit that a row joins: CTAs [first, first + n).
struct Spills {
  int first, n;
  bool cut;       // the unit was cut between its tiles
};

// For a unit at `begin` of a line, of a fixed length `unit` and `tiles` key
// tiles, `row_tiles` of them seen by the row (a unit's two query tiles may see
// different numbers).
__device__ __forceinline__ Spills spills_of(int64_t begin, int unit, int tiles, int row_tiles,
                                            int64_t total, int ctas) {
  Spills s = {0, 0, false};
  // the first cut behind the unit's first tile, from an estimate that is off
  // by one at most
  int c = (int)((float)begin * (float)ctas / (float)total) - 1;
  c = c < 0 ? 0 : c;
  while (c < ctas && step_cut(c, total, ctas) <= begin + unit) ++c;
  s.first = c;
  // (a CTA's part is at least one long: tiles bounds the cuts)
  for (; c < ctas; ++c) {
    const int64_t tile = step_cut(c, total, ctas) - begin - unit;   // first tile behind it
    if (tile >= tiles) break;
    s.cut = true;
    if (tile < row_tiles) ++s.n;
  }
  return s;
}

__global__ void __launch_bounds__(kJoinWarps * 32)
    step_combine_kernel(DevStep ds, ShapeInfo shp, StepWorkspace ws,
                        __nv_bfloat16* __restrict__ o) {
  __shared__ Spills spills[2 * kJoinHeads];     // [KV head of the block][own, prefix]
  ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  const StepPlan plan = step_plan(ds.plan, ds.num_seqs, ds.max_tokens);
  const StepWork work = step_work(ds, shp, plan);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = shp.g, H_kv = shp.H_kv, tpt = step_tile_tokens(g);
  const int T = plan.header[kPlanRows];
  const int s_ctas = (int)min((int64_t)ws.stream_grid, work.stream_total);
  const int t_ctas = (int)min((int64_t)ws.tile_grid, work.tile_total);
  const bool pre = ds.prefix_len > 0;
  const bool pre_streamed = work.prefix_stream_tiles > 0;
  const int h0 = blockIdx.x * kJoinHeads, h1 = min(h0 + kJoinHeads, shp.H_q);
  const int kv0 = h0 / g, n_kv = (h1 - 1) / g - kv0 + 1;
  for (int t = blockIdx.y; t < T; t += gridDim.y) {
    const StepRow r = plan.rows[t];
    int own_row = r.token * g;          // row of the sequence's first head in a spill
    const int pair = r.token / (2 * tpt), in_pair = r.token - pair * 2 * tpt;
    if (r.unit < 0)
      own_row = in_pair < tpt ? in_pair * g : kStepTileRows + (in_pair - tpt) * g;
    if (threadIdx.x < 2 * n_kv) {
      const int kvh = kv0 + (threadIdx.x >> 1);
      int64_t begin, total = work.stream_total;
      int unit = kStepStreamUnit, tiles, seen_tiles, ctas = s_ctas;
      if (threadIdx.x & 1) {
        if (pre_streamed) {
          tiles = work.prefix_stream_tiles;
          begin = work.stream_own + (int64_t)kvh * (tiles + unit);
        } else {
          tiles = work.prefix_tile_steps;
          unit = kStepTileUnit;
          begin = ((int64_t)kvh * work.prefix_pairs + t / (2 * tpt)) * (tiles + unit);
          total = work.tile_total;
          ctas = t_ctas;
        }
        seen_tiles = tiles;
      } else if (r.unit >= 0) {
        seen_tiles = tiles = r.tiles;
        begin = (int64_t)H_kv * r.cum + (int64_t)kvh * (tiles + unit);
      } else {
        const StepSeq e = plan.tiled[-1 - r.unit];
        const int seen = e.ctx - e.n_new;
        tiles = step_pair_tiles(seen, e.n_new, 2 * tpt, pair);
        // key tiles of the row's own query tile
        const int end = min(e.n_new, (2 * pair + (in_pair < tpt ? 1 : 2)) * tpt);
        seen_tiles = (seen + end + kStepTileKeys - 1) / kStepTileKeys;
        unit = kStepTileUnit;
        begin = work.tile_prefix + (int64_t)H_kv * r.cum + (int64_t)kvh * r.tiles +
                step_len_before(seen, 2 * tpt, pair);
        total = work.tile_total;
        ctas = t_ctas;
      }
      Spills s = {0, 0, false};
      if (pre || !(threadIdx.x & 1)) s = spills_of(begin, unit, tiles, seen_tiles, total, ctas);
      spills[threadIdx.x] = s;
    }
    __syncthreads();
    for (int h = h0 + warp; h < h1; h += kJoinWarps) {
      const int64_t w = (int64_t)t * shp.H_q + h;
      const int kvh = h / g, hh = h - kvh * g;
      const Spills a = spills[2 * (kvh - kv0)], p = spills[2 * (kvh - kv0) + 1];
      if (!pre && !a.cut) continue;      // the unit was whole: its kernel wrote O
      // sources: the unit's own rows, the prefix's, and the spills of both
      const int base = pre ? 2 : 1, n = base + a.n + p.n;
      float M = -INFINITY, L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s0 = 0; s0 < n; s0 += 32) {
        const int i = s0 + lane;
        const float* src = ws.own_o + w * 128;
        const float* lse = ws.own_lse + w;
        if (i == 1 && pre) {
          src = ws.pre_o + w * 128;
          lse = ws.pre_lse + w;
        } else if (i >= base) {
          const bool mine = i < base + a.n;
          const bool streamed = mine ? r.unit >= 0 : pre_streamed;
          const int c = mine ? a.first + i - base : p.first + i - base - a.n;
          int at = hh;
          if (mine) at += own_row;
          else if (streamed) at += t * g;
          else at += ((t / tpt) & 1) * kStepTileRows + (t % tpt) * g;
          const int64_t row = streamed ? (int64_t)c * kStepPackedRows + at
                                       : (int64_t)c * 2 * kStepTileRows + at;
          src = (streamed ? ws.stream_o : ws.tile_o) + row * 128;
          lse = (streamed ? ws.stream_lse : ws.tile_lse) + row;
        }
        const float l = i < n ? *lse : -INFINITY;
        float m = l;
#pragma unroll
        for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        m = fmaxf(m, M);
        // (a source without a visible key has log-sum-exp -inf and weight 0)
        const float wt = l == -INFINITY ? 0.f : exp2f(l - m);
        const float keep = M == -INFINITY ? 0.f : exp2f(M - m);
        float sum = wt;
#pragma unroll
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        M = m;
        L = L * keep + sum;
        acc.x *= keep;
        acc.y *= keep;
        acc.z *= keep;
        acc.w *= keep;
        const int count = min(32, n - s0);
#pragma unroll 8
        for (int k = 0; k < count; ++k) {
          const float* from = reinterpret_cast<const float*>(
              __shfl_sync(0xffffffffu, (unsigned long long)src, k));
          const float f = __shfl_sync(0xffffffffu, wt, k);
          const float4 v = reinterpret_cast<const float4*>(from)[lane];
          if (f != 0.f) {   // (an empty source's rows hold no sum: 0 x NaN is NaN)
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
          }
        }
      }
      const float inv = L > 0.f ? 1.f / L : 0.f;
      uint2 out;
      out.x = ptx::pack_bf16x2(acc.x * inv, acc.y * inv);
      out.y = ptx::pack_bf16x2(acc.z * inv, acc.w * inv);
      reinterpret_cast<uint2*>(o + w * 128)[lane] = out;
    }
    __syncthreads();   // the next row's spills replace these
  }
}

}  // namespace

bool step_fast_supported(const ShapeInfo& s) {
  const bool block_ok = (s.B % kStepTileKeys == 0) || (kStepTileKeys % s.B == 0 && s.B % 8 == 0);
  return s.dtype == 0 && s.D == 128 && s.g <= 64 && block_ok;
}

size_t step_workspace(const ShapeInfo& s, int32_t max_tokens, int sms, void* base,
                      StepWorkspace* w) {
  size_t at = 0;
  auto take = [&](int64_t floats) -> float* {
    float* p = base ? reinterpret_cast<float*>((char*)base + at) : nullptr;
    at += ((size_t)floats * 4 + 255) / 256 * 256;
    return p;
  };
  const int64_t rows = (int64_t)max_tokens * s.H_q;
  StepWorkspace v;
  v.stream_grid = 2 * sms;
  v.tile_grid = sms;
  v.own_o = take(rows * 128);
  v.pre_o = take(rows * 128);
  v.own_lse = take(rows);
  v.pre_lse = take(rows);
  v.stream_o = take((int64_t)v.stream_grid * kStepPackedRows * 128);
  v.stream_lse = take((int64_t)v.stream_grid * kStepPackedRows);
  v.tile_o = take((int64_t)v.tile_grid * 2 * kStepTileRows * 128);
  v.tile_lse = take((int64_t)v.tile_grid * 2 * kStepTileRows);
  if (w) *w = v;
  return at;
}

cudaError_t launch_step_stream(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w,
                               const void* q, const void* k_cache, const void* v_cache, void* o,
                               bool first, cudaStream_t st) {
  const int64_t rows = (int64_t)ds.num_blocks * s.H_kv * s.B;
  const int box_rows = s.B < kKeys ? s.B : kKeys;
  Maps maps;
  cudaError_t e;
  if (box_rows < 16) {
    e = make_cache_tmap(&maps.k, k_cache, rows, s.D, box_rows);
    if (e == cudaSuccess) e = make_cache_tmap(&maps.v, v_cache, rows, s.D, box_rows);
    maps.k_one = maps.k;
    maps.v_one = maps.v;
  } else {
    e = make_group_tmap(&maps.k, k_cache, rows, box_rows / 16);
    if (e == cudaSuccess) e = make_group_tmap(&maps.v, v_cache, rows, box_rows / 16);
    if (e == cudaSuccess) e = make_group_tmap(&maps.k_one, k_cache, rows, 1);
    if (e == cudaSuccess) e = make_group_tmap(&maps.v_one, v_cache, rows, 1);
  }
  if (e != cudaSuccess) return e;
  // the shared-memory limit is raised once per device
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load() & bit)) {
    e = cudaFuncSetAttribute(step_stream_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(step_stream_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)w.stream_grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, step_stream_kernel, maps, ds, s, w, (const __nv_bfloat16*)q,
                            (__nv_bfloat16*)o, first ? 1 : 0);
}

cudaError_t launch_step_combine(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w,
                                void* o, cudaStream_t st) {
  const int chunks = (s.H_q + kJoinHeads - 1) / kJoinHeads;
  const int rows = std::min(ds.max_tokens, std::max(1, w.tile_grid * 16 / chunks));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)chunks, (unsigned)std::min(rows, 65535));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, step_combine_kernel, ds, s, w, (__nv_bfloat16*)o);
}

}  // namespace rbkv
