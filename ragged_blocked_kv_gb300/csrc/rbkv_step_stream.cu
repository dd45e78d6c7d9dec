// Streaming attention of a step: units of at most 16 packed query rows (a
// sequence's new tokens x the heads of one KV group) over the sequence's own
// keys; every cached K/V byte is read once, so HBM bounds it.
//
// The units lie on one line in groups of 16 keys, cut evenly (rbkv_step.h) over
// eight warps per SM, in two CTAs - or four in one CTA beside a CTA of the tile
// kernel, whose tensor-core work then runs under the memory traffic of this
// one (they share an SM's registers and shared memory by design: 98 and 130
// KB).  Each warp is a pipeline of its own: it keeps a ring of three 8 KB groups
// (16 keys of K and V, 16 bytes per lane and copy) in flight, and multiplies,
// exponentiates and accumulates a group at a time:
//   S^T = K Q^T   (m16n8k16: 16 keys x 8 query rows, one or two such tiles)
//   P^T = exp2(S^T - running maximum of the row), rounded to bf16
//   O^T += V^T P^T (16 head dims x 8 rows per MMA)
// with the keys and head dims on the MMAs' 16-row side, so a group of 4 or 8
// heads wastes at most half of the narrow side, where Q on the 16-row side
// would waste three quarters.  No warp waits for another: no merge, no block
// barrier; 192 KB in flight per SM cover the latency.  (Four warps sharing
// 64-key tiles of a common ring, merged per unit, held 5.2 TB/s on 512
// sequences of 256 keys: the merge idled the ring.)  Beside the tile kernel the
// two contend for the SM's issue slots, not for the memory: with its
// arithmetic left out the whole step took 102 instead of 127 us, and half of
// the tile kernel's operand bytes made no difference.  The copies are the lanes'
// own (cp.async): as one bulk tensor copy per group they took 99 us for those
// 512 sequences instead of 93 (5.8 TB/s), and held up the tile kernel's tensor
// copies on the same SM: 137 instead of 127 us for both.
#include <algorithm>
#include <atomic>

#include "rbkv_step.h"
#include "rbkv_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace rbkv {

namespace {

constexpr int kWarps = kStepPipes;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kKeys = kStepStreamKeys;        // keys of a group
constexpr int kHalf = kKeys * 128;            // 16 rows x 128 B (64 bf16 of head_dim)
constexpr int kGroup = 2 * kHalf;             // a group of K or V, head_dim 128
constexpr int kStage = 2 * kGroup;            // K + V
constexpr int kRows = kStepPackedRows;
constexpr int kSegments = kStages + 2;        // segments that a warp's window can meet
constexpr int kSmemBytes =
    kWarps * (kStages * kStage + kSegments * 32);
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024 &&
              kSmemBytes + kStepTileSmem + 2 * 1024 <= 228 * 1024,
              "two CTAs per SM, or one beside the tile kernel's");
constexpr float kLog2e = 1.4426950408889634f;

// Byte offset, inside a group, of the 16-byte chunk holding elements d..d+7
// (d % 8 == 0) of key row `key`: two halves of the head dim, 128-byte swizzle.
__device__ __forceinline__ uint32_t group_off(int key, int d) {
  return (d >> 6) * kHalf + key * 128 + ((((d & 63) >> 3) ^ (key & 7)) << 4);
}

// The 8 x 8 transpose of a matrix of 16-bit elements held two per lane (row
// lane / 4, columns 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// One segment of a unit.
struct __align__(16) Segment {
  int row, n_tok;        // first row and tokens of the unit
  int kv_head;
  int group, groups;     // first group of keys, and number of them (0: no more)
  int keys;              // keys of the unit's last row
  int cuts;              // at a unit's head: pipelines that begin inside it behind this
  int flags;
};
static_assert(sizeof(Segment) == 32, "Segment is 8 int32");
enum { kPrefix = 1, kHead = 2, kWhole = 4 };

// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
               "l"(src), "r"(live ? 16 : 0), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's walk over its part [x, end) of the line, one group per issue().
// Every lane holds the same state; block ids are held 32 to a warp.  Units
// follow one another without a division: the next KV head, then the next
// sequence, whose entry is loaded one sequence ahead and whose first ids when
// the current sequence's last head begins.
struct Walk {
  int64_t end, unit0;    // end of the part; the unit's place on the line
  int64_t next_x;        // where the unit after this one begins
  int unit, kv_head;
  int left;              // groups of the segment not issued yet
  int entry, sub;        // of the next group: block list entry, group in the block
  int window;            // first entry of the ids held
  int ids, ids_next;     // this lane's
  StepSeq cur, next;
  const int32_t* table;
  uint32_t seg;          // segments published
  bool missing;          // a block id outside the pool has been met
  StreamCuts cuts;
  int32_t pipe;          // this pipeline
  uint64_t once;         // the L2 policy of the loads
  const __nv_bfloat16 *k_cache, *v_cache;

  __device__ __forceinline__ int load_ids(const int32_t* t, int from, int n, int lane) const {
    return from + lane < n ? t[from + lane] : 0;
  }
  // entries of the block list that the unit's keys take
  __device__ __forceinline__ int entries(int keys, int B) const { return (keys + B - 1) / B; }

  __device__ __forceinline__ void enter(const DevStep& ds, const ShapeInfo& s,
                                        const StepWork& work) {
    if (unit < work.streamed) {
      unit0 = (int64_t)s.H_kv * cur.cum + (int64_t)kv_head * (cur.tiles + kStepStreamUnit);
      table = ds.block_table + (int64_t)cur.seq * ds.max_blocks;
    } else {
      cur.row = 0;
      cur.n_new = work.rows;
      cur.ctx = ds.prefix_len;
      cur.tiles = work.prefix_stream_tiles;
      unit0 = work.stream_own + (int64_t)kv_head * (cur.tiles + kStepStreamUnit);
      table = ds.prefix_table;
    }
  }

  __device__ __forceinline__ void start(int64_t x, const DevStep& ds, const ShapeInfo& s,
                                        const StepPlan& plan, const StepWork& work, int lane) {
    int64_t base = work.stream_own;
    unit = work.streamed;
    int len = work.prefix_stream_tiles + kStepStreamUnit;
    if (x < work.stream_own) {
      // the last sequence at or before x: 32 places tested at a time
      const int32_t v = (int32_t)step_div(x, s.H_kv);
      int lo = 0, n = unit;
      while (n > 1) {
        const int step = (n + 31) >> 5;
        const bool le = lane * step < n && plan.streamed[lo + lane * step].cum <= v;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));   // lane 0 always holds
        lo += k * step;
        n = min(step, n - k * step);
      }
      unit = lo;
      cur = plan.streamed[unit];
      next = plan.streamed[min(unit + 1, ds.num_seqs - 1)];
      base = (int64_t)s.H_kv * cur.cum;
      len = cur.tiles + kStepStreamUnit;
    }
    kv_head = (int)step_div(x - base, len);
    enter(ds, s, work);
    next_x = x;
    left = 0;
    seg = 0;
    missing = false;
    window = -1;
    ids_next = 0;
    if (unit < work.streamed && kv_head == s.H_kv - 1) prefetch(ds, s, work, lane);
  }

  __device__ __forceinline__ void prefetch(const DevStep& ds, const ShapeInfo& s,
                                           const StepWork& work, int lane) {
    if (unit + 1 < work.streamed)
      ids_next = load_ids(ds.block_table + (int64_t)next.seq * ds.max_blocks, 0,
                          entries(next.ctx, s.B), lane);
  }

  // Publishes the next segment of the part; false when there is none.
  __device__ __forceinline__ bool advance(Segment* segments, const DevStep& ds,
                                          const ShapeInfo& s, const StepPlan& plan,
                                          const StepWork& work, int lane) {
    while (next_x < end) {
      if (next_x > unit0 + cur.tiles + kStepStreamUnit - 1) {   // on to the next unit
        bool moved = false;
        if (++kv_head == s.H_kv) {
          kv_head = 0;
          ++unit;
          cur = next;
          moved = true;
        }
        enter(ds, s, work);
        if (moved) {
          window = -1;
          if (unit < work.streamed) {
            next = plan.streamed[min(unit + 1, ds.num_seqs - 1)];
            ids = ids_next;
            window = 0;
          }
        }
        if (unit < work.streamed && kv_head == s.H_kv - 1) prefetch(ds, s, work, lane);
      }
      const int n = cur.tiles;
      const int64_t from = next_x - unit0 - kStepStreamUnit, to = end - unit0 - kStepStreamUnit;
      const int first = (int)(from < 0 ? 0 : from);
      const int last = (int)(to < 0 ? 0 : to < n ? to : n);
      next_x = unit0 + n + kStepStreamUnit;
      if (first >= last) continue;
      left = last - first;
      const bool prefix = unit >= work.streamed;
      if (s.B >= kKeys) {
        const int per = s.B / kKeys;
        entry = first / per;
        sub = first - entry * per;
      } else {
        entry = 2 * first;
        sub = 0;
      }
      const int n_entries = entries(cur.ctx, s.B);
      if (window < 0 || entry < window || entry >= window + 32) {
        window = entry;
        ids = load_ids(table, window, n_entries, lane);
      }
      Segment g;
      g.row = cur.row;
      g.n_tok = cur.n_new;
      g.kv_head = kv_head;
      g.group = first;
      g.groups = left;
      g.keys = cur.ctx;
      g.flags = (prefix ? kPrefix : 0) | (first == 0 ? kHead : 0) |
                (first == 0 && last == n ? kWhole : 0);
      // pipelines that begin inside the unit, behind this segment at its head
      g.cuts = 0;
      if (first == 0 && last < n) g.cuts = cuts.first(next_x) - (pipe + 1);
      segments[seg % kSegments] = g;      // (every lane the same values)
      ++seg;
      return true;
    }
    return false;
  }

  // The next block id of the list.
  __device__ __forceinline__ int id_at(int e, const ShapeInfo& s, int lane) {
    if (e >= window + 32 || e < window) {
      window = e;
      ids = load_ids(table, window, entries(cur.ctx, s.B), lane);
    }
    return __shfl_sync(0xffffffffu, ids, e - window);
  }

  // Loads the next group into `stage`, if the part has one.  Lane l copies the
  // 16-byte chunk l % 16 of rows l / 16, + 2, ...; rows past the unit's last key
  // are zero (unwritten cache slots: 0 * V has to be 0), and so are those of a
  // block id outside the pool, whose scores are then taken for -inf.
  __device__ __forceinline__ void issue(uint8_t* stage, Segment* segments, const DevStep& ds,
                                        const ShapeInfo& s, const StepPlan& plan,
                                        const StepWork& work, int lane) {
    if (left == 0 && !advance(segments, ds, s, plan, work, lane)) return;
    --left;
    const int c = lane & 15, r0 = lane >> 4;
    const uint32_t dst = ptx::smem_u32(stage) + (c >> 3) * kHalf + r0 * 128;
    const int keys = cur.ctx - entry * s.B - sub * kKeys;     // of the unit, from here
    bool bad = false;
    auto half = [&](int blk, int row_in_block, int first) {   // eight rows
      const bool ok = (uint32_t)blk < (uint32_t)ds.num_blocks;
      bad |= !ok;
      const int64_t at =
          (((int64_t)(ok ? blk : 0) * s.H_kv + kv_head) * s.B + row_in_block + r0) * 128 + c * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t to = dst + (first + 2 * i) * 128 + ((((c & 7) ^ r0) ^ (2 * i)) << 4);
        const bool live = ok && first + 2 * i + r0 < keys;
        copy16(to, k_cache + at + i * 256, live, once);
        copy16(to + kGroup, v_cache + at + i * 256, live, once);
      }
    };
    const int blk = id_at(entry, s, lane);
    if (s.B >= kKeys) {
      half(blk, sub * kKeys, 0);
      half(blk, sub * kKeys + 8, 8);
      if (++sub * kKeys == s.B) {
        sub = 0;
        ++entry;
      }
    } else {
      // 8-key blocks: a group is two of them, or one at the unit's end
      const int blk1 = keys > 8 ? id_at(entry + 1, s, lane) : blk;
      half(blk, 0, 0);
      half(blk1, 0, 8);
      entry += 2;
    }
    if (bad) {
      missing = true;
      if (lane == 0) atomicCAS(ds.status, 0, kDevBounds);
    }
  }
};

// The queries of a unit as the B operand of S^T = K Q^T: row n of tile i is
// packed row 8 i + n (token / g, head % g); rows past the unit's are zero.
template <int NT>
__device__ __forceinline__ void load_q(uint32_t (&qb)[NT][8][2], const Segment& u,
                                       const ShapeInfo& s, const __nv_bfloat16* q, int lane) {
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int r = 8 * i + (lane >> 2), tok = r / s.g;
    const bool live = tok < u.n_tok;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(
                            q + ((int64_t)(u.row + tok) * s.H_q + u.kv_head * s.g +
                                 (r - tok * s.g)) * 128) + (lane & 3);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      qb[i][kk][0] = live ? __ldg(p + kk * 8) : 0u;
      qb[i][kk][1] = live ? __ldg(p + kk * 8 + 4) : 0u;
    }
  }
}

// Moves a group's non-finite values, if there are any, from V (in shared
// memory) to the accumulators of the rows that see them: lane's rows 8 i + 2
// (lane % 4) + e, dims 16 t + lane / 4 (+ 8).
template <int NT, bool kDraft>
__device__ __forceinline__ void add_nonfinite(uint8_t* v, int key0, const int (&lim)[NT][2],
                                              const uint32_t (&own)[NT][2],
                                              float (&acc)[NT][8][4], int lane) {
  bool any = false;
#pragma unroll
  for (int e = 0; e < kGroup / 16; e += 32) {
    const uint4 w = *reinterpret_cast<const uint4*>(v + (e + lane) * 16);
    any |= (nonfinite2(w.x) | nonfinite2(w.y) | nonfinite2(w.z) | nonfinite2(w.w)) != 0;
  }
  if (!__any_sync(0xffffffffu, any)) return;
#pragma unroll 1
  for (int key = 0; key < kKeys; ++key) {
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const uint32_t w = *reinterpret_cast<const uint16_t*>(v + group_off(key, 8 * u) +
                                                            (lane >> 2) * 2);
      if (nonfinite2(w)) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (key0 + key < lim[i][e] || (kDraft && (own[i][e] >> key & 1u)))
              acc[i][u / 2][(u & 1) * 2 + e] += __uint_as_float(w << 16);
      }
    }
  }
  __syncwarp();
  for (int e = lane; e < kGroup / 16; e += 32) zero_nonfinite(reinterpret_cast<uint4*>(v) + e);
  __syncwarp();
}

// A warp's ring.
struct Ring {
  uint8_t* stages;
  Segment* segments;
  uint32_t taken;
};

// Works through one segment: NT tiles of 8 packed rows.
template <int NT, bool kDraft>
__device__ __forceinline__ void run_segment(const Segment& it, Ring& ring, Walk& walk,
                                            const DevStep& ds, const ShapeInfo& s,
                                            const StepPlan& plan,
                                            const StepWork& work, const StepWorkspace& ws,
                                            const __nv_bfloat16* q, __nv_bfloat16* o,
                                            int64_t pipe, int lane) {
  uint32_t qb[NT][8][2];
  load_q<NT>(qb, it, s, q, lane);
  const float qk_scale = s.scale * kLog2e;
  const int c2 = (lane & 3) * 2;               // this lane's query rows: 8 i + c2, + 1
  const int kr = lane >> 2;                    // ... and keys (or head dims): kr, kr + 8
  int lim[NT][2];                              // keys that they see
  float m[NT][2], l[NT][2], acc[NT][8][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      lim[i][e] = it.flags & kPrefix
                      ? it.keys
                      : min(it.keys, it.keys - it.n_tok + 1 + (8 * i + c2 + e) / s.g);
      m[i][e] = -INFINITY;
      l[i][e] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) acc[i][t][0] = acc[i][t][1] = acc[i][t][2] = acc[i][t][3] = 0.f;
  }
  // keys that every row of the unit sees
  const bool tree = kDraft && !(it.flags & kPrefix);
  const int seen = it.keys - it.n_tok;
  const int all_see = it.flags & kPrefix ? it.keys : tree ? seen : seen + 1;
  if (tree) {
    // a row that does not follow every token before it sees the cached keys, and
    // then those of its ancestors
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tok = (8 * i + c2 + e) / s.g;
        if (tok < it.n_tok && !draft_is_run(ds, it.row + tok, seen, tok)) lim[i][e] = seen;
      }
  }
  // ldmatrix rows of this lane: K as [key][dim] tiles, V transposed
  const int k_key = (lane & 7) + ((lane >> 3) & 1) * 8, k_d = (lane >> 4) * 8;
  const int v_key = (lane & 7) + (lane >> 4) * 8, v_d = ((lane >> 3) & 1) * 8;

  for (int j = 0; j < it.groups; ++j) {
    const int st = ring.taken % kStages;
    copies_wait<kStages - 1>();
    __syncwarp();
    const int key0 = (it.group + j) * kKeys;
    uint8_t* stage = ring.stages + st * kStage;
    const uint32_t kt = ptx::smem_u32(stage), vt = kt + kGroup;
    // S^T = K Q^T, the head dim in two chains of MMAs
    float sc[NT][4], sd[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) sc[i][x] = sd[i][x] = 0.f;
#pragma unroll
    for (int kk = 0; kk < 8; kk += 2) {
      uint32_t a[4], b[4];
      ptx::ldsm_x4(kt + group_off(k_key, kk * 16 + k_d), a[0], a[1], a[2], a[3]);
      ptx::ldsm_x4(kt + group_off(k_key, kk * 16 + 16 + k_d), b[0], b[1], b[2], b[3]);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        ptx::mma_bf16_16816(sc[i], a, qb[i][kk][0], qb[i][kk][1]);
        ptx::mma_bf16_16816(sd[i], b, qb[i][kk + 1][0], qb[i][kk + 1][1]);
      }
    }
    // keys without a block (this group's or one issued later has some)
    if (walk.missing) {
      const int32_t* table = ds.prefix_table;
      if (!(it.flags & kPrefix))
        table = ds.block_table +
                (int64_t)plan.streamed[plan.rows[it.row].unit].seq * ds.max_blocks;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int key = key0 + 8 * half;
        if (key >= it.keys || (uint32_t)table[key / s.B] < (uint32_t)ds.num_blocks) continue;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          sc[i][2 * half] = sc[i][2 * half + 1] = -INFINITY;
          sd[i][2 * half] = sd[i][2 * half + 1] = 0.f;
        }
      }
    }
    uint32_t pb[NT][2];
    // bit k: key key0 + k is that of an ancestor (at most 16 tokens: one word; looked
    // up in the one or two groups that hold them)
    uint32_t own[NT][2];
#pragma unroll
    for (int i = 0; i < NT; ++i) own[i][0] = own[i][1] = 0;
    if (tree && key0 + kKeys > seen) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tok = (8 * i + c2 + e) / s.g;
          const uint32_t w = tok < it.n_tok ? ds.ancestors[it.row + tok].x & 0xffffu : 0u;
          const int by = key0 - seen;             // -15 .. 15
          own[i][e] = by >= 0 ? w >> by : w << -by;
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // rows' scores of keys kr and kr + 8, masked; the row's maximum over
        // the eight lanes that share it
        float x = (sc[i][e] + sd[i][e]) * qk_scale, y = (sc[i][2 + e] + sd[i][2 + e]) * qk_scale;
        bool sees_x = key0 + kr < lim[i][e], sees_y = key0 + kr + 8 < lim[i][e];
        if (kDraft) {
          sees_x |= own[i][e] >> kr & 1u;
          sees_y |= own[i][e] >> (kr + 8) & 1u;
        }
        x = sees_x ? x : -INFINITY;
        y = sees_y ? y : -INFINITY;
        float top = fmaxf(x, y);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const float mn = fmaxf(m[i][e], top);
        // a row with no visible key so far keeps max -inf: its terms are 0
        const float base = mn == -INFINITY ? 0.f : mn;
        const float corr = ptx::ex2(m[i][e] - base);
        m[i][e] = mn;
        x = ptx::ex2(x - base);
        y = ptx::ex2(y - base);
        l[i][e] = fmaf(l[i][e], corr, x + y);
        sc[i][e] = x;
        sc[i][2 + e] = y;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          acc[i][t][e] *= corr;
          acc[i][t][2 + e] *= corr;
        }
      }
      // the weights enter the value product as bf16 (its operand type): each
      // off by at most 2^-8 of itself; their sum above stays fp32.  [key][row]
      // pairs become the [row][key] pairs of the B operand.
      pb[i][0] = transpose8(ptx::pack_bf16x2(sc[i][0], sc[i][1]));
      pb[i][1] = transpose8(ptx::pack_bf16x2(sc[i][2], sc[i][3]));
    }
    if (key0 + kKeys > all_see && all_see < it.keys)
      add_nonfinite<NT, kDraft>(stage + kGroup, key0, lim, own, acc, lane);
    // O^T += V^T P^T: 8 tiles of 16 head dims
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      uint32_t a[4];
      ptx::ldsm_x4_t(vt + group_off(v_key, t * 16 + v_d), a[0], a[1], a[2], a[3]);
#pragma unroll
      for (int i = 0; i < NT; ++i) ptx::mma_bf16_16816(acc[i][t], a, pb[i][0], pb[i][1]);
    }
    ++ring.taken;
    __syncwarp();
    // the stage is free: the next group of the part
    walk.issue(stage, ring.segments, ds, s, plan, work, lane);
    copies_commit();
  }

  // ---- the segment's result: O itself when nothing is to be joined, the
  // unit's rows of the workspace, or this warp's spill rows ----
  const bool head = it.flags & kHead, pre = it.flags & kPrefix;
  const bool direct = (it.flags & kWhole) && ds.prefix_len == 0;
  float* part = head ? (pre ? ws.pre_o : ws.own_o) : ws.stream_o;
  float* lse = head ? (pre ? ws.pre_lse : ws.own_lse) : ws.stream_lse;
  const int nrg = it.n_tok * s.g;
  if (head && lane == 0)
    (pre ? ws.pre_cut : ws.own_cut)[(int64_t)it.row * s.H_kv + it.kv_head] =
        Spills{(int32_t)pipe + 1, it.cuts};
  auto place = [&](int r) -> int64_t {
    const int tok = r / s.g;
    return head ? (int64_t)(it.row + tok) * s.H_q + it.kv_head * s.g + (r - tok * s.g)
                : pipe * kRows + r;
  };
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    float inv[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[i][e];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      inv[e] = sum > 0.f ? 1.f / sum : 0.f;
      const int r = 8 * i + c2 + e;
      if (!direct && r < nrg) {
        const int64_t to = place(r);
        if (kr == 0) lse[to] = sum > 0.f ? m[i][e] + log2f(sum) : -INFINITY;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          part[to * 128 + t * 16 + kr] = acc[i][t][e] * inv[e];
          part[to * 128 + t * 16 + kr + 8] = acc[i][t][2 + e] * inv[e];
        }
      }
    }
    if (direct) {
      const int r = 8 * i + kr;               // after the transpose: one row, two dims
      const int64_t to = r < nrg ? place(r) : 0;
#pragma unroll
      for (int t = 0; t < 8; ++t) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t v = transpose8(ptx::pack_bf16x2(acc[i][t][2 * x] * inv[0],
                                                         acc[i][t][2 * x + 1] * inv[1]));
          if (r < nrg)
            *reinterpret_cast<uint32_t*>(o + to * 128 + t * 16 + 8 * x + c2) = v;
        }
      }
    }
  }
}

template <bool kDraft>
__global__ void __launch_bounds__(kThreads, 2)
    step_stream_kernel(DevStep ds, ShapeInfo shp, StepWorkspace ws,
                       const __nv_bfloat16* __restrict__ q,
                       const __nv_bfloat16* __restrict__ k_cache,
                       const __nv_bfloat16* __restrict__ v_cache, __nv_bfloat16* __restrict__ o,
                       int first) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (first) ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const StepPlan plan = step_plan(ds.plan, ds.num_seqs, ds.max_tokens);
  if (!step_matches<kDraft>(ds, shp, plan)) {
    ptx::pdl_wait_previous();
    return;
  }
  const StepWork work = step_work(ds, shp, plan);
  const StreamCuts cuts = step_stream_cuts(ws, work);
  // neighbouring parts on different SMs; the second half of the grid is late
  const int half = ws.stream_grid / 2;
  const bool late = (int)blockIdx.x >= half;
  const int mine = warp * half + ((int)blockIdx.x - (late ? half : 0));
  const int pipe = late ? cuts.early + mine : mine;
  const bool works = mine < (late ? cuts.late : cuts.early);
  if (works) {
    Ring ring;
    ring.stages = smem_raw + warp * kStages * kStage;
    ring.segments =
        reinterpret_cast<Segment*>(smem_raw + kWarps * kStages * kStage) + warp * kSegments;
    ring.taken = 0;
    Walk walk;
    walk.cuts = cuts;
    walk.pipe = pipe;
    // own keys are read once: they are not to push the prefix, the queries and
    // the partial outputs out of the L2
    walk.once = ptx::policy_evict_first();
    walk.k_cache = k_cache;
    walk.v_cache = v_cache;
    walk.end = cuts.at(pipe + 1);
    walk.start(cuts.at(pipe), ds, shp, plan, work, lane);
    for (int i = 0; i < kStages; ++i) {
      walk.issue(ring.stages + i * kStage, ring.segments, ds, shp, plan, work, lane);
      copies_commit();
    }
    __syncwarp();
    for (uint32_t n = 0; n < walk.seg; ++n) {
      const Segment it = ring.segments[n % kSegments];
      if (it.n_tok * shp.g <= 8)
        run_segment<1, kDraft>(it, ring, walk, ds, shp, plan, work, ws, q, o, pipe, lane);
      else
        run_segment<2, kDraft>(it, ring, walk, ds, shp, plan, work, ws, q, o, pipe, lane);
      __syncwarp();
    }
  }
  ptx::pdl_wait_previous();   // the grid's completion covers its predecessor
}

// ---------------------------------------------------------------------------
// The join: W warps to a (row, query head), or V of them to a warp.
// ---------------------------------------------------------------------------
// O = sum_i 2^(L_i - M) O_i / sum_i 2^(L_i - M) over the row's partial
// outputs: its own part and the prefix's, each with the spills of the CTAs (or
// pipelines) that begin inside its unit, which the segment at the unit's head
// has written down.  The partials come from the L2, they were just written; the
// chain of dependent loads (place, spills, their rows) bounds a step of few
// rows, the instructions of finding the sources one of many.  So a step of at
// most 16 rows, which may have a hundred sources to a row (every pipeline
// streamed a piece of a long prefix), gives a row eight warps (a whole step of
// 1, 4, 8, 16 rows behind 4096 keys: 10.3, 12.6, 14.8, 18.0 us; with a warp
// each 29.6, 31.9, 16.9, 18.0; 32 rows 28.0 and 27.6); one whose rows all fit
// the SMs at once, a warp each; and a larger one has four rows in each
// warp, which find their sources together: 512 rows of 32 heads 6.0 us (10.0
// with a warp each, 6.6 with two rows to a warp), 1088 rows 12.5 us (17.1,
// 13.5); a step of 64 rows takes 68.4 us with a warp each and 71.6 with four.
constexpr int kJoinWarps = 8;
constexpr int kJoinBlocks = 4;      // blocks per SM
constexpr int kJoinWideRows = 16;   // steps of at most this many rows: W = 8
constexpr int kJoinVecs = 4;        // rows of a warp in steps of many rows

// Partial outputs of one part (own or prefix): source k's row.
struct Part {
  const float *o, *lse;
  int row, stride;
};

// V float4 per lane: columns 4 (lane + i lanes) .. + 3, i < V.
template <int V>
struct Join {
  float M, L;
  float4 acc[V];
  // N more sources (missing ones and those without a visible key have
  // log-sum-exp -inf)
  template <int N>
  __device__ __forceinline__ void add(const float (&l)[N], const float4 (&v)[N][V]) {
    float m = M;
#pragma unroll
    for (int u = 0; u < N; ++u) m = fmaxf(m, l[u]);
    const float base = m == -INFINITY ? 0.f : m;
    const float keep = ptx::ex2(M - base);
    M = m;
    L *= keep;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      acc[i].x *= keep;
      acc[i].y *= keep;
      acc[i].z *= keep;
      acc[i].w *= keep;
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const float w = ptx::ex2(l[u] - base);
      L += w;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        acc[i].x = fmaf(w, v[u][i].x, acc[i].x);
        acc[i].y = fmaf(w, v[u][i].y, acc[i].y);
        acc[i].z = fmaf(w, v[u][i].z, acc[i].z);
        acc[i].w = fmaf(w, v[u][i].w, acc[i].w);
      }
    }
  }
};

__device__ __forceinline__ int bounded(const Spills& s, int rows) {
  return s.first >= 0 && s.first <= rows && s.n > 0 && s.n <= rows - s.first ? s.n : 0;
}

template <int W, int V, bool kDraft>
__global__ void __launch_bounds__(kJoinWarps * 32, W > 1 ? 2 : kJoinBlocks)
    step_combine_kernel(DevStep ds, ShapeInfo shp, StepWorkspace ws,
                        __nv_bfloat16* __restrict__ o) {
  static_assert(W == 1 || V == 1, "several warps to a row, or several rows to a warp");
  constexpr int kLanes = 32 / V;                         // of a row
  constexpr int kHeads = kJoinWarps * V / W;             // query heads of a block
  __shared__ float4 wide_acc[W > 1 ? kJoinWarps * 32 : 1];
  __shared__ float wide_ml[W > 1 ? kJoinWarps * 2 : 1];
  ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x % kLanes;
  const int g = shp.g, tpt = step_tile_tokens(g);
  const bool pre = ds.prefix_len > 0;
  const int h = blockIdx.x * kHeads + threadIdx.x / (kLanes * W), wi = warp % W;
  if (h >= shp.H_q) return;      // (W = 8: the block is one head, in range)
  const int kvh = h / g, hh = h - kvh * g;
  const bool pre_streamed = pre && step_prefix_streamed(ds.max_tokens, g);
  const StepPlan plan = step_plan(ds.plan, ds.num_seqs, ds.max_tokens);
  const int T = step_rows<kDraft>(ds, shp, plan);
  for (int t = blockIdx.y; t < T; t += gridDim.y) {
    const int64_t w = (int64_t)t * shp.H_q + h;
    // the two main sources, requested before anything that depends on the
    // row's place
    float l2[2] = {-INFINITY, -INFINITY};
    float4 v2[2][V];
#pragma unroll
    for (int i = 0; i < V; ++i) v2[0][i] = v2[1][i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (wi == 0) {
      l2[0] = ws.own_lse[w];
#pragma unroll
      for (int i = 0; i < V; ++i)
        v2[0][i] = reinterpret_cast<const float4*>(ws.own_o + w * 128)[lane + i * kLanes];
      if (pre) {
        l2[1] = ws.pre_lse[w];
#pragma unroll
        for (int i = 0; i < V; ++i)
          v2[1][i] = reinterpret_cast<const float4*>(ws.pre_o + w * 128)[lane + i * kLanes];
      }
    }
    Spills a, p = {0, 0};
    const int pre_in = pre_streamed ? t : t % tpt;      // the row in its prefix unit
    if (pre) p = ws.pre_cut[(int64_t)(t - pre_in) * shp.H_kv + kvh];
    const StepRow r = plan.rows[t];
    const int own_in = r.unit >= 0 ? r.token : r.token % tpt;
    a = ws.own_cut[(int64_t)(t - own_in) * shp.H_kv + kvh];
    // (after a wait that gave up, a unit's Spills may not have been written:
    // nothing outside the spill rows is read then either)
    int apart = 1;           // (CTAs from one spill of a unit to the next)
    if constexpr (kDraft) {
      if (a.n & kSpillsApart) {
        apart = 2;
        a.n &= ~kSpillsApart;
        // (the last one's place, as below)
        if (a.n > 0 && 2 * a.n - 1 > ws.tile_grid - a.first) a.n = 0;
      }
    }
    a.n = bounded(a, r.unit >= 0 ? ws.stream_grid * kStepPipes : ws.tile_grid);
    p.n = bounded(p, pre_streamed ? ws.stream_grid * kStepPipes : ws.tile_grid);
    Join<V> j;
    j.M = -INFINITY;
    j.L = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) j.acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    j.template add<2>(l2, v2);
    const int n = a.n + p.n;
    if (n > wi) {
      const Part mine = r.unit >= 0
          ? Part{ws.stream_o, ws.stream_lse, a.first * kStepPackedRows + own_in * g + hh,
                 kStepPackedRows}
          : Part{ws.tile_o, ws.tile_lse, a.first * kStepTileRows + own_in * g + hh,
                 kStepTileRows * apart};
      const Part theirs = pre_streamed
          ? Part{ws.stream_o, ws.stream_lse, p.first * kStepPackedRows + pre_in * g + hh,
                 kStepPackedRows}
          : Part{ws.tile_o, ws.tile_lse, p.first * kStepTileRows + pre_in * g + hh,
                 kStepTileRows};
      constexpr int kAtOnce = W > 1 ? 8 : 4 / V;
      for (int k0 = wi; k0 < n; k0 += kAtOnce * W) {
        float l[kAtOnce];
        float4 v[kAtOnce][V];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int k = k0 + u * W;
          l[u] = -INFINITY;
#pragma unroll
          for (int i = 0; i < V; ++i) v[u][i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < n) {
            const bool m = k < a.n;
            const int row = m ? mine.row + k * mine.stride
                              : theirs.row + (k - a.n) * theirs.stride;
            l[u] = (m ? mine.lse : theirs.lse)[row];
            const float4* from =
                reinterpret_cast<const float4*>((m ? mine.o : theirs.o) + (int64_t)row * 128);
#pragma unroll
            for (int i = 0; i < V; ++i) v[u][i] = from[lane + i * kLanes];
          }
        }
        j.template add<kAtOnce>(l, v);
      }
    }
    if constexpr (W > 1) {
      wide_acc[threadIdx.x] = j.acc[0];
      if (lane == 0) {
        wide_ml[warp * 2] = j.M;
        wide_ml[warp * 2 + 1] = j.L;
      }
      __syncthreads();
      if (wi == 0) {
#pragma unroll
        for (int x = 1; x < W; ++x) {
          float m = wide_ml[x * 2], base = fmaxf(j.M, m);
          base = base == -INFINITY ? 0.f : base;
          const float keep = ptx::ex2(j.M - base), f = ptx::ex2(m - base);
          const float4 v = wide_acc[x * 32 + lane];
          j.M = fmaxf(j.M, m);
          j.L = j.L * keep + wide_ml[x * 2 + 1] * f;
          j.acc[0].x = j.acc[0].x * keep + v.x * f;
          j.acc[0].y = j.acc[0].y * keep + v.y * f;
          j.acc[0].z = j.acc[0].z * keep + v.z * f;
          j.acc[0].w = j.acc[0].w * keep + v.w * f;
        }
      }
    }
    // (a unit that was whole and alone: its kernel wrote O)
    if (wi == 0 && (pre || a.n > 0)) {
      const float inv = j.L > 0.f ? 1.f / j.L : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        uint2 out;
        out.x = ptx::pack_bf16x2(j.acc[i].x * inv, j.acc[i].y * inv);
        out.y = ptx::pack_bf16x2(j.acc[i].z * inv, j.acc[i].w * inv);
        reinterpret_cast<uint2*>(o + w * 128)[lane + i * kLanes] = out;
      }
    }
    if (W > 1) __syncthreads();   // the next row's sums replace these
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
  v.stream_o = take((int64_t)v.stream_grid * kStepPipes * kStepPackedRows * 128);
  v.stream_lse = take((int64_t)v.stream_grid * kStepPipes * kStepPackedRows);
  v.tile_o = take((int64_t)v.tile_grid * kStepTileRows * 128);
  v.tile_lse = take((int64_t)v.tile_grid * kStepTileRows);
  v.own_cut = reinterpret_cast<Spills*>(take(2 * (int64_t)max_tokens * s.H_kv));
  v.pre_cut = reinterpret_cast<Spills*>(take(2 * (int64_t)max_tokens * s.H_kv));
  if (w) *w = v;
  return at;
}

namespace {
template <bool kDraft>
cudaError_t launch_stream(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w,
                          const void* q, const void* k_cache, const void* v_cache, void* o,
                          bool first, cudaStream_t st) {
  cudaError_t e;
  // the shared-memory limit is raised once per device
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load() & bit)) {
    e = cudaFuncSetAttribute(step_stream_kernel<kDraft>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(step_stream_kernel<kDraft>,
                               cudaFuncAttributePreferredSharedMemoryCarveout,
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
  return cudaLaunchKernelEx(&cfg, step_stream_kernel<kDraft>, ds, s, w, (const __nv_bfloat16*)q,
                            (const __nv_bfloat16*)k_cache, (const __nv_bfloat16*)v_cache,
                            (__nv_bfloat16*)o, first ? 1 : 0);
}
}  // namespace

cudaError_t launch_step_stream(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w,
                               const void* q, const void* k_cache, const void* v_cache, void* o,
                               bool first, cudaStream_t st) {
  return (ds.place ? launch_stream<true> : launch_stream<false>)(ds, s, w, q, k_cache, v_cache, o,
                                                                 first, st);
}

cudaError_t launch_step_combine(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w,
                                void* o, cudaStream_t st) {
  const bool wide = ds.max_tokens <= kJoinWideRows;
  // one row per warp while all of them fit the SMs at once
  const bool few =
      (int64_t)ds.max_tokens * s.H_q <= (int64_t)w.tile_grid * kJoinBlocks * kJoinWarps;
  const int heads = wide ? 1 : kJoinWarps * (few ? 1 : kJoinVecs);
  const int chunks = (s.H_q + heads - 1) / heads;
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
  auto kernel = ds.place ? (wide  ? step_combine_kernel<kJoinWarps, 1, true>
                            : few ? step_combine_kernel<1, 1, true>
                                  : step_combine_kernel<1, kJoinVecs, true>)
                         : (wide  ? step_combine_kernel<kJoinWarps, 1, false>
                            : few ? step_combine_kernel<1, 1, false>
                                  : step_combine_kernel<1, kJoinVecs, false>);
  return cudaLaunchKernelEx(&cfg, kernel, ds, s, w, (__nv_bfloat16*)o);
}

}  // namespace rbkv
