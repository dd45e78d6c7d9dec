// Drafted tokens of a step: the trees' plans, the acceptance of a path, and the
// kept rows' move.
//
// Plan: token i of a sequence follows parent[i] < i.  A(i) = {i} and A(parent[i]),
// a set of at most 128 bits; depth(i) = |A(i)| - 1, place = seen + depth.  The sets
// grow by doubling: S(i) starts as {i} with a pointer to the parent; a round
// unites S(i) with the set that the pointer names and follows that one's pointer,
// so S(i) holds the nearest 2^k tokens of the path after k rounds: as many rounds
// as the greatest depth has bits, 7 at most.
//
// Acceptance: from the last given token, the lowest child whose token is the
// one chosen, until there is none.  (i is a child of c when c is the highest bit
// of A(i) below i.)  A warp holds a sequence's tree in registers, four tokens to a
// lane.  Let M be the tokens that are the choice at their parents; then the path
// holds those tokens that follow the last given one and have no ancestor behind it
// outside M - all of them at once, in votes.  Only where siblings are alike does
// that find more than a path (a token on it is then not the parent of the next), and
// the path is walked, a broadcast, four compares and votes to a step: of 256 trees
// of up to 60 tokens, chains among them, 15 us, where the votes take 5.  The new
// blocks' bits are written as the path leaves them, held or free (0.1 to 0.25 us
// more than setting the free ones alone), so that a second acceptance may keep more
// than the first.
//
// Move: kept token d of a sequence lies in the slot of token p_d >= d, and
// goes to the slot of token d.  p rises, so a row is never written before it has
// been read when a thread moves its columns in the order of d.
//
// All three are latency: a few dependent loads, for a few KB (acceptance and move of
// 16 trees of 8 in a graph 3.5 and 2.8 us, of 256 of 60 5.1 and 3.2).
#include <algorithm>

#include "rbkv_step.h"
#include "rbkv_ptx.cuh"

#include <cuda_runtime.h>

namespace rbkv {

namespace {

constexpr int kNodes = kStepTreeTokens;
constexpr int kPlanThreads = kNodes;
constexpr int kMoveThreads = 128;
constexpr uint32_t kAll = 0xffffffffu;

// Whether the step was built for these tables; else, if it has rows, it is
// recorded as RBKV_ERR_INVALID.  `stage`: what must have been done to its trees.
enum { kBuilt, kPlanned, kAccepted };
__device__ __forceinline__ bool usable(const DraftArgs& a, const StepPlan& plan, int stage) {
  const int32_t* h = plan.header;
  const StepLanes* done = reinterpret_cast<const StepLanes*>(a.work);
  const bool ok = h[kPlanSeqs] == a.num_seqs && h[kPlanTokens] == a.max_tokens &&
                  h[kPlanMaxBlocks] == a.max_blocks && h[kPlanBlock] == a.block_size &&
                  h[kPlanPool] == a.num_blocks &&
                  (stage < kPlanned || done->single_cum == h[kPlanSerial]) &&
                  (stage < kAccepted || done->pair_cum == h[kPlanSerial]);
  if (!ok && threadIdx.x == 0 && h[kPlanRows] > 0) atomicCAS(a.status, 0, kDevInvalid);
  return ok;
}

// The tiled sequences' places on the tile kernel's road: a scan over them, a run of
// sequences to a thread.
__device__ __forceinline__ void plan_lanes(const DraftArgs& a, const StepPlan& plan) {
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ int sums[2][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  StepLanes* out = reinterpret_cast<StepLanes*>(a.work);
  const int n = plan.header[kPlanTiled], tokens = step_tile_tokens(plan.header[kPlanGroup]);
  const int per = (n + kPlanThreads - 1) / kPlanThreads;
  const int i0 = min(tid * per, n), i1 = min(i0 + per, n);
  auto lengths = [&](int i, int& single, int& pair) {
    const StepSeq e = plan.tiled[i];
    const int seen = e.ctx - e.n_new, pairs = step_pairs(seen, e.n_new, tokens);
    single = step_singles_len(seen, e.n_new, tokens, pairs);
    pair = step_pairs_len(seen, e.n_new, tokens, pairs);
  };
  // (the first few sequences of a thread are kept for the second pass)
  constexpr int kHeld = 4;
  int mine[2] = {0, 0}, at[2], held[2][kHeld];
#pragma unroll
  for (int x = 0; x < kHeld; ++x) {
    held[0][x] = held[1][x] = 0;
    if (i0 + x < i1) lengths(i0 + x, held[0][x], held[1][x]);
    mine[0] += held[0][x];
    mine[1] += held[1][x];
  }
  for (int i = i0 + kHeld; i < i1; ++i) {
    int single, pair;
    lengths(i, single, pair);
    mine[0] += single;
    mine[1] += pair;
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    at[x] = mine[x];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int up = __shfl_up_sync(kAll, at[x], off);
      if (lane >= off) at[x] += up;
    }
    if (lane == 31) sums[x][warp] = at[x];
  }
  __syncthreads();
  int total[2] = {0, 0};
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    at[x] -= mine[x];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at[x] += sums[x][w];
      total[x] += sums[x][w];
    }
  }
  auto put = [&](int i, int single, int pair) {
    out[1 + i] = StepLanes{at[0], single, at[1], pair};
    at[0] += single;
    at[1] += pair;
  };
#pragma unroll
  for (int x = 0; x < kHeld; ++x)
    if (i0 + x < i1) put(i0 + x, held[0][x], held[1][x]);
  for (int i = i0 + kHeld; i < i1; ++i) {
    int single, pair;
    lengths(i, single, pair);
    put(i, single, pair);
  }
  const int serial = plan.header[kPlanSerial];
  if (tid == 0) out[0] = StepLanes{serial, total[0], ~serial, total[1]};
}

__global__ void __launch_bounds__(kPlanThreads) draft_plan_kernel(DraftArgs a) {
  __shared__ uint4 set[kNodes];
  __shared__ int next[kNodes];
  ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  const StepPlan plan = step_plan(a.plan, a.num_seqs, a.max_tokens);
  if (!usable(a, plan, kBuilt)) return;
  const int tid = threadIdx.x;
  if (blockIdx.x == gridDim.x - 1) {      // (one block more than the trees')
    plan_lanes(a, plan);
    return;
  }
  const int blocks = gridDim.x - 1;
  const int T = plan.header[kPlanRows];
  uint4* sets = reinterpret_cast<uint4*>(a.ancestors);
  for (int64_t r = T + (int64_t)blockIdx.x * kPlanThreads + tid; r < a.max_tokens;
       r += (int64_t)blocks * kPlanThreads) {
    a.place[r] = -1;
    sets[r] = make_uint4(0, 0, 0, 0);
  }
  for (int s = blockIdx.x; s < a.num_seqs; s += blocks) {
    const int q0 = a.q_start[s], n = a.q_start[s + 1] - q0;
    if (n == 0) continue;
    const int seen = a.position[q0];
    if (n > kNodes) {
      bool bad = false;
      for (int i = tid; i < n; i += kPlanThreads) {
        bad |= a.parent[q0 + i] != i - 1;
        a.place[q0 + i] = seen + i;
        sets[q0 + i] = make_uint4(0, 0, 0, 0);
      }
      if (bad) atomicCAS(a.status, 0, kDevInvalid);
      continue;
    }
    const bool mine = tid < n;
    int p = mine ? a.parent[q0 + tid] : -1;
    const bool ok = !mine || (p >= -1 && p < tid);
    // (also: the previous sequence's sets are no longer needed)
    if (!__syncthreads_and(ok)) {
      p = mine ? tid - 1 : -1;
      if (tid == 0) atomicCAS(a.status, 0, kDevInvalid);
    }
    uint4 m = make_uint4(tid < 32 ? 1u << tid : 0u, (tid >> 5) == 1 ? 1u << (tid & 31) : 0u,
                         (tid >> 5) == 2 ? 1u << (tid & 31) : 0u,
                         (tid >> 5) == 3 ? 1u << (tid & 31) : 0u);
    set[tid] = m;
    next[tid] = p;
    while (__syncthreads_or(p >= 0)) {
      uint4 o = make_uint4(0, 0, 0, 0);
      if (p >= 0) {
        o = set[p];
        p = next[p];
      }
      m = make_uint4(m.x | o.x, m.y | o.y, m.z | o.z, m.w | o.w);
      __syncthreads();
      set[tid] = m;
      next[tid] = p;
    }
    if (mine) {
      a.place[q0 + tid] = seen + __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w) - 1;
      sets[q0 + tid] = m;
    }
  }
}

// The highest bit of a set below bit i; -1 if there is none.
__device__ __forceinline__ int parent_of(const uint4& m, int i) {
  const uint32_t w[4] = {m.x, m.y, m.z, m.w};
  int best = -1;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int below = i - 32 * x;      // bits of this word that lie below i
    const uint32_t v = below <= 0 ? 0u : below >= 32 ? w[x] : w[x] & ((1u << below) - 1u);
    if (v) best = 32 * x + 31 - __clz(v);
  }
  return best;
}

constexpr int kAcceptWarps = 4;

__global__ void __launch_bounds__(kAcceptWarps * 32) draft_accept_kernel(DraftArgs a) {
  ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  const StepPlan plan = step_plan(a.plan, a.num_seqs, a.max_tokens);
  if (!usable(a, plan, kPlanned)) return;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0)
    reinterpret_cast<StepLanes*>(a.work)->pair_cum = plan.header[kPlanSerial];
  const int T = plan.header[kPlanRows];
  const bool turned = plan.header[kPlanTurned] == plan.header[kPlanSerial];
  for (int64_t r = T + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < a.max_tokens;
       r += (int64_t)gridDim.x * blockDim.x)
    a.path[r] = -1;
  const int warps = gridDim.x * kAcceptWarps;
  for (int s = blockIdx.x * kAcceptWarps + (threadIdx.x >> 5); s < a.num_seqs; s += warps) {
    const int q0 = a.q_start[s], n = a.q_start[s + 1] - q0, length = a.ctx[s];
    // (a sequence with new tokens has a length, unless it has been released since: its
    // blocks are free, and it keeps nothing)
    if (n == 0 || length == 0) {
      for (int i = lane; i < n; i += 32) a.path[q0 + i] = -1;
      if (lane == 0) {
        a.accepted[s] = 0;
        a.next_token[s] = -1;
      }
      continue;
    }
    const int seen = a.position[q0];
    int given = a.given ? a.given[s] : 1;
    if (given < 1 || given > n) {
      if (lane == 0) atomicCAS(a.status, 0, kDevInvalid);
      given = given < 1 ? 1 : n;
    }
    int kept = given, cur = given - 1, next;
    if (n <= kNodes) {
      // token lane + 32 x of the tree, its parent, and the token chosen there
      int parent[4], token[4], chosen[4], path[4];
      uint4 set[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = lane + 32 * x;
        parent[x] = -1;
        token[x] = chosen[x] = 0;
        path[x] = i;
        set[x] = make_uint4(0, 0, 0, 0);
        if (i < n) {
          set[x] = reinterpret_cast<const uint4*>(a.ancestors)[q0 + i];
          parent[x] = parent_of(set[x], i);
          token[x] = a.tokens[q0 + i];
          chosen[x] = a.chosen[q0 + i];
        }
      }
      // Rows that were rotated by their places: a given token that does not follow the one
      // before it would come to lie at another position.
      if (turned && given > 1) {
        int chain = given;
#pragma unroll
        for (int x = 3; x >= 0; --x) {
          const int i = lane + 32 * x;
          const uint32_t v = __ballot_sync(kAll, i >= 1 && i < given && parent[x] != i - 1);
          if (v) chain = 32 * x + __ffs(v) - 1;
        }
        if (chain < given) {
          if (lane == 0) atomicCAS(a.status, 0, kDevInvalid);
          kept = given = chain;
          cur = given - 1;
        }
      }
      // M, and the path
      const int words = (n + 31) >> 5;
      uint32_t good[4], on[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        good[x] = on[x] = 0;
        if (x >= words) continue;
        int want = 0;
#pragma unroll
        for (int y = 0; y <= x; ++y) {
          const int c = __shfl_sync(kAll, chosen[y], parent[x] & 31);
          if ((parent[x] >> 5) == y) want = c;
        }
        good[x] = __ballot_sync(kAll, parent[x] >= 0 && token[x] == want);
      }
      int before = cur;                  // the path's last token so far
      bool single = true;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (x >= words) continue;
        const uint32_t w[4] = {set[x].x, set[x].y, set[x].z, set[x].w};
        bool follows = false, all = true;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int from = given - 32 * y;         // bits of this word that are given
          const uint32_t behind = from <= 0 ? kAll : from >= 32 ? 0u : kAll << from;
          if ((cur >> 5) == y) follows = w[y] >> (cur & 31) & 1u;
          all &= (w[y] & behind & ~good[y]) == 0;
        }
        on[x] = __ballot_sync(kAll, lane + 32 * x >= given && follows && all);
        // each token's parent has to be the one before it
        const uint32_t below = on[x] & ((1u << lane) - 1u);
        const int last = below ? 32 * x + 31 - __clz(below) : before;
        single &= !(on[x] >> lane & 1u) || parent[x] == last;
        if (on[x]) before = 32 * x + 31 - __clz(on[x]);
      }
      if (__all_sync(kAll, single)) {
        // token i of the path's tokens goes to place kept + its rank among them
        int rank = given;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (x >= words) continue;
          if (lane + 32 * x < given) a.path[q0 + lane + 32 * x] = q0 + lane + 32 * x;
          if (on[x] >> lane & 1u)
            a.path[q0 + rank + __popc(on[x] & ((1u << lane) - 1u))] = q0 + lane + 32 * x;
          rank += __popc(on[x]);
        }
        kept = rank;
        cur = before;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int i = lane + 32 * x;
          if (i >= kept && i < n) a.path[q0 + i] = -1;
        }
        next = chosen[0];
#pragma unroll
        for (int x = 1; x < 4; ++x)
          if ((cur >> 5) == x) next = chosen[x];
        next = __shfl_sync(kAll, next, cur & 31);
      } else {
        while (true) {
          int want = chosen[0];
#pragma unroll
          for (int x = 1; x < 4; ++x)
            if ((cur >> 5) == x) want = chosen[x];
          want = __shfl_sync(kAll, want, cur & 31);
          next = want;
          int child = -1;
#pragma unroll
          for (int x = 3; x >= 0; --x) {
            if (32 * x >= n) continue;
            const uint32_t v = __ballot_sync(kAll, parent[x] == cur && token[x] == want);
            if (v) child = 32 * x + __ffs(v) - 1;
          }
          if (child < 0) break;
          cur = child;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (lane + 32 * x == kept) path[x] = child;
          ++kept;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int i = lane + 32 * x;
          if (i < n) a.path[q0 + i] = i < kept ? q0 + path[x] : -1;
        }
      }
    } else {
      // a chain: up to the first token that is not the one chosen before it
      kept = n;
      for (int i0 = given; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t v =
            __ballot_sync(kAll, i < n && a.tokens[q0 + i] != a.chosen[q0 + i - 1]);
        if (v) {
          kept = i0 + __ffs(v) - 1;
          break;
        }
      }
      for (int i = lane; i < n; i += 32) a.path[q0 + i] = i < kept ? q0 + i : -1;
      next = a.chosen[q0 + kept - 1];
    }
    if (lane == 0) {
      a.accepted[s] = kept;
      a.next_token[s] = next;
      a.ctx[s] = seen + kept;
    }
    // The step's new blocks: those behind the kept tokens are free, the others held
    // (an earlier acceptance of this step may have freed them).  Bits that no other
    // warp changes: the order does not matter.
    const uint32_t B = (uint32_t)a.block_size;
    const int first = (int)(((uint32_t)seen + B - 1) / B);
    const int from = (int)(((uint32_t)(seen + kept) + B - 1) / B);
    const int to = (int)(((uint32_t)(seen + n) + B - 1) / B);
    for (int c = first + lane; c < to; c += 32) {
      const int32_t id = a.table[(int64_t)s * a.max_blocks + c];
      if (id < 0 || id >= a.num_blocks) {
        atomicCAS(a.status, 0, kDevBounds);
        continue;
      }
      unsigned int* word = (unsigned int*)&a.free_words[id >> 5];
      if (c < from)
        atomicAnd(word, ~(1u << (id & 31)));
      else
        atomicOr(word, 1u << (id & 31));
    }
  }
}

// A block: 128 of a sequence's 2 H_kv D / 8 (bf16) 16-byte columns.  A warp
// looks 32 kept tokens up at a time, a lane each, and moves those that are not
// in their places, four in flight.
__global__ void __launch_bounds__(kMoveThreads)
    draft_compact_kernel(DraftArgs a, int32_t H_kv, int32_t vec_per_row, uint4* k_cache,
                         uint4* v_cache) {
  ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  const StepPlan plan = step_plan(a.plan, a.num_seqs, a.max_tokens);
  if (!usable(a, plan, kAccepted)) return;
  const int lane = threadIdx.x & 31;
  const int per = H_kv * vec_per_row;
  const int column = blockIdx.x * kMoveThreads + threadIdx.x;
  const bool live = column < 2 * per;
  uint4* cache = column < per ? k_cache : v_cache;
  const int c = column < per ? column : column - per;
  const int head = c / vec_per_row, vec = c - head * vec_per_row;
  auto at = [&](int slot) {
    const int blk = slot / a.block_size;
    return (((int64_t)blk * H_kv + head) * a.block_size + (slot - blk * a.block_size)) *
               vec_per_row + vec;
  };
  for (int s = blockIdx.y; s < a.num_seqs; s += gridDim.y) {
    const int q0 = a.q_start[s], kept = min(a.accepted[s], a.q_start[s + 1] - q0);
    for (int d0 = 0; d0 < kept; d0 += 32) {
      const int d = d0 + lane;
      int from = -1, to = -1;
      if (d < kept) {
        const int row = a.path[q0 + d];
        // (rows of this sequence only, whatever the array holds)
        if (row > q0 + d && row < a.q_start[s + 1]) {
          from = a.slot[row];
          to = a.slot[q0 + d];
          const int slots = a.num_blocks * a.block_size;
          if (from < 0 || to < 0 || from >= slots || to >= slots) {
            atomicCAS(a.status, 0, kDevBounds);
            from = to = -1;
          }
        }
      }
      uint32_t moves = __ballot_sync(kAll, to >= 0);
      while (moves) {
        uint4 v[4];
        int64_t dst[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          dst[u] = -1;
          if (!moves) continue;
          const int x = __ffs(moves) - 1;
          moves &= moves - 1;
          const int src = __shfl_sync(kAll, from, x);
          dst[u] = at(__shfl_sync(kAll, to, x));
          if (live) v[u] = cache[at(src)];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (live && dst[u] >= 0) cache[dst[u]] = v[u];
      }
    }
  }
}

template <class... Args, class... Given>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t st,
                   Given... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_draft_plan(const DraftArgs& a, cudaStream_t st) {
  const int blocks = std::min(a.num_seqs, 1 << 16);
  return launch(draft_plan_kernel, dim3((unsigned)blocks + 1), kPlanThreads, st, a);
}

cudaError_t launch_draft_accept(const DraftArgs& a, cudaStream_t st) {
  const int blocks = std::min((a.num_seqs - 1) / kAcceptWarps + 1, 1 << 16);
  return launch(draft_accept_kernel, dim3((unsigned)blocks), kAcceptWarps * 32, st, a);
}

cudaError_t launch_draft_compact(const DraftArgs& a, const ShapeInfo& s, void* k_cache,
                                 void* v_cache, cudaStream_t st) {
  const int vec = s.D * (s.dtype == 0 ? 2 : 4) / 16;
  const int64_t columns = 2 * (int64_t)s.H_kv * vec;
  const dim3 grid((unsigned)((columns + kMoveThreads - 1) / kMoveThreads),
                  (unsigned)std::min(a.num_seqs, 65535));
  return launch(draft_compact_kernel, grid, kMoveThreads, st, a, s.H_kv, (int32_t)vec,
                (uint4*)k_cache, (uint4*)v_cache);
}

}  // namespace rbkv
