// Block tables and slot maps of a step, built on the device from the
// requests' lengths, and the return of finished requests' blocks.
//
// Sequence s holds seen[s] tokens and takes n_new[s] more:
//   held = ceil(seen / B), need = ceil((seen + n_new) / B), grow = need - held
//   q_start = exclusive sum of n_new;  first = exclusive sum of grow
//   the k-th new block of the step is the k-th lowest free id (one bit per
//   block, set = free): the rule of the host's block pool, in sequence order
//   row r of sequence s: position = seen + r - q_start[s],
//   slot = table[position / B] * B + position % B
// Three prefix sums (tokens, blocks, free bits) and two scatters: a few
// hundred KB at most, so the time is latency - launches and dependent loads.
#include <algorithm>

#include "rbkv_step.h"

#include <cuda_runtime.h>

namespace rbkv {

namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

constexpr int32_t kErrInvalid = -1, kErrNoBlocks = -2, kErrCapacity = -6;
constexpr int64_t kMaxLen = (int64_t)1 << 30;   // line length of one KV head

// Block counts of a sequence, clamped to its table row (a sequence out of
// range is reported and nothing is scheduled; the clamps keep the copy of its
// row in bounds).
__device__ __forceinline__ void blocks_of(int64_t seen, int64_t n_new, int32_t B,
                                          int32_t max_blocks, int32_t& held, int32_t& need) {
  const int64_t h = seen > 0 ? (seen + B - 1) / B : 0;
  const int64_t c = seen + n_new;
  const int64_t e = c > 0 ? (c + B - 1) / B : 0;
  held = (int32_t)(h < max_blocks ? h : max_blocks);
  need = (int32_t)(e < max_blocks ? e : max_blocks);
}

enum { kTokens = 0, kGrow, kStreamed, kTiled, kStreamLen, kTileLen, kSums };

struct Sums {
  int64_t v[kSums];
};

// One sequence's contribution to the sums; false when its lengths are wrong.
__device__ __forceinline__ int32_t measure(const BuildArgs& a, int32_t seen, int32_t n_new,
                                           Sums& s) {
#pragma unroll
  for (int i = 0; i < kSums; ++i) s.v[i] = 0;
  if (seen < 0 || n_new < 0) return kErrInvalid;
  const int64_t ctx = (int64_t)seen + n_new;
  const int64_t need = (ctx + a.block_size - 1) / a.block_size;
  if (need > a.max_blocks || ctx > 0x7fffffff) return kErrCapacity;
  if (n_new > a.max_tokens) return kErrCapacity;
  s.v[kTokens] = n_new;
  s.v[kGrow] = need - ((int64_t)seen + a.block_size - 1) / a.block_size;
  if (n_new == 0) return 0;
  if ((int64_t)n_new * a.group <= kStepPackedRows) {
    s.v[kStreamed] = 1;
    s.v[kStreamLen] = (ctx + kStepStreamKeys - 1) / kStepStreamKeys + kStepStreamUnit;
  } else {
    s.v[kTiled] = 1;
    s.v[kTileLen] = step_seq_len(seen, n_new, 2 * step_tile_tokens(a.group));
  }
  return 0;
}

struct Shared {
  int64_t sums[kSums];     // this CTA's, read by the other CTAs of the cluster
  int64_t free_bits;
  int32_t err;
  int32_t warp_sum[kSums + 1][kWarps];
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  const uint32_t local = (uint32_t)__cvta_generic_to_shared(p);
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}
__device__ __forceinline__ int64_t remote_i64(const int64_t* p, uint32_t rank) {
  int64_t v;
  asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ int32_t remote_i32(const int32_t* p, uint32_t rank) {
  int32_t v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(remote(p, rank)) : "memory");
  return v;
}

// Exclusive block-wide prefix sums of N counters at once; `total` gets the
// block's sums.  Every thread of the block calls it.
template <int N>
__device__ __forceinline__ void block_scan(int32_t (&v)[N], int32_t (&total)[N], Shared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t inc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) inc[i] = v[i];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int32_t up = __shfl_up_sync(0xffffffffu, inc[i], off);
      if (lane >= off) inc[i] += up;
    }
  }
  __syncthreads();   // the previous use of warp_sum is over
  if (lane == 31) {
#pragma unroll
    for (int i = 0; i < N; ++i) sh.warp_sum[i][warp] = inc[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int32_t w = lane < kWarps ? sh.warp_sum[i][lane] : 0;
    int32_t sum = w, before = lane < warp ? w : 0;
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, off);
      before += __shfl_xor_sync(0xffffffffu, before, off);
    }
    total[i] = sum;
    v[i] = inc[i] - v[i] + before;
  }
}

// The first cluster of the grid builds the step; every further CTA copies the
// part of the table that no sequence grows into (when the table is not built
// in place).  The eight CTAs of the building cluster each own a slice of the
// sequences and of the bitmap, exchange their sums through distributed shared
// memory, and meet again once the new ids are written.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    build_kernel(BuildArgs a) {
  __shared__ Shared sh;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31;
  const int S = a.num_seqs, B = a.block_size;

  if (blockIdx.x >= kCluster) {
    const int64_t warps = (int64_t)(gridDim.x - kCluster) * kWarps;
    for (int64_t s = (int64_t)(blockIdx.x - kCluster) * kWarps + (tid >> 5); s < S; s += warps) {
      int32_t held, need;
      blocks_of(a.seen[s], a.n_new[s], B, a.max_blocks, held, need);
      const int32_t* src = a.table_in + s * a.max_blocks;
      int32_t* dst = a.table + s * a.max_blocks;
#pragma unroll 4
      for (int c = lane; c < a.max_blocks; c += 32)
        if (c < held || c >= need) dst[c] = src[c];
    }
    return;
  }

  const StepPlan plan = step_plan(a.plan, S, a.max_tokens);
  const uint32_t rank = cluster_rank();
  const int per = (S + kCluster - 1) / kCluster;
  const int s0 = min((int)rank * per, S), s1 = min(s0 + per, S);
  const int W = (a.num_blocks + 31) / 32;
  const int wper = (W + kCluster - 1) / kCluster;
  const int w0 = min((int)rank * wper, W), w1 = min(w0 + wper, W);
  // bits past the pool's last block count for nothing
  auto pool_word = [&](int w) -> uint32_t {
    const uint32_t x = (uint32_t)a.free_in[w];
    const int left = a.num_blocks - w * 32;
    return left >= 32 ? x : x & ((1u << left) - 1u);
  };

  // ---- this CTA's sums ----
  Sums mine = {};
  int64_t bits = 0;
  int32_t err = 0;
  for (int s = s0 + tid; s < s1; s += kThreads) {
    Sums x;
    err = min(err, measure(a, a.seen[s], a.n_new[s], x));
#pragma unroll
    for (int i = 0; i < kSums; ++i) mine.v[i] += x.v[i];
  }
  for (int w = w0 + tid; w < w1; w += kThreads) bits += __popc(pool_word(w));
  if (tid < kSums) sh.sums[tid] = 0;
  if (tid == 0) {
    sh.free_bits = 0;
    sh.err = 0;
  }
  __syncthreads();
#pragma unroll
  for (int off = 16; off; off >>= 1) {
#pragma unroll
    for (int i = 0; i < kSums; ++i) mine.v[i] += __shfl_xor_sync(0xffffffffu, mine.v[i], off);
    bits += __shfl_xor_sync(0xffffffffu, bits, off);
    err = min(err, __shfl_xor_sync(0xffffffffu, err, off));
  }
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kSums; ++i)
      atomicAdd((unsigned long long*)&sh.sums[i], (unsigned long long)mine.v[i]);
    atomicAdd((unsigned long long*)&sh.free_bits, (unsigned long long)bits);
    atomicMin(&sh.err, err);
  }
  cluster_sync();

  // ---- the cluster's sums, and those before this CTA ----
  int64_t total[kSums], before[kSums], free_total = 0, free_before = 0;
  err = 0;
#pragma unroll
  for (int i = 0; i < kSums; ++i) total[i] = before[i] = 0;
  for (uint32_t r = 0; r < kCluster; ++r) {
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
      const int64_t x = remote_i64(&sh.sums[i], r);
      total[i] += x;
      before[i] += r < rank ? x : 0;
    }
    const int64_t f = remote_i64(&sh.free_bits, r);
    free_total += f;
    free_before += r < rank ? f : 0;
    err = min(err, remote_i32(&sh.err, r));
  }
  if (err == 0 && (total[kTokens] > a.max_tokens || total[kStreamLen] > kMaxLen ||
                   total[kTileLen] > kMaxLen))
    err = kErrCapacity;
  if (err == 0 && total[kGrow] > free_total) err = kErrNoBlocks;
  const bool ok = err == 0;
  const int32_t T = ok ? (int32_t)total[kTokens] : 0;
  const int32_t grow_total = ok ? (int32_t)total[kGrow] : 0;

  // ---- per sequence: offsets and work lists ----
  int32_t carry[kSums];
#pragma unroll
  for (int i = 0; i < kSums; ++i) carry[i] = ok ? (int32_t)before[i] : 0;
  for (int base = s0; base < s1; base += kThreads) {
    const int s = base + tid;
    const bool live = s < s1;
    const int32_t seen = live ? a.seen[s] : 0, n_new = live ? a.n_new[s] : 0;
    if (!ok) {
      if (live) {
        int32_t held, need;
        blocks_of(seen, n_new, B, a.max_blocks, held, need);
        if (a.table != a.table_in)
          for (int c = held; c < need; ++c)
            a.table[(int64_t)s * a.max_blocks + c] = a.table_in[(int64_t)s * a.max_blocks + c];
        a.ctx[s] = seen;
        a.q_start[s] = 0;
      }
      continue;
    }
    Sums x;
    measure(a, seen, n_new, x);
    int32_t v[kSums], sum[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) v[i] = (int32_t)x.v[i];
    block_scan<kSums>(v, sum, sh);
    if (live) {
#pragma unroll
      for (int i = 0; i < kSums; ++i) v[i] += carry[i];
      a.ctx[s] = seen + n_new;
      a.q_start[s] = v[kTokens];
      StepRow of = {0, v[kGrow], 0, 0};
      StepSeq e = {s, v[kTokens], n_new, seen + n_new, 0, 0, {0, 0}};
      if (x.v[kStreamed]) {
        of.unit = v[kStreamed];
        of.cum = e.cum = v[kStreamLen];
        of.tiles = e.tiles = (int32_t)x.v[kStreamLen] - kStepStreamUnit;
        plan.streamed[of.unit] = e;
      } else if (x.v[kTiled]) {
        of.unit = -1 - v[kTiled];
        of.cum = e.cum = v[kTileLen];
        of.tiles = e.tiles = (int32_t)x.v[kTileLen];
        plan.tiled[v[kTiled]] = e;
      }
      plan.of_seq[s] = of;
    }
#pragma unroll
    for (int i = 0; i < kSums; ++i) carry[i] += sum[i];
  }
  if (rank == 0 && tid == 0) {
    a.q_start[S] = T;
    plan.header[kPlanRows] = T;
    plan.header[kPlanStreamed] = ok ? (int32_t)total[kStreamed] : 0;
    plan.header[kPlanTiled] = ok ? (int32_t)total[kTiled] : 0;
    plan.header[kPlanStreamLen] = ok ? (int32_t)total[kStreamLen] : 0;
    plan.header[kPlanTileLen] = ok ? (int32_t)total[kTileLen] : 0;
    if (!ok) atomicCAS(a.status, 0, err);
  }

  // ---- the lowest free ids, taken out of the bitmap ----
  int32_t rank0 = (int32_t)min(free_before, (int64_t)0x7fffffff);
  for (int base = w0; base < w1; base += kThreads) {
    const int w = base + tid;
    const bool live = w < w1;
    const uint32_t pool = live ? pool_word(w) : 0u;
    int32_t v[1] = {__popc(pool)}, sum[1];
    block_scan<1>(v, sum, sh);
    if (live) {
      uint32_t taken = 0, left = pool;
      int32_t k = rank0 + v[0];
      while (left && k < grow_total) {
        const int b = __ffs(left) - 1;
        left &= left - 1;
        taken |= 1u << b;
        plan.new_ids[k++] = w * 32 + b;
      }
      a.free_words[w] = (int32_t)((uint32_t)a.free_in[w] & ~taken);
    }
    rank0 += sum[0];
  }
  cluster_sync();

  // ---- rows: positions, slots, and the entry of each block that begins ----
  for (int r = (int)rank * kThreads + tid; r < a.max_tokens; r += kCluster * kThreads) {
    if (r >= T) {
      a.position[r] = -1;
      a.slot[r] = -1;
      continue;
    }
    // the last sequence that starts at or before row r and is not empty: the
    // first one that ends behind it
    int lo = 0, hi = S - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.q_start[mid + 1] > r) hi = mid;
      else lo = mid + 1;
    }
    const int s = lo;
    const int q0 = a.q_start[s], n = a.q_start[s + 1] - q0;
    const int seen = a.ctx[s] - n, pos = seen + r - q0;
    const int held = (int)(((int64_t)seen + B - 1) / B);
    const int c = pos / B, off = pos - c * B;
    StepRow of = plan.of_seq[s];
    int32_t id;
    if (c < held) {
      id = a.table_in[(int64_t)s * a.max_blocks + c];
    } else {
      id = plan.new_ids[of.token + c - held];
      if (off == 0) a.table[(int64_t)s * a.max_blocks + c] = id;
    }
    of.token = r - q0;
    plan.rows[r] = of;
    a.position[r] = pos;
    if (id < 0 || id >= a.num_blocks) {
      atomicCAS(a.status, 0, kDevBounds);
      a.slot[r] = -1;
    } else {
      a.slot[r] = id * B + off;
    }
  }
}

// One warp per sequence: its blocks' bits are set again (an or: the order of
// the sequences does not matter).
__global__ void __launch_bounds__(256)
    release_kernel(BuildArgs a, const int32_t* __restrict__ done) {
  const int s = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  if (s >= a.num_seqs || done[s] == 0) return;
  const int32_t ctx = a.ctx[s];
  int32_t held, need;
  blocks_of(ctx, 0, a.block_size, a.max_blocks, held, need);
  for (int c = lane; c < held; c += 32) {
    const int32_t id = a.table[(int64_t)s * a.max_blocks + c];
    if (id < 0 || id >= a.num_blocks)
      atomicCAS(a.status, 0, kDevBounds);
    else
      atomicOr((unsigned int*)&a.free_words[id >> 5], 1u << (id & 31));
  }
  __syncwarp();
  if (lane == 0) a.ctx[s] = 0;
}

}  // namespace

cudaError_t launch_step_build(const BuildArgs& a, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int copies = 0;
  if (a.table != a.table_in) {
    const int64_t warps = a.num_seqs;
    copies = (int)std::min<int64_t>((warps + kWarps - 1) / kWarps, std::max(1, 2 * sms));
    copies = (copies + kCluster - 1) / kCluster * kCluster;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster + copies);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, build_kernel, a);
}

cudaError_t launch_step_release(const BuildArgs& a, const int32_t* done, cudaStream_t st) {
  release_kernel<<<(unsigned)((a.num_seqs + 7) / 8), 256, 0, st>>>(a, done);
  return cudaGetLastError();
}

}  // namespace rbkv
