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
// hundred KB, so the time is latency - the launch and about eight dependent
// memory accesses and block barriers (3.9 us for 16 sequences, 6.6 for 512 of up
// to 8192 tokens).  Only a table that is copied on the way is traffic: 4096
// sequences of 513 entries in a pool of 1.3 million blocks, 17 MB, 16.8 us.
#include <algorithm>
#include <atomic>

#include "rbkv_step.h"

#include <cuda_runtime.h>

namespace rbkv {

namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
// What one CTA builds; larger steps take a cluster.  One CTA against eight, us:
// 16 sequences 3.9 / 10.3, 512 6.6 / 10.9, 1024 10.2 / 10.9, 1536 14.7 / 11.1,
// 4096 47 / 12.3; 512 sequences in a pool of 524,288 blocks 10.5 / 11.5, of a
// million 15.4 / 11.8; 64 sequences with a prompt of 8192 rows 14.4 / 21.9 (a
// sequence's rows are one CTA's).
constexpr int kOneSeqs = 1024, kOneBlocks = 524288, kOneRows = 8192;
constexpr int kSmemSeqs = 2048;       // sequences of a CTA whose offsets stay on chip

constexpr int32_t kErrInvalid = kDevInvalid, kErrNoBlocks = -2, kErrCapacity = -6;
// Tokens of a sequence, at most.
constexpr uint32_t kMaxTokens = 1u << 30;
// Lengths of the work lines of one KV head, and rows, stay below this.
constexpr float kMaxLen = 1073741824.f;

// Block counts of a sequence, clamped to its table row (a sequence out of
// range is reported and nothing is scheduled; the clamps keep the copy of its
// row in bounds).
__device__ __forceinline__ void blocks_of(int32_t seen, int32_t n_new, int32_t B,
                                          int32_t max_blocks, int32_t& held, int32_t& need) {
  const int64_t c = (int64_t)seen + n_new;
  const int64_t h = seen > 0 ? step_div((int64_t)seen + B - 1, B) : 0;
  const int64_t e = c > 0 ? step_div(c + B - 1, B) : 0;
  held = (int32_t)(h < max_blocks ? h : max_blocks);
  need = (int32_t)(e < max_blocks ? e : max_blocks);
}

enum { kTokens = 0, kGrow, kStreamed, kTiled, kStreamLen, kTileLen, kFreeBits, kSums };

// One sequence's contribution to the sums (0 where its lengths are wrong).
__device__ __forceinline__ int32_t measure(const BuildArgs& a, int32_t seen, int32_t n_new,
                                           int32_t (&v)[kSums]) {
#pragma unroll
  for (int i = 0; i < kSums; ++i) v[i] = 0;
  if (seen < 0 || n_new < 0) return kErrInvalid;
  const uint32_t ctx = (uint32_t)seen + (uint32_t)n_new, B = (uint32_t)a.block_size;
  if (ctx > kMaxTokens || n_new > a.max_tokens) return kErrCapacity;
  const uint32_t need = (ctx + B - 1) / B;
  if (need > (uint32_t)a.max_blocks) return kErrCapacity;
  v[kTokens] = n_new;
  v[kGrow] = (int32_t)(need - ((uint32_t)seen + B - 1) / B);
  if (n_new == 0) return 0;
  if ((int64_t)n_new * a.group <= kStepPackedRows) {
    v[kStreamed] = 1;
    v[kStreamLen] = (int32_t)((ctx + kStepStreamKeys - 1) / kStepStreamKeys) + kStepStreamUnit;
  } else {
    v[kTiled] = 1;
    const int64_t len = step_seq_len(seen, n_new, step_tile_tokens(a.group));
    if (len >= (int64_t)kMaxLen) return kErrCapacity;
    v[kTileLen] = (int32_t)len;
  }
  return 0;
}

struct Shared {
  int32_t sums[kSums];     // this CTA's, read by the other CTAs of the cluster
  float big;               // an upper bound of the sums that could overflow
  int32_t err;
  int32_t warp_sum[kSums][kWarps];
  float warp_big[kWarps];
  int32_t warp_err[kWarps];
  int32_t q_start[kSmemSeqs + 1];
  int32_t seen[kSmemSeqs];
  StepRow of[kSmemSeqs];
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// (also orders the CTAs' global writes before the reads that follow it)
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote_b32(const void* p, uint32_t rank) {
  const uint32_t local = (uint32_t)__cvta_generic_to_shared(p);
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(local), "r"(rank));
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// C CTAs (one, or a cluster of eight) build the step, each a slice of the
// sequences and of the bitmap; every further CTA copies the part of the table
// that no sequence grows into (when the table is not built in place).  A
// thread owns consecutive sequences and bitmap words, so one block-wide scan
// of all sums gives every offset; the CTAs exchange their totals through
// distributed shared memory and meet again once the new ids are written.
// One CTA has no cluster barrier and no exchange: it is the faster one up to
// the sizes that its caller allows it.
template <int C>
__global__ void __launch_bounds__(kThreads) build_kernel(BuildArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = a.num_seqs, B = a.block_size;

  if (blockIdx.x >= C) {
    const int warps = (gridDim.x - C) * kWarps;
    for (int s = (blockIdx.x - C) * kWarps + warp; s < S; s += warps) {
      int32_t held, need;
      blocks_of(a.seen[s], a.n_new[s], B, a.max_blocks, held, need);
      const int32_t* src = a.table_in + (int64_t)s * a.max_blocks;
      int32_t* dst = a.table + (int64_t)s * a.max_blocks;
#pragma unroll 4
      for (int c = lane; c < a.max_blocks; c += 32)
        if (c < held || c >= need) dst[c] = src[c];
    }
    return;
  }

  const StepPlan plan = step_plan(a.plan, S, a.max_tokens);
  const uint32_t rank = C > 1 ? cluster_rank() : 0;
  const int per = (S + C - 1) / C;
  const int s0 = min((int)rank * per, S), n_seqs = min(per, S - s0);
  const int W = (a.num_blocks - 1) / 32 + 1;      // (num_blocks + 31 may pass 2^31)
  const int wper = (W + C - 1) / C;
  const int w0 = min((int)rank * wper, W), n_words = min(wper, W - w0);
  // this thread's sequences [sa, sb) and this warp's words [wa, wb) of the CTA's
  const int ks = (n_seqs + kThreads - 1) / kThreads;
  const int sa = min(tid * ks, n_seqs), sb = min(sa + ks, n_seqs);
  const int kw = ((n_words + kWarps - 1) / kWarps + 31) & ~31;
  const int wa = min(warp * kw, n_words), wb = min(wa + kw, n_words);
  const bool on_chip = n_seqs <= kSmemSeqs;
  // bits past the pool's last block count for nothing
  auto pool_word = [&](int w) -> uint32_t {
    const uint32_t x = (uint32_t)a.free_in[w];
    const int left = a.num_blocks - w * 32;
    return left >= 32 ? x : x & ((1u << left) - 1u);
  };

  const int32_t serial = rank == 0 && tid == 0 ? plan.header[kPlanSerial] : 0;

  // ---- the thread's sums, and their scan over the block ----
  int32_t mine[kSums], err = 0;
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < kSums; ++i) mine[i] = 0;
  for (int i = sa; i < sb; ++i) {
    int32_t v[kSums];
    err = min(err, measure(a, a.seen[s0 + i], a.n_new[s0 + i], v));
    big += (float)v[kTokens] + (float)v[kStreamLen] + (float)v[kTileLen];
#pragma unroll
    for (int x = 0; x < kSums; ++x) mine[x] += v[x];
  }
#pragma unroll 4
  for (int w = wa + lane; w < wb; w += 32) mine[kFreeBits] += __popc(pool_word(w0 + w));
  int32_t at[kSums];       // sums before this thread
#pragma unroll
  for (int i = 0; i < kSums; ++i) at[i] = mine[i];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
      const int32_t up = __shfl_up_sync(0xffffffffu, at[i], off);
      if (lane >= off) at[i] += up;
    }
    big += __shfl_xor_sync(0xffffffffu, big, off);
    err = min(err, __shfl_xor_sync(0xffffffffu, err, off));
  }
  if (lane == 31) {
#pragma unroll
    for (int i = 0; i < kSums; ++i) sh.warp_sum[i][warp] = at[i];
    sh.warp_big[warp] = big;
    sh.warp_err[warp] = err;
  }
  __syncthreads();
  if (warp < kSums) {
    // warp i scans sum i over the warps
    const int32_t w = sh.warp_sum[warp][lane];
    int32_t inc = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int32_t up = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += up;
    }
    sh.warp_sum[warp][lane] = inc - w;
    if (lane == 31) sh.sums[warp] = inc;
  } else if (warp == kSums) {
    float b = sh.warp_big[lane];
    int32_t e = sh.warp_err[lane];
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      b += __shfl_xor_sync(0xffffffffu, b, off);
      e = min(e, __shfl_xor_sync(0xffffffffu, e, off));
    }
    if (lane == 0) {
      sh.big = b;
      sh.err = e;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kFreeBits; ++i) at[i] += sh.warp_sum[i][warp] - mine[i];
  at[kFreeBits] = sh.warp_sum[kFreeBits][warp];   // before the warp

  // ---- the step's totals, and what the CTAs before this one hold ----
  int32_t total[kSums];
  if constexpr (C == 1) {
#pragma unroll
    for (int i = 0; i < kSums; ++i) total[i] = sh.sums[i];
    big = sh.big;
    err = sh.err;
  } else {
    cluster_sync();
    // lane r reads CTA r's; the warp adds them up
    const uint32_t r = lane & (C - 1);
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
      const int32_t x = (int32_t)remote_b32(&sh.sums[i], r);
      int32_t sum = x, before = r < rank ? x : 0;
#pragma unroll
      for (int off = C / 2; off; off >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, off);
        before += __shfl_xor_sync(0xffffffffu, before, off);
      }
      total[i] = sum;
      at[i] += before;
    }
    big = __uint_as_float(remote_b32(&sh.big, r));
    err = (int32_t)remote_b32(&sh.err, r);
#pragma unroll
    for (int off = C / 2; off; off >>= 1) {
      big += __shfl_xor_sync(0xffffffffu, big, off);
      err = min(err, __shfl_xor_sync(0xffffffffu, err, off));
    }
  }
  // (below kMaxLen the 32-bit sums are exact)
  if (err == 0 && (big >= kMaxLen || total[kTokens] > a.max_tokens)) err = kErrCapacity;
  if (err == 0 && total[kGrow] > total[kFreeBits]) err = kErrNoBlocks;
  const bool ok = err == 0;
  const int32_t T = ok ? total[kTokens] : 0, grow = ok ? total[kGrow] : 0;

  // ---- per sequence: offsets and work lists ----
  for (int i = sa; i < sb; ++i) {
    const int s = s0 + i;
    const int32_t seen = a.seen[s], n_new = a.n_new[s];
    if (!ok) {
      if (a.table != a.table_in) {
        int32_t held, need;
        blocks_of(seen, n_new, B, a.max_blocks, held, need);
        for (int c = held; c < need; ++c)
          a.table[(int64_t)s * a.max_blocks + c] = a.table_in[(int64_t)s * a.max_blocks + c];
      }
      a.ctx[s] = seen;
      a.q_start[s] = 0;
      continue;
    }
    int32_t v[kSums];
    measure(a, seen, n_new, v);
    a.ctx[s] = seen + n_new;
    a.q_start[s] = at[kTokens];
    StepRow of = {0, at[kGrow], {0, 0}};
    StepSeq e = {s, at[kTokens], n_new, seen + n_new, 0, 0, {0, 0}};
    if (v[kStreamed]) {
      of.unit = at[kStreamed];
      e.cum = at[kStreamLen];
      e.tiles = v[kStreamLen] - kStepStreamUnit;
      plan.streamed[of.unit] = e;
    } else if (v[kTiled]) {
      of.unit = -1 - at[kTiled];
      e.cum = at[kTileLen];
      e.tiles = v[kTileLen];
      plan.tiled[at[kTiled]] = e;
    }
    if (on_chip) {
      sh.q_start[i] = at[kTokens];
      sh.seen[i] = seen;
      sh.of[i] = of;
    } else {
      plan.of_seq[s] = of;
    }
#pragma unroll
    for (int x = 0; x < kFreeBits; ++x) at[x] += v[x];
    if (i == n_seqs - 1 && on_chip) sh.q_start[n_seqs] = at[kTokens];
  }
  if (rank == 0 && tid == 0) {
    a.q_start[S] = T;
    plan.header[kPlanRows] = T;
    plan.header[kPlanStreamed] = ok ? total[kStreamed] : 0;
    plan.header[kPlanTiled] = ok ? total[kTiled] : 0;
    plan.header[kPlanStreamLen] = ok ? total[kStreamLen] : 0;
    plan.header[kPlanTileLen] = ok ? total[kTileLen] : 0;
    plan.header[kPlanGroup] = a.group;
    plan.header[kPlanBlock] = B;
    plan.header[kPlanSeqs] = S;
    plan.header[kPlanTokens] = a.max_tokens;
    plan.header[kPlanMaxBlocks] = a.max_blocks;
    plan.header[kPlanPool] = a.num_blocks;
    plan.header[kPlanSerial] = serial + 1;
    if (!ok) atomicCAS(a.status, 0, err);
  }

  // ---- the lowest free ids, taken out of the bitmap ----
  const bool in_place = a.free_words == a.free_in;
  int32_t before = at[kFreeBits];
  for (int i = wa; i < wb; i += 32) {
    if (before >= grow && in_place) break;      // what is left stays as it is
    const int w = w0 + i + lane;
    const bool live = i + lane < wb;
    const uint32_t word = live ? (uint32_t)a.free_in[w] : 0u;
    uint32_t taken = 0;
    if (before < grow) {
      uint32_t rest = live ? pool_word(w) : 0u;
      int32_t inc = __popc(rest), n = inc;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int32_t up = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += up;
      }
      for (int32_t k = before + inc - n; rest && k < grow; ++k) {
        const uint32_t low = rest & (0u - rest);
        rest ^= low;
        taken |= low;
        plan.new_ids[k] = w * 32 + 31 - __clz(low);
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (live && (taken || !in_place)) a.free_words[w] = (int32_t)(word & ~taken);
  }

  // ---- rows past the step's ----
  for (int64_t r = T + (int64_t)rank * kThreads + tid; r < a.max_tokens;
       r += (int64_t)C * kThreads) {
    a.position[r] = -1;
    a.slot[r] = -1;
  }
  if constexpr (C == 1) __syncthreads();
  else cluster_sync();
  if (!ok || n_seqs <= 0) return;

  // ---- the rows of this CTA's sequences: positions, slots, and the entry of
  // each block that begins ----
  const int32_t* q_start = on_chip ? sh.q_start : a.q_start + s0;
  const int r1 = q_start[n_seqs];
  for (int r = q_start[0] + tid; r < r1; r += kThreads) {
    // the first sequence that ends behind row r
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (q_start[mid + 1] > r) hi = mid;
      else lo = mid + 1;
    }
    const int s = s0 + lo, q0 = q_start[lo];
    const int seen = on_chip ? sh.seen[lo] : a.ctx[s] - (q_start[lo + 1] - q0);
    StepRow of = on_chip ? sh.of[lo] : plan.of_seq[s];
    const int pos = seen + r - q0;
    const int held = (int)(((uint32_t)seen + B - 1) / (uint32_t)B);
    const int c = (int)((uint32_t)pos / (uint32_t)B), off = pos - c * B;
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
// the sequences does not matter).  Latency: 16 sequences 1.8 us in a graph, 512 of
// up to 8192 tokens 3.5.
__global__ void __launch_bounds__(256)
    release_kernel(BuildArgs a, const int32_t* __restrict__ done) {
  const int s = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5), lane = threadIdx.x & 31;
  const int32_t* h = a.plan;
  if (h[kPlanBlock] != 0 &&      // (0: no step has been built yet)
      (h[kPlanBlock] != a.block_size || h[kPlanSeqs] != a.num_seqs ||
       h[kPlanMaxBlocks] != a.max_blocks || h[kPlanPool] != a.num_blocks)) {
    if (threadIdx.x == 0) atomicCAS(a.status, 0, kErrInvalid);
    return;
  }
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
  const bool one = a.num_seqs <= kOneSeqs && a.num_blocks <= kOneBlocks &&
                   a.max_tokens <= kOneRows;
  const int ctas = one ? 1 : kCluster;
  int copies = 0;
  if (a.table != a.table_in) {
    copies = std::min((a.num_seqs + kWarps - 1) / kWarps, std::max(1, sms));
    copies = (copies + ctas - 1) / ctas * ctas;
  }
  auto fn = one ? build_kernel<1> : build_kernel<kCluster>;
  // the shared-memory limit is raised once per device
  static std::atomic<uint64_t> attr_done{0};
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load() & bit)) {
    e = cudaFuncSetAttribute(build_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(Shared));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(build_kernel<kCluster>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas + copies));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = one ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, fn, a);
}

cudaError_t launch_step_release(const BuildArgs& a, const int32_t* done, cudaStream_t st) {
  release_kernel<<<(unsigned)((a.num_seqs + 7) / 8), 256, 0, st>>>(a, done);
  return cudaGetLastError();
}

}  // namespace rbkv
