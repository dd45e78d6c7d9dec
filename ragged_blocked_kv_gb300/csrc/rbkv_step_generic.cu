// Attention of a step on the CUDA cores: every type, head dim and block size
// (fp32 steps, and bf16 shapes off the tensor-core kernels).
//
// A block takes eight packed rows (row = token * g + head) of one KV head, or
// four.  Over the prefix all of them see the same keys; behind it each token sees its
// own sequence's.  Keys go 32 at a time, one per lane, so that one read of a
// key row serves all rows (its dot products take q from shared memory as
// broadcasts); the weights pass through shared memory to the value product,
// where the lanes hold the head dim and one read of a value row serves all
// rows.  The 32-key chunks of both parts are dealt to the block's eight warps
// (and, where there are few rows, to `splits` blocks); each warp keeps an
// online softmax per row, and the warps are joined by their maxima and sums
// in shared memory.  All arithmetic is fp32 FMAs.  Bound by the shared-memory
// reads of q and the weights, and by latency at the sizes it is used for: 69
// rows of 8 heads, dim 64, fp32, behind 333 keys and up to 100 own ones take
// 18.9 us (eight rows of a block everywhere: 20.9).
#include <algorithm>
#include <atomic>

#include "rbkv_step.h"
#include "rbkv_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace rbkv {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;

template <class T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <class T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Four consecutive elements.
__device__ __forceinline__ float4 load4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u),
                     __uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Shared memory: q [rows][D], each warp's weights [32 keys][rows], and for
// the join O [warp][row][D] and (max, sum) [warp][row].
__host__ __device__ constexpr int smem_floats(int D, int rows) {
  return rows * D + kWarps * 32 * rows + kWarps * rows * D + kWarps * rows * 2;
}

// kPer: head-dim elements per lane, D = 32 dpl with dpl <= kPer.  kRows: packed
// rows of a block, 4 or 8.
template <class T, int kPer, int kRows>
__global__ void __launch_bounds__(kThreads)
    step_generic_kernel(DevStep ds, ShapeInfo s, const T* __restrict__ q,
                        const T* __restrict__ k_cache, const T* __restrict__ v_cache,
                        T* __restrict__ o, float* __restrict__ part_o,
                        float* __restrict__ part_lse, int splits) {
  extern __shared__ __align__(16) float smem[];
  ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  const StepPlan plan = step_plan(ds.plan, ds.num_seqs, ds.max_tokens);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int D = s.D, B = s.B, H_kv = s.H_kv, g = s.g, dpl = D / 32;
  float* q_s = smem;
  float* p_s = smem + kRows * D + warp * 32 * kRows;
  float* join_o = smem + kRows * D + kWarps * 32 * kRows;
  float* join_ml = join_o + kWarps * kRows * D;
  const int T_rows = step_rows(ds, s, plan);
  const int n_rows = T_rows * g;               // packed rows of a KV head
  const int kvh = blockIdx.y, split = blockIdx.z;
  const int stride = kWarps * splits, mine = split * kWarps + warp;

  for (int row0 = blockIdx.x * kRows; row0 < n_rows; row0 += gridDim.x * kRows) {
    const int rows = min(kRows, n_rows - row0);
    for (int e = threadIdx.x; e < kRows * D; e += kThreads) {
      const int r = e / D, d = e - r * D, t = (row0 + r) / g, h = kvh * g + (row0 + r) % g;
      q_s[e] = r < rows ? to_f(q[((int64_t)t * s.H_q + h) * D + d]) * (s.scale * kLog2e) : 0.f;
    }
    __syncthreads();
    float m[kRows], l[kRows], acc[kRows][kPer];
    int tok[kRows];        // the rows' tokens (rows of the step)
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      tok[r] = (row0 + r) / g;
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[r][i] = 0.f;
    }

    // One 32-key chunk for the rows [ra, rb) of the block; row r sees the keys
    // below lim0 + (token of r - tok0), or all n.
    auto chunk = [&](const int32_t* ids, int k0, int n, int ra, int rb, int lim0, int tok0,
                     bool causal) {
      const int key = k0 + lane;
      int64_t off = -1;
      if (key < n) {
        const int blk = ids[key / B];
        if ((uint32_t)blk < (uint32_t)ds.num_blocks)
          off = (((int64_t)blk * H_kv + kvh) * B + key % B) * D;
        else
          atomicCAS(ds.status, 0, kDevBounds);
      }
      float x[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) x[r] = 0.f;
      // (all of a 32-element piece of the key row requested before any of it is used)
      const T* kr = k_cache + max((int64_t)0, off);
      for (int d0 = 0; d0 < D; d0 += 32) {
        float4 k[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) k[u] = load4(kr + d0 + 4 * u);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            const float4 a = *reinterpret_cast<const float4*>(q_s + r * D + d0 + 4 * u);
            x[r] = fmaf(a.x, k[u].x, fmaf(a.y, k[u].y, fmaf(a.z, k[u].z, fmaf(a.w, k[u].w, x[r]))));
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        // (other sequences' rows see none of these keys: their terms are 0)
        const int lim = r < ra || r >= rb ? 0 : causal ? lim0 + tok[r] - tok0 : n;
        const bool sees = off >= 0 && key < lim;
        const float sc = sees ? x[r] : -INFINITY;
        const float mn = fmaxf(m[r], warp_max(sc));
        // a row with no visible key so far keeps max -inf: its terms are 0
        const float base = mn == -INFINITY ? 0.f : mn;
        const float corr = ptx::ex2(m[r] - base), p = ptx::ex2(sc - base);
        m[r] = mn;
        l[r] = fmaf(l[r], corr, p);       // this lane's keys; summed at the end
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[r][i] *= corr;
        p_s[lane * kRows + r] = sees ? p : -1.f;
      }
      __syncwarp();
      // several value rows in flight: their latency is what a chunk waits for
      const int count = min(32, n - k0);
      constexpr int kAhead = 16 / kPer;
      for (int j0 = 0; j0 < count; j0 += kAhead) {
        float v[kAhead][kPer];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          // (a key that no row sees is left out below: any row may stand in)
          const int64_t at = max((int64_t)0, __shfl_sync(0xffffffffu, off, j0 + u));
          const T* vr = v_cache + at + lane;
#pragma unroll
          for (int i = 0; i < kPer; ++i) v[u][i] = to_f(vr[32 * min(i, dpl - 1)]);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          float w[kRows];
#pragma unroll
          for (int r = 0; r < kRows; r += 4)
            *reinterpret_cast<float4*>(w + r) =
                *reinterpret_cast<const float4*>(p_s + (j0 + u) * kRows + r);
          // (a weight of -1 leaves the sum alone: the row does not see the key, whose
          // value may be another sequence's or a later token's, finite or not; one
          // that underflowed to 0 does not: a value that is not finite reaches
          // every row that sees it)
#pragma unroll
          for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int i = 0; i < kPer; ++i)
              acc[r][i] = w[r] < 0.f ? acc[r][i] : fmaf(w[r], v[u][i], acc[r][i]);
        }
      }
      __syncwarp();
    };

    int c = 0;      // chunks dealt so far
    for (int k0 = 0; k0 < ds.prefix_len; k0 += 32, ++c)
      if (c % stride == mine) chunk(ds.prefix_table, k0, ds.prefix_len, 0, rows, 0, 0, false);
    for (int ra = 0; ra < rows;) {
      // the rows of one sequence: row0 + ra .. row0 + rb - 1
      const int t = (row0 + ra) / g;
      const StepRow info = plan.rows[t];
      const StepSeq e = info.unit >= 0 ? plan.streamed[info.unit] : plan.tiled[-1 - info.unit];
      const int rb = min(rows, (e.row + e.n_new) * g - row0);
      const int lim0 = e.ctx - e.n_new + info.token + 1;      // keys that token t sees
      const int n = lim0 + (row0 + rb - 1) / g - t;           // and the last one
      const int32_t* table = ds.block_table + (int64_t)e.seq * ds.max_blocks;
      for (int k0 = 0; k0 < n; k0 += 32, ++c)
        if (c % stride == mine) chunk(table, k0, n, ra, rb, lim0, t, true);
      ra = rb;
    }

    // ---- join the warps ----
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
      for (int f = 16; f; f >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], f);
      if (lane == 0) {
        join_ml[(warp * kRows + r) * 2] = m[r];
        join_ml[(warp * kRows + r) * 2 + 1] = l[r];
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < dpl) join_o[(warp * kRows + r) * D + lane + 32 * i] = acc[r][i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < rows * D; e += kThreads) {
      const int r = e / D, d = e - r * D;
      float M = -INFINITY, L = 0.f, a = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, join_ml[(w * kRows + r) * 2]);
      const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(join_ml[(w * kRows + r) * 2] - base);
        L = fmaf(f, join_ml[(w * kRows + r) * 2 + 1], L);
        a = fmaf(f, join_o[(w * kRows + r) * D + d], a);
      }
      const float inv = L > 0.f ? 1.f / L : 0.f;
      const int64_t at = (int64_t)((row0 + r) / g) * s.H_q + kvh * g + (row0 + r) % g;
      if (splits == 1) {
        o[at * D + d] = from_f<T>(a * inv);
      } else {
        const int64_t to = (int64_t)split * ds.max_tokens * s.H_q + at;
        part_o[to * D + d] = a * inv;
        if (d == 0) part_lse[to] = L > 0.f ? M + log2f(L) : -INFINITY;
      }
    }
    __syncthreads();
  }
}

// O of the splits of a step: one warp per (row, query head).
template <class T>
__global__ void __launch_bounds__(128)
    step_generic_join_kernel(DevStep ds, ShapeInfo s, const float* __restrict__ part_o,
                             const float* __restrict__ part_lse, T* __restrict__ o, int splits) {
  ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  const StepPlan plan = step_plan(ds.plan, ds.num_seqs, ds.max_tokens);
  const int lane = threadIdx.x & 31, D = s.D;
  const int64_t rows = (int64_t)step_rows(ds, s, plan) * s.H_q;
  const int64_t all = (int64_t)ds.max_tokens * s.H_q;
  for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); w < rows;
       w += (int64_t)gridDim.x * 4) {
    const float mine = lane < splits ? part_lse[lane * all + w] : -INFINITY;
    float M = mine;
#pragma unroll
    for (int f = 16; f; f >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, f));
    float f = mine == -INFINITY ? 0.f : exp2f(mine - M);
    float sum = f;
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    f = sum > 0.f ? f / sum : 0.f;
    for (int d = lane; d < D; d += 32) {
      float a = 0.f;
#pragma unroll 4
      for (int i = 0; i < splits; ++i) {
        const float wt = __shfl_sync(0xffffffffu, f, i);
        a = fmaf(wt, part_o[(i * all + w) * D + d], a);
      }
      o[w * D + d] = from_f<T>(a);
    }
  }
}

}  // namespace

namespace {
// Packed rows of a block: four where eight would leave SMs without one (74
// blocks of eight rows, fp32: 20.9 us; 148 of four: half the dot products per
// key and twice the blocks).
int rows_of(const ShapeInfo& s, int32_t max_tokens, int sms) {
  return ((int64_t)max_tokens * s.g + 7) / 8 * s.H_kv < sms ? 4 : 8;
}
}  // namespace

// Blocks that share a block of rows: as many as bring the grid near two blocks
// per SM, at most one per 256 keys of the prefix or of the longest sequence
// the tables hold (a split costs a second launch).  One row of 8 heads, dim 64,
// behind 2000 keys: 23.6 us with splits, 50.3 without; 32 rows 36.8 and 57.3;
// behind 333 keys the rule gives none.
int step_generic_splits(const ShapeInfo& s, int32_t max_tokens, int32_t max_blocks,
                        int32_t prefix_len, int sms) {
  const int rows = rows_of(s, max_tokens, sms);
  const int64_t units = ((int64_t)max_tokens * s.g + rows - 1) / rows * s.H_kv;
  const int64_t keys = (int64_t)prefix_len + (int64_t)max_blocks * s.B;
  const int64_t n = std::min<int64_t>(2 * (int64_t)sms / units, keys / 256);
  return (int)std::max<int64_t>(1, std::min<int64_t>(n, kStepGenericSplits));
}

size_t step_generic_workspace(const ShapeInfo& s, int32_t max_tokens, int splits) {
  if (splits == 1) return 0;
  return (size_t)splits * max_tokens * s.H_q * (s.D + 1) * 4;
}

namespace {

template <class T, int kPer, int kRows>
cudaError_t launch_rows(const DevStep& ds, const ShapeInfo& s, const void* q, const void* k_cache,
                        const void* v_cache, void* o, float* part_o, float* part_lse, int splits,
                        int sms, cudaStream_t st) {
  const int bytes = smem_floats(s.D, kRows) * 4;
  // the shared-memory limit is raised once per device
  static std::atomic<uint64_t> attr_done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_done.load() & bit)) {
    e = cudaFuncSetAttribute(step_generic_kernel<T, kPer, kRows>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem_floats(kPer * 32, kRows) * 4);
    if (e != cudaSuccess) return e;
    attr_done.fetch_or(bit);
  }
  const int64_t tiles = ((int64_t)ds.max_tokens * s.g + kRows - 1) / kRows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(tiles, (int64_t)sms * 16), (unsigned)s.H_kv,
                     (unsigned)splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, step_generic_kernel<T, kPer, kRows>, ds, s, (const T*)q,
                         (const T*)k_cache, (const T*)v_cache, (T*)o, part_o, part_lse, splits);
  if (e != cudaSuccess || splits == 1) return e;
  const int64_t warps = (int64_t)ds.max_tokens * s.H_q;
  cfg.gridDim = dim3((unsigned)std::min<int64_t>((warps + 3) / 4, (int64_t)sms * 16));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, step_generic_join_kernel<T>, ds, s, (const float*)part_o,
                            (const float*)part_lse, (T*)o, splits);
}

template <class T>
cudaError_t launch_type(const DevStep& ds, const ShapeInfo& s, const void* q, const void* k_cache,
                        const void* v_cache, void* o, float* po, float* pl, int splits, int sms,
                        cudaStream_t st) {
  const bool few = rows_of(s, ds.max_tokens, sms) == 4;
  auto fn = s.D <= 64    ? (few ? launch_rows<T, 2, 4> : launch_rows<T, 2, 8>)
            : s.D <= 128 ? (few ? launch_rows<T, 4, 4> : launch_rows<T, 4, 8>)
                         : (few ? launch_rows<T, 8, 4> : launch_rows<T, 8, 8>);
  return fn(ds, s, q, k_cache, v_cache, o, po, pl, splits, sms, st);
}

}  // namespace

cudaError_t launch_step_generic(const DevStep& ds, const ShapeInfo& s, const void* q,
                                const void* k_cache, const void* v_cache, void* o,
                                void* workspace, int splits, int sms, cudaStream_t st) {
  float* po = (float*)workspace;
  float* pl = po ? po + (size_t)splits * ds.max_tokens * s.H_q * s.D : nullptr;
  if (s.dtype == 0)
    return launch_type<__nv_bfloat16>(ds, s, q, k_cache, v_cache, o, po, pl, splits, sms, st);
  return launch_type<float>(ds, s, q, k_cache, v_cache, o, po, pl, splits, sms, st);
}

}  // namespace rbkv
