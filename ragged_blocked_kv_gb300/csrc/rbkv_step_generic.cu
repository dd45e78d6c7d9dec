// Attention of a step on the CUDA cores: every type, head dim and block size.
//
// Row t of sequence s, query head h: softmax over the prefix's keys
// 0 .. prefix_len - 1 and the sequence's own keys 0 .. position[t].  One warp
// per (row, head) walks the keys 32 at a time, one per lane, with a running
// maximum and sum; the value rows are then added with the lanes spread over
// the head dim.
#include "rbkv_step.h"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace rbkv {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxDPerLane = 8;   // head_dim <= 256
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

template <class T>
__global__ void __launch_bounds__(kWarps * 32)
    step_generic_kernel(DevStep ds, ShapeInfo s, const T* __restrict__ q,
                        const T* __restrict__ k_cache, const T* __restrict__ v_cache,
                        T* __restrict__ o) {
  __shared__ float q_s[kWarps][256];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const StepPlan plan = step_plan(ds.plan, ds.num_seqs, ds.max_tokens);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int D = s.D, B = s.B, H_kv = s.H_kv, dpl = D / 32;
  const int64_t items = (int64_t)plan.header[kPlanRows] * s.H_q;
  for (int64_t w = (int64_t)blockIdx.x * kWarps + warp; w < items;
       w += (int64_t)gridDim.x * kWarps) {
    const int t = (int)(w / s.H_q), h = (int)(w % s.H_q), kvh = h / s.g;
    const StepRow r = plan.rows[t];
    const StepSeq e = r.unit >= 0 ? plan.streamed[r.unit] : plan.tiled[-1 - r.unit];
    const int seq = e.seq, own = e.ctx - e.n_new + r.token + 1;   // keys the row sees
    const int32_t* table = ds.block_table + (int64_t)seq * ds.max_blocks;
    const T* qrow = q + ((int64_t)t * s.H_q + h) * D;
    for (int d = lane; d < D; d += 32) q_s[warp][d] = to_f(qrow[d]) * (s.scale * kLog2e);
    __syncwarp();
    float m = -INFINITY, l = 0.f;
    float acc[kMaxDPerLane];
#pragma unroll
    for (int i = 0; i < kMaxDPerLane; ++i) acc[i] = 0.f;
    for (int part = 0; part < 2; ++part) {
      const int n = part ? own : ds.prefix_len;
      const int32_t* ids = part ? table : ds.prefix_table;
      for (int k0 = 0; k0 < n; k0 += 32) {
        const int key = k0 + lane;
        float sc = -INFINITY;
        int64_t row_off = -1;
        if (key < n) {
          const int32_t blk = ids[key / B];
          if (blk >= 0 && blk < ds.num_blocks) {
            row_off = (((int64_t)blk * H_kv + kvh) * B + key % B) * D;
            const T* krow = k_cache + row_off;
            float dot = 0.f;
            for (int d = 0; d < D; ++d) dot = fmaf(q_s[warp][d], to_f(krow[d]), dot);
            sc = dot;
          } else {
            atomicCAS(ds.status, 0, kDevBounds);
          }
        }
        float top = sc;
#pragma unroll
        for (int off = 16; off; off >>= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float m_new = fmaxf(m, top);
        if (m_new == -INFINITY) continue;   // every key so far skipped
        const float corr = exp2f(m - m_new);
        const float p = exp2f(sc - m_new);
        float sum = p;
#pragma unroll
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l = l * corr + sum;
#pragma unroll
        for (int i = 0; i < kMaxDPerLane; ++i) acc[i] *= corr;
        for (int j = 0; j < 32; ++j) {
          const float pj = __shfl_sync(0xffffffffu, p, j);
          const int64_t roff = __shfl_sync(0xffffffffu, row_off, j);
          if (roff < 0) continue;
          const T* vrow = v_cache + roff;
#pragma unroll
          for (int i = 0; i < kMaxDPerLane; ++i)
            if (i < dpl) acc[i] = fmaf(pj, to_f(vrow[lane + 32 * i]), acc[i]);
        }
        m = m_new;
      }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    T* orow = o + ((int64_t)t * s.H_q + h) * D;
#pragma unroll
    for (int i = 0; i < kMaxDPerLane; ++i)
      if (i < dpl) orow[lane + 32 * i] = from_f<T>(acc[i] * inv);
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_step_generic(const DevStep& ds, const ShapeInfo& s, const void* q,
                                const void* k_cache, const void* v_cache, void* o,
                                cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t warps = (int64_t)ds.max_tokens * s.H_q;
  int64_t blocks = (warps + kWarps - 1) / kWarps;
  if (blocks > (int64_t)sms * 16) blocks = (int64_t)sms * 16;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (s.dtype == 0)
    return cudaLaunchKernelEx(&cfg, step_generic_kernel<__nv_bfloat16>, ds, s,
                              (const __nv_bfloat16*)q, (const __nv_bfloat16*)k_cache,
                              (const __nv_bfloat16*)v_cache, (__nv_bfloat16*)o);
  return cudaLaunchKernelEx(&cfg, step_generic_kernel<float>, ds, s, (const float*)q,
                            (const float*)k_cache, (const float*)v_cache, (float*)o);
}

}  // namespace rbkv
