// The append with a rotary position embedding on the way: rotated queries to
// q_out, rotated keys and the values to their cache slots, in one pass over
// the new rows.
//
// Pair i of a head's first R elements, (x, y) = elements (i, i + R/2) or
// (2 i, 2 i + 1), is turned by the angle a = 2 pi p f_i of its row's position p:
//   x' = (x cos a - y sin a) scale,   y' = (y cos a + x sin a) scale.
// f_i comes as a fraction of a turn in units of 2^-64, so p f_i modulo one turn
// is one 64-bit product that wraps around: exact at any position, with no 64-bit
// floating-point arithmetic (which this GPU has little of).  Its upper bits, as
// fp32 in half turns, go to sincospif: each off by at most 2^-24 of a half turn
// before it.
//
// A block takes a row: a thread each works out one pair's sine and cosine into
// shared memory, for all heads, while its first vectors are on their way; then
// every thread rotates units of two 16-byte vectors that hold both elements of
// their pairs (so that q_out may be q).  Values and the elements behind R are
// units that are only copied.  Where R / 2 elements are not whole vectors a unit
// is one pair (kVec = 1).
#include <algorithm>
#include <cstring>
#include <string>

#include "rbkv_internal.h"
#include "rbkv_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace rbkv {

namespace {

constexpr int kThreads = 128;       // at least the pairs of a head: 256 / 2
constexpr int kUnroll = 4;          // units of a thread in flight

// kVec elements as one word, and as fp32.
template <class T, int kVec> struct Pack;
template <> struct Pack<__nv_bfloat16, 8> {
  using Raw = uint4;
  static __device__ __forceinline__ void open(const Raw& r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ Raw close(const float* x) {
    return make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]),
                      ptx::pack_bf16x2(x[4], x[5]), ptx::pack_bf16x2(x[6], x[7]));
  }
};
template <> struct Pack<float, 4> {
  using Raw = uint4;
  static __device__ __forceinline__ void open(const Raw& r, float* x) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ Raw close(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <> struct Pack<__nv_bfloat16, 1> {
  using Raw = uint16_t;
  static __device__ __forceinline__ void open(const Raw& r, float* x) {
    x[0] = __uint_as_float((uint32_t)r << 16);
  }
  static __device__ __forceinline__ Raw close(const float* x) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
  }
};
template <> struct Pack<float, 1> {
  using Raw = uint32_t;
  static __device__ __forceinline__ void open(const Raw& r, float* x) {
    x[0] = __uint_as_float(r);
  }
  static __device__ __forceinline__ Raw close(const float* x) { return __float_as_uint(x[0]); }
};

struct Heads {
  int32_t q, kv, dim, block;
  uint32_t per, inverse;       // units per head, and ceil(2^32 / per)
  int32_t rotating;            // of which hold pairs
};

template <class T, int kVec>
__global__ void __launch_bounds__(kThreads)
    append_rotary_kernel(DevPass dp, Heads h, rbkv_rotary r, int32_t offset, const void* q,
                         void* q_out, const void* __restrict__ k_new,
                         const void* __restrict__ v_new, void* __restrict__ k_cache,
                         void* __restrict__ v_cache) {
  using P = Pack<T, kVec>;
  using Raw = typename P::Raw;
  __shared__ __align__(16) float cos_s[kThreads], sin_s[kThreads];
  // Launched to overlap its predecessor's tail: wait for it (it may have
  // produced the inputs, or still read cache blocks that are written here).
  ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  const int rows = pass_count(dp, kCountTokens, dp.num_tokens);
  const int tid = threadIdx.x;
  if (dp.built_for[0] &&
      (*dp.built_for[0] != h.block || *dp.built_for[1] != dp.num_tokens ||
       (dp.built_for[2] && *dp.built_for[2] != *dp.built_for[3]))) {
    if (tid == 0 && rows > 0) atomicCAS(dp.status, 0, kDevInvalid);
    return;
  }
  const uint32_t units_q = (uint32_t)h.q * h.per, units_k = (uint32_t)h.kv * h.per;
  const uint32_t units = units_q + 2 * units_k;
  const int half = r.rotary_dim / 2;
  // a unit: its head's tensor (0 q, 1 k, 2 v), head, and its two vectors' places
  struct Unit {
    int kind, head, col, e0, e1;
  };
  auto locate = [&](uint32_t u) {
    Unit x;
    x.kind = u < units_q ? 0 : u < units_q + units_k ? 1 : 2;
    u -= x.kind == 0 ? 0 : x.kind == 1 ? units_q : units_q + units_k;
    x.head = h.per == 1 ? u : __umulhi(u, h.inverse);
    x.col = (int)(u - (uint32_t)x.head * h.per);
    const bool apart = x.kind != 2 && x.col < h.rotating && !r.interleaved;
    x.e0 = (apart ? 1 : 2) * x.col * kVec;
    x.e1 = x.e0 + (apart ? half : kVec);
    return x;
  };
  for (int row = blockIdx.x; row < rows; row += gridDim.x) {
    for (uint32_t u0 = tid; u0 - tid < units; u0 += kUnroll * kThreads) {
      Raw a[kUnroll], b[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const uint32_t u = u0 + i * kThreads;
        if (u >= units) continue;
        const Unit x = locate(u);
        const void* src = x.kind == 0 ? q : x.kind == 1 ? k_new : v_new;
        const T* p = (const T*)src +
                     ((int64_t)row * (x.kind == 0 ? h.q : h.kv) + x.head) * h.dim;
        a[i] = *reinterpret_cast<const Raw*>(p + x.e0);
        b[i] = *reinterpret_cast<const Raw*>(p + x.e1);
      }
      const int slot = dp.slot[row];
      if (u0 == (uint32_t)tid) {
        const uint32_t at = (uint32_t)(dp.position[row] + offset);
        __syncthreads();      // (the previous row's are no longer needed)
        if (tid < half) {
          float s, c;
          sincospif((float)(int64_t)(r.turns[tid] * at) * 0x1p-63f, &s, &c);
          cos_s[tid] = c * r.scale;
          sin_s[tid] = s * r.scale;
        }
        __syncthreads();
      }
      const int blk = slot / h.block, in_block = slot - blk * h.block;
      const bool inside = slot >= 0 && blk < dp.num_blocks;
      if (!inside && tid == 0) atomicCAS(dp.status, 0, kDevBounds);
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const uint32_t u = u0 + i * kThreads;
        if (u >= units) continue;
        const Unit x = locate(u);
        if (x.kind != 2 && x.col < h.rotating) {
          float m[2 * kVec], c[kVec], s[kVec];
          P::open(a[i], m);
          P::open(b[i], m + kVec);
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            c[e] = cos_s[x.col * kVec + e];
            s[e] = sin_s[x.col * kVec + e];
          }
          if (r.interleaved) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
              const float v = m[2 * e], w = m[2 * e + 1];
              m[2 * e] = v * c[e] - w * s[e];
              m[2 * e + 1] = w * c[e] + v * s[e];
            }
          } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
              const float v = m[e], w = m[kVec + e];
              m[e] = v * c[e] - w * s[e];
              m[kVec + e] = w * c[e] + v * s[e];
            }
          }
          a[i] = P::close(m);
          b[i] = P::close(m + kVec);
        }
        T* to;
        if (x.kind == 0) {
          to = (T*)q_out + ((int64_t)row * h.q + x.head) * h.dim;
        } else {
          if (!inside) continue;
          to = (T*)(x.kind == 1 ? k_cache : v_cache) +
               (((int64_t)blk * h.kv + x.head) * h.block + in_block) * h.dim;
        }
        *reinterpret_cast<Raw*>(to + x.e0) = a[i];
        *reinterpret_cast<Raw*>(to + x.e1) = b[i];
      }
    }
  }
}

template <class T, int kVec>
cudaError_t launch(const DevPass& dp, const ShapeInfo& s, const rbkv_rotary& r, int32_t offset,
                   const void* q, void* q_out, const void* k_new, const void* v_new,
                   void* k_cache, void* v_cache, cudaStream_t st, bool overlap_previous) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  Heads h;
  h.q = s.H_q;
  h.kv = s.H_kv;
  h.dim = s.D;
  h.block = s.B;
  h.per = (uint32_t)(s.D / (2 * kVec));
  // (u / per = umulhi(u, inverse) for the units of a tensor's row: u per < 2^32)
  h.inverse = (uint32_t)((((uint64_t)1 << 32) + h.per - 1) / h.per);
  h.rotating = r.rotary_dim / (2 * kVec);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(dp.num_tokens, std::max(1, sms) * 16));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = overlap_previous ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, append_rotary_kernel<T, kVec>, dp, h, r, offset, q, q_out,
                            k_new, v_new, k_cache, v_cache);
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

}  // namespace

rbkv_status check_append_rotary(const rbkv_config* c, const rbkv_rotary* r, int64_t rows,
                                const void* q, const void* q_out, const void* k_new,
                                const void* v_new, const void* k_cache, const void* v_cache) {
  auto invalid = [](const char* msg) { return set_error(RBKV_ERR_INVALID, msg); };
  if (!r || !r->turns) return invalid("rotary or its turns is NULL");
  if ((uintptr_t)r->turns % 8) return invalid("turns must be 8-byte aligned");
  if (r->rotary_dim < 2 || r->rotary_dim > c->head_dim || r->rotary_dim % 2)
    return invalid("rotary_dim must be even, in [2, head_dim]");
  if (r->interleaved != 0 && r->interleaved != 1) return invalid("interleaved must be 0 or 1");
  const void* all[] = {q, q_out, k_new, v_new, k_cache, v_cache};
  for (const void* p : all) {
    if (!p) return invalid("NULL tensor");
    if ((uintptr_t)p % 16) return invalid("tensors must be 16-byte aligned");
  }
  if ((int64_t)c->num_heads_q * c->head_dim >= (int64_t)1 << 24)
    return set_error(RBKV_ERR_UNSUPPORTED, "too many heads for one rotary append");
  const int64_t size = c->dtype == RBKV_BF16 ? 2 : 4;
  const int64_t q_bytes = rows * c->num_heads_q * c->head_dim * size;
  const int64_t kv_bytes = rows * c->num_heads_kv * c->head_dim * size;
  const int64_t cache =
      (int64_t)c->num_blocks * c->block_size * c->num_heads_kv * c->head_dim * size;
  if (q != q_out && overlap(q, q_bytes, q_out, q_bytes))
    return invalid("q_out overlaps q in part");
  if (overlap(q_out, q_bytes, k_new, kv_bytes) || overlap(q_out, q_bytes, v_new, kv_bytes) ||
      overlap(q_out, q_bytes, k_cache, cache) || overlap(q_out, q_bytes, v_cache, cache) ||
      overlap(q_out, q_bytes, r->turns, 4 * (int64_t)r->rotary_dim))
    return invalid("q_out overlaps another tensor");
  return RBKV_OK;
}

cudaError_t launch_append_rotary(const DevPass& dp, const ShapeInfo& s, const rbkv_rotary& r,
                                 int32_t offset, const void* q, void* q_out, const void* k_new,
                                 const void* v_new, void* k_cache, void* v_cache, cudaStream_t st,
                                 bool overlap_previous) {
  if (dp.num_tokens == 0) return cudaSuccess;
  // both vectors of a unit lie among the rotated elements, or both behind them
  const bool vectors = r.rotary_dim % (s.dtype == 0 ? 16 : 8) == 0;
  auto fn = s.dtype == 0 ? (vectors ? launch<__nv_bfloat16, 8> : launch<__nv_bfloat16, 1>)
                         : (vectors ? launch<float, 4> : launch<float, 1>);
  return fn(dp, s, r, offset, q, q_out, k_new, v_new, k_cache, v_cache, st, overlap_previous);
}

}  // namespace rbkv
