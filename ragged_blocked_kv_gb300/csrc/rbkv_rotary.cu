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
// shared memory, for all heads, while its first vectors are on their way.  A unit
// is two 16-byte vectors that hold both elements of their pairs (so that q_out may
// be q); a thread has the same units' column in every few heads, and so keeps its
// pairs' turns in registers.  Values and the elements behind R are only copied.
// Where R / 2 elements are not whole vectors the words are narrower, down to one
// element (kVec = 1).
//
// Bound by memory and, in few rows, by the call: 2048 rows of 32 and 8 heads of
// 128, bf16, 50 MB, 10.6 us (4.8 TB/s with the launch; the copy alone would take
// 7.4), 16 rows 6.9 (the host's time).  With the turns read from shared memory for
// every unit 12.4 us, all of a unit's elements as fp32 at once 11.8, four units in
// flight instead of three (48 heads are three to a thread) 12.8, two 12.2.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>

#include "rbkv_internal.h"
#include "rbkv_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace rbkv {

namespace {

constexpr int kThreads = 128;       // at least the pairs of a head: 256 / 2
constexpr int kUnroll = 3;          // units of a thread in flight

// (x, y) turned by an angle of cosine t.x and sine t.y.
__device__ __forceinline__ void turn(float& x, float& y, const float2& t) {
  const float u = x * t.x - y * t.y;
  y = y * t.x + x * t.y;
  x = u;
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A unit: two words of kVec elements, whose pairs lie across the words ("half") or
// side by side in them, and the turns of its kVec pairs.  (A few elements at a time:
// all of a unit's as fp32 at once took registers that the loads in flight need.)
template <class T, int kVec> struct Unit;
template <> struct Unit<__nv_bfloat16, 8> {
  using Word = uint4;
  static __device__ __forceinline__ void rotate(uint4& a, uint4& b, const float2* t, bool beside) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (beside) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x = low(w[i]), y = high(w[i]);
        turn(x, y, t[i]);
        w[i] = ptx::pack_bf16x2(x, y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x0 = low(w[i]), x1 = high(w[i]), y0 = low(w[4 + i]), y1 = high(w[4 + i]);
        turn(x0, y0, t[2 * i]);
        turn(x1, y1, t[2 * i + 1]);
        w[i] = ptx::pack_bf16x2(x0, x1);
        w[4 + i] = ptx::pack_bf16x2(y0, y1);
      }
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
  }
};
template <> struct Unit<float, 4> {
  using Word = float4;
  static __device__ __forceinline__ void rotate(float4& a, float4& b, const float2* t,
                                                bool beside) {
    turn(a.x, beside ? a.y : b.x, t[0]);
    turn(beside ? a.z : a.y, beside ? a.w : b.y, t[1]);
    turn(beside ? b.x : a.z, beside ? b.y : b.z, t[2]);
    turn(beside ? b.z : a.w, b.w, t[3]);
  }
};
template <> struct Unit<__nv_bfloat16, 2> {
  using Word = uint32_t;
  static __device__ __forceinline__ void rotate(uint32_t& a, uint32_t& b, const float2* t,
                                                bool beside) {
    float x0 = low(a), x1 = high(a), y0 = low(b), y1 = high(b);
    turn(x0, beside ? x1 : y0, t[0]);
    turn(beside ? y0 : x1, y1, t[1]);
    a = ptx::pack_bf16x2(x0, x1);
    b = ptx::pack_bf16x2(y0, y1);
  }
};
template <> struct Unit<__nv_bfloat16, 4> {
  using Word = uint2;
  static __device__ __forceinline__ void rotate(uint2& a, uint2& b, const float2* t,
                                                bool beside) {
    if (beside) {
      Unit<__nv_bfloat16, 2>::rotate(a.x, a.y, t, true);
      Unit<__nv_bfloat16, 2>::rotate(b.x, b.y, t + 2, true);
    } else {
      Unit<__nv_bfloat16, 2>::rotate(a.x, b.x, t, false);
      Unit<__nv_bfloat16, 2>::rotate(a.y, b.y, t + 2, false);
    }
  }
};
template <> struct Unit<float, 2> {
  using Word = float2;
  static __device__ __forceinline__ void rotate(float2& a, float2& b, const float2* t,
                                                bool beside) {
    turn(a.x, beside ? a.y : b.x, t[0]);
    turn(beside ? b.x : a.y, b.y, t[1]);
  }
};
template <> struct Unit<__nv_bfloat16, 1> {
  using Word = uint16_t;
  static __device__ __forceinline__ void rotate(uint16_t& a, uint16_t& b, const float2* t, bool) {
    float x = low(a), y = low(b);
    turn(x, y, t[0]);
    a = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    b = __bfloat16_as_ushort(__float2bfloat16_rn(y));
  }
};
template <> struct Unit<float, 1> {
  using Word = float;
  static __device__ __forceinline__ void rotate(float& a, float& b, const float2* t, bool) {
    turn(a, b, t[0]);
  }
};

struct Heads {
  int32_t q, kv, dim, block;
  int32_t per;                 // units per head,
  int32_t rotating;            // of which hold pairs
};

// Where pair p's turn lies in shared memory: a thread reads the kVec pairs of its
// column 16 bytes at a time, and eight columns' pieces then fall into different banks.
template <int kVec>
__device__ __forceinline__ int turn_at(int p) {
  const int col = p / kVec, e = p % kVec;
  const int flip = kVec == 8 ? (col >> 1) & 3 : kVec == 4 ? (col >> 2) & 1 : 0;
  return col * kVec + (e ^ (flip << 1));
}

template <class T, int kVec>
__global__ void __launch_bounds__(kThreads, 8)
    append_rotary_kernel(DevPass dp, DevTurns pos, Heads h, rbkv_rotary r, const void* q,
                         void* q_out, const void* __restrict__ k_new,
                         const void* __restrict__ v_new, void* __restrict__ k_cache,
                         void* __restrict__ v_cache) {
  using Word = typename Unit<T, kVec>::Word;
  __shared__ __align__(16) float2 turns_s[kThreads];
  // Launched to overlap its predecessor's tail: wait for it (it may have
  // produced the inputs, or still read cache blocks that are written here).
  ptx::pdl_wait_previous();
  ptx::pdl_launch_dependents();
  const int rows = pass_count(dp, kCountTokens, dp.num_tokens);
  const int tid = threadIdx.x;
  if (dp.built_for[0] &&
      (*dp.built_for[0] != h.block || *dp.built_for[1] != dp.num_tokens ||
       (pos.noted && *pos.planned_for[0] != *pos.planned_for[1]))) {
    if (tid == 0 && rows > 0) atomicCAS(dp.status, 0, kDevInvalid);
    return;
  }
  if (pos.noted && blockIdx.x == 0 && tid == 0) *pos.noted = *pos.planned_for[0];
  // A thread's units: one column of every `step`-th head (of Q's, then K's, then V's)
  const int step = kThreads / h.per, heads = h.q + 2 * h.kv, half = r.rotary_dim / 2;
  const int head0 = tid / h.per, col = tid - head0 * h.per;
  const bool turns = col < h.rotating, apart = turns && !r.interleaved;
  const int e0 = (apart ? 1 : 2) * col * kVec, e1 = e0 + (apart ? half : kVec);
  const int v0 = 2 * col * kVec, v1 = v0 + kVec;
  const bool live = head0 < step;
  for (int row = blockIdx.x; row < rows; row += gridDim.x) {
    float2 t[kVec];
    for (int x0 = 0; x0 < heads; x0 += kUnroll * step) {
      Word a[kUnroll], b[kUnroll];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int x = x0 + i * step + head0;
        if (!live || x >= heads) continue;
        const bool is_q = x < h.q, is_v = x >= h.q + h.kv;
        const T* p = is_q ? (const T*)q + ((int64_t)row * h.q + x) * h.dim
                          : (const T*)(is_v ? v_new : k_new) +
                                ((int64_t)row * h.kv + (x - h.q - (is_v ? h.kv : 0))) * h.dim;
        a[i] = *reinterpret_cast<const Word*>(p + (is_v ? v0 : e0));
        b[i] = *reinterpret_cast<const Word*>(p + (is_v ? v1 : e1));
      }
      const int slot = dp.slot[row];
      if (x0 == 0) {
        const uint32_t at = (uint32_t)(pos.position[row] + pos.offset);
        __syncthreads();      // (the previous row's are no longer needed)
        if (tid < half) {
          float s, c;
          sincospif((float)(int64_t)(r.turns[tid] * at) * 0x1p-63f, &s, &c);
          turns_s[turn_at<kVec>(tid)] = make_float2(c * r.scale, s * r.scale);
        }
        __syncthreads();
        if (turns) {
#pragma unroll
          for (int e = 0; e < kVec; ++e) t[e] = turns_s[turn_at<kVec>(col * kVec + e)];
        }
      }
      const int blk = slot / h.block, in_block = slot - blk * h.block;
      const bool inside = slot >= 0 && blk < dp.num_blocks;
      if (!inside && tid == 0) atomicCAS(dp.status, 0, kDevBounds);
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int x = x0 + i * step + head0;
        if (!live || x >= heads) continue;
        const bool is_q = x < h.q, is_v = x >= h.q + h.kv;
        if (turns && !is_v) Unit<T, kVec>::rotate(a[i], b[i], t, r.interleaved);
        if (!is_q && !inside) continue;
        T* to = is_q ? (T*)q_out + ((int64_t)row * h.q + x) * h.dim
                     : (T*)(is_v ? v_cache : k_cache) +
                           (((int64_t)blk * h.kv + (x - h.q - (is_v ? h.kv : 0))) * h.block +
                            in_block) * h.dim;
        *reinterpret_cast<Word*>(to + (is_v ? v0 : e0)) = a[i];
        *reinterpret_cast<Word*>(to + (is_v ? v1 : e1)) = b[i];
      }
    }
  }
}

template <class T, int kVec>
cudaError_t launch(const DevPass& dp, const DevTurns& at, const ShapeInfo& s,
                   const rbkv_rotary& r, const void* q, void* q_out, const void* k_new,
                   const void* v_new, void* k_cache, void* v_cache, cudaStream_t st,
                   bool overlap_previous) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  Heads h;
  h.q = s.H_q;
  h.kv = s.H_kv;
  h.dim = s.D;
  h.block = s.B;
  h.per = s.D / (2 * kVec);        // (at most kThreads: 256 / 2)
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
  return cudaLaunchKernelEx(&cfg, append_rotary_kernel<T, kVec>, dp, at, h, r, q, q_out,
                            k_new, v_new, k_cache, v_cache);
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
  if (!std::isfinite(r->scale)) return invalid("scale must be finite");
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
  if (overlap(k_cache, cache, v_cache, cache)) return invalid("the caches overlap");
  for (const void* c2 : {k_cache, v_cache})
    if (overlap(c2, cache, q, q_bytes) || overlap(c2, cache, k_new, kv_bytes) ||
        overlap(c2, cache, v_new, kv_bytes) ||
        overlap(c2, cache, r->turns, 4 * (int64_t)r->rotary_dim))
      return invalid("a cache overlaps what the call reads");
  return RBKV_OK;
}

cudaError_t launch_append_rotary(const DevPass& dp, const DevTurns& at, const ShapeInfo& s,
                                 const rbkv_rotary& r, const void* q, void* q_out,
                                 const void* k_new, const void* v_new, void* k_cache,
                                 void* v_cache, cudaStream_t st, bool overlap_previous) {
  if (dp.num_tokens == 0) return cudaSuccess;
  // the widest words of which both of a unit lie among the rotated elements, or both
  // behind them (512 rows of 32 and 8 heads of 128, bf16: 20 elements rotated in words
  // of one 10.4 us, of two 6.9, the call's own time; 24 in words of four 7.0)
  const int R = r.rotary_dim;
  auto fn = launch<float, 1>;
  if (s.dtype == 0)
    fn = R % 16 == 0  ? launch<__nv_bfloat16, 8>
         : R % 8 == 0 ? launch<__nv_bfloat16, 4>
         : R % 4 == 0 ? launch<__nv_bfloat16, 2>
                      : launch<__nv_bfloat16, 1>;
  else
    fn = R % 8 == 0 ? launch<float, 4> : R % 4 == 0 ? launch<float, 2> : launch<float, 1>;
  return fn(dp, at, s, r, q, q_out, k_new, v_new, k_cache, v_cache, st, overlap_previous);
}

}  // namespace rbkv
