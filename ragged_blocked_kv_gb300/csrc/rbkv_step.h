// Structures of a step whose metadata lives on the device (rbkv_step_*):
// shared by its host side (rbkv_step.cpp) and kernels.
#pragma once

#include "rbkv_internal.h"

namespace rbkv {

// Sequences whose packed query rows (new tokens x heads of a KV group) number
// at most this go to the streaming kernel, longer ones to the tile kernel.
constexpr int kStepPackedRows = 16;
constexpr int kStepStreamKeys = 64;     // keys per tile of the streaming kernel
constexpr int kStepTileKeys = 128;      // keys per tile of the tensor-core kernel
constexpr int kStepTileRows = 128;      // packed query rows per tensor-core tile

// Tokens whose packed rows fill one tensor-core query tile.
__host__ __device__ __forceinline__ int step_tile_tokens(int g) { return kStepTileRows / g; }

// Header words of the plan.
enum {
  kPlanRows = 0,        // query rows of the step (q_start[num_seqs])
  kPlanStreamed = 1,    // sequences on the streaming kernel
  kPlanTiled = 2,       // sequences on the tile kernel
  kPlanStreamTiles = 3, // 64-key tiles of the streamed sequences, for one KV head
  kPlanTileSteps = 4,   // key-tile steps of the tiled sequences, for one KV head
  kPlanHeader = 16
};

// The plan: int32 arrays in one buffer.
struct StepPlan {
  int32_t* header;      // [kPlanHeader]
  int32_t* row_seq;     // [max_tokens] sequence of each row
  int32_t* seq_unit;    // [S] index into stream_seq, or -1 - index into tile_seq
  int32_t* stream_seq;  // [S] streamed sequences, in order
  int32_t* stream_cum;  // [S + 1] 64-key tiles before each of them
  int32_t* tile_seq;    // [S] tiled sequences, in order
  int32_t* tile_cum;    // [S + 1] key-tile steps before each of them
  int32_t* first_new;   // [S] scratch: rank of a sequence's first new block
  int32_t* new_ids;     // [max_tokens] scratch: the new block ids, by rank
};

__host__ __device__ __forceinline__ int64_t step_plan_ints(int64_t num_seqs, int64_t max_tokens) {
  return kPlanHeader + 2 * max_tokens + 6 * num_seqs + 2;
}

__host__ __device__ __forceinline__ StepPlan step_plan(int32_t* p, int32_t num_seqs,
                                                       int32_t max_tokens) {
  StepPlan v;
  const int64_t S = num_seqs;
  v.header = p;
  v.row_seq = p + kPlanHeader;
  v.seq_unit = v.row_seq + max_tokens;
  v.stream_seq = v.seq_unit + S;
  v.stream_cum = v.stream_seq + S;
  v.tile_seq = v.stream_cum + S + 1;
  v.tile_cum = v.tile_seq + S;
  v.first_new = v.tile_cum + S + 1;
  v.new_ids = v.first_new + S;
  return v;
}

// Sum of floor((a i + b) / m) over i = 0 .. n - 1, for n, a, b >= 0 and m > 0.
// The whole multiples of m in a and b are summed in closed form; what is left
// counts lattice points under a line, which is the same sum with the axes
// exchanged: as many rounds as Euclid's algorithm takes on (a, m).
__host__ __device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t total = 0;
  while (n > 0) {
    total += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const int64_t top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const int64_t t = a;
    a = m;
    m = t;
  }
  return total;
}

// A tiled sequence's new tokens are taken in pairs of tensor-core tiles of
// `pair` tokens together.  Pair k sees the keys below
// seen + min(n_new, (k + 1) pair): its key-tile steps, and those before it.
__host__ __device__ __forceinline__ int32_t step_pair_steps(int32_t seen, int32_t n_new,
                                                            int32_t pair, int32_t k) {
  const int64_t end = (int64_t)(k + 1) * pair;
  const int64_t keys = seen + (end < n_new ? end : (int64_t)n_new);
  return (int32_t)((keys + kStepTileKeys - 1) / kStepTileKeys);
}
__host__ __device__ __forceinline__ int64_t step_steps_before(int32_t seen, int32_t pair,
                                                              int32_t k) {
  // every pair before another one is whole
  return floor_sum(k, kStepTileKeys, pair, (int64_t)seen + pair + kStepTileKeys - 1);
}
__host__ __device__ __forceinline__ int64_t step_seq_steps(int32_t seen, int32_t n_new,
                                                           int32_t pair) {
  const int32_t pairs = (int32_t)(((int64_t)n_new + pair - 1) / pair);
  return step_steps_before(seen, pair, pairs - 1) +
         step_pair_steps(seen, n_new, pair, pairs - 1);
}

// What the kernels of a step see.
struct DevStep {
  int32_t num_seqs, max_blocks, max_tokens, num_blocks;
  const int32_t* block_table;   // [S][max_blocks]
  const int32_t* q_start;       // [S + 1]
  const int32_t* ctx;           // [S]
  int32_t* plan;
  int32_t* status;
  const int32_t* prefix_table;
  int32_t prefix_len;
};

// Work is cut evenly over the CTAs of a persistent grid.  All key tiles of a
// kernel's work units lie on one line, units one after the other; with
// G' = min(grid, total), CTA c walks the tiles [start(c), start(c + 1)),
// start(c) = floor(c total / G').  A unit is so cut into one segment per CTA
// that meets it.  The segment at a unit's first tile writes its result to the
// unit's own rows of the workspace; a segment that begins inside a unit can
// only be the first of its CTA, and goes to that CTA's spill rows.
__host__ __device__ __forceinline__ int64_t step_cut(int64_t c, int64_t total, int64_t ctas) {
  return c * total / ctas;
}

// The units of the streaming kernel: (streamed sequence, KV head), the KV
// heads of a sequence in order; then, when the whole step has at most
// kStepPackedRows packed rows, the prefix as one more sequence.
// The units of the tile kernel: (KV head, pair of query tiles) over the
// prefix unless it is streamed; then (tiled sequence, KV head, pair).
struct StepWork {
  int64_t stream_own, stream_total;   // 64-key tiles
  int64_t tile_prefix, tile_total;    // key-tile steps
  int32_t prefix_stream_tiles;        // 64-key tiles of the prefix, when streamed
  int32_t prefix_tile_steps;          // 128-key tiles of the prefix, when tiled
  int32_t prefix_pairs;               // pairs of query tiles over the prefix
};

__host__ __device__ __forceinline__ bool step_prefix_streamed(int32_t max_tokens, int32_t g) {
  return (int64_t)max_tokens * g <= kStepPackedRows;
}

#ifdef __CUDACC__
__device__ __forceinline__ StepWork step_work(const DevStep& ds, const ShapeInfo& s,
                                              const StepPlan& plan) {
  StepWork w;
  const int32_t T = plan.header[kPlanRows];
  const bool streamed = step_prefix_streamed(ds.max_tokens, s.g);
  const int32_t P = T > 0 ? ds.prefix_len : 0;
  w.prefix_stream_tiles = streamed ? (P + kStepStreamKeys - 1) / kStepStreamKeys : 0;
  w.prefix_tile_steps = streamed ? 0 : (int32_t)(((int64_t)P + kStepTileKeys - 1) / kStepTileKeys);
  const int32_t pair = 2 * step_tile_tokens(s.g);
  w.prefix_pairs = (T + pair - 1) / pair;
  w.stream_own = (int64_t)plan.header[kPlanStreamTiles] * s.H_kv;
  w.stream_total = w.stream_own + (int64_t)w.prefix_stream_tiles * s.H_kv;
  w.tile_prefix = (int64_t)s.H_kv * w.prefix_pairs * w.prefix_tile_steps;
  w.tile_total = w.tile_prefix + (int64_t)plan.header[kPlanTileSteps] * s.H_kv;
  return w;
}
#endif

// The workspace: fp32 partial outputs (head dim 128) and base-2 log-sum-exps.
struct StepWorkspace {
  float *own_o, *pre_o;         // [max_tokens][H_q][128]
  float *own_lse, *pre_lse;     // [max_tokens][H_q]
  float *stream_o, *stream_lse; // spill rows [stream grid][kStepPackedRows]
  float *tile_o, *tile_lse;     // spill rows [tile grid][2 kStepTileRows]
  int32_t stream_grid, tile_grid;
};

bool step_fast_supported(const ShapeInfo& s);
// Carve a workspace at `base` (may be null); returns its bytes.
size_t step_workspace(const ShapeInfo& s, int32_t max_tokens, int sms, void* base,
                      StepWorkspace* w);

struct BuildArgs {
  int32_t num_seqs, max_blocks, max_tokens, num_blocks;
  int32_t block_size, group;
  const int32_t *seen, *n_new, *table_in, *free_in;
  int32_t *table, *free_words, *q_start, *ctx, *position, *slot, *plan, *status;
};

cudaError_t launch_step_build(const BuildArgs& a, cudaStream_t st);
cudaError_t launch_step_release(const BuildArgs& a, const int32_t* done, cudaStream_t st);
// CUDA-core attention of a step: every type and shape.
cudaError_t launch_step_generic(const DevStep& ds, const ShapeInfo& s, const void* q,
                                const void* k_cache, const void* v_cache, void* o,
                                cudaStream_t st);
// The fast path's three kernels.  The first one launched of the first two
// waits for the stream's previous kernel (`first`); the other starts beside
// it and waits for it before ending; the combine waits for both.
cudaError_t launch_step_tile(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w,
                             const void* q, const void* k_cache, const void* v_cache, void* o,
                             bool first, cudaStream_t st);
cudaError_t launch_step_stream(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w,
                               const void* q, const void* k_cache, const void* v_cache, void* o,
                               bool first, cudaStream_t st);
cudaError_t launch_step_combine(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w,
                                void* o, cudaStream_t st);
}  // namespace rbkv
