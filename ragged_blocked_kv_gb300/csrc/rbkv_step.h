// Structures of a step whose metadata lives on the device (rbkv_step_*):
// shared by its host side (rbkv_step.cpp) and kernels.
#pragma once

#include "rbkv_internal.h"

namespace rbkv {

// Sequences whose packed query rows (new tokens x heads of a KV group) number
// at most this go to the streaming kernel, longer ones to the tile kernel.
constexpr int kStepPackedRows = 16;
constexpr int kStepStreamKeys = 16;     // keys per tile of the streaming kernel
constexpr int kStepPipes = 4;           // its pipelines (warps) per CTA
constexpr int kStepTileKeys = 128;      // keys per tile of the tensor-core kernel
constexpr int kStepTileRows = 128;      // packed query rows per tensor-core tile

// Drafted tokens of a sequence, at most (a set of ancestors is four words).
constexpr int kStepTreeTokens = RBKV_DRAFT_TOKENS;

// Tokens whose packed rows fill one tensor-core query tile.
__host__ __device__ __forceinline__ int step_tile_tokens(int g) { return kStepTileRows / g; }

// Shared memory of a tile kernel CTA (beside which a streaming one fits).
constexpr int kStepTileSmem = 4 * 32768 + 1024;

// What a unit of work costs beside its key tiles (queries in, results out), in
// key tiles of its kernel, for the even cut of the work over the CTAs.
constexpr int kStepStreamUnit = 3;
constexpr int kStepTileUnit = 5;
// Key tiles of a sequence from which on its query tiles are walked in pairs.
constexpr int kStepPairTiles = 8;

// Header words of the plan.
enum {
  kPlanRows = 0,        // query rows of the step (q_start[num_seqs])
  kPlanStreamed = 1,    // sequences on the streaming kernel
  kPlanTiled = 2,       // sequences on the tile kernel
  kPlanStreamLen = 3,   // line length of the streamed sequences, for one KV head
  kPlanTileLen = 4,     // line length of the tiled sequences, for one KV head
  // what the step was built for: the plan's layout, work lists and lengths
  // depend on these, so its readers compare them with what they were given
  kPlanGroup = 5,       // query heads per KV head
  kPlanBlock = 6,       // block size
  kPlanSeqs = 7,
  kPlanTokens = 8,
  kPlanMaxBlocks = 9,
  kPlanPool = 10,       // blocks of the pool
  kPlanSerial = 11,     // builds so far
  kPlanTurned = 12,     // serial of the last build whose rows were rotated by their places
  kPlanHeader = 16
};

// A sequence of a kernel's work list.  cum: line length before it, for one KV
// head; tiles: 16-key tiles (streamed) or line length (tiled).
struct StepSeq {
  int32_t seq, row, n_new, ctx, cum, tiles;
  int32_t pad[2];
};
static_assert(sizeof(StepSeq) == 32, "StepSeq is 8 int32");

// A query row: unit >= 0: entry of the streamed list; else -1 - unit: entry of
// the tiled list.  token: its index among its sequence's new tokens.
struct StepRow {
  int32_t unit, token, pad[2];
};
static_assert(sizeof(StepRow) == 16, "StepRow is 4 int32");

// The plan: one int32 buffer (16-byte aligned).
struct StepPlan {
  int32_t* header;      // [kPlanHeader]
  StepRow* rows;        // [max_tokens]
  StepSeq* streamed;    // [S], in sequence order
  StepSeq* tiled;       // [S], in sequence order
  StepRow* of_seq;      // [S] scratch: unit of a sequence; token is the rank of its
                        // first new block
  int32_t* new_ids;     // [max_tokens] scratch: the new block ids, by rank
};

__host__ __device__ __forceinline__ int64_t step_plan_ints(int64_t num_seqs, int64_t max_tokens) {
  return kPlanHeader + 5 * max_tokens + 20 * num_seqs;
}

__host__ __device__ __forceinline__ StepPlan step_plan(int32_t* p, int32_t num_seqs,
                                                       int32_t max_tokens) {
  StepPlan v;
  v.header = p;
  v.rows = reinterpret_cast<StepRow*>(p + kPlanHeader);
  v.streamed = reinterpret_cast<StepSeq*>(v.rows + max_tokens);
  v.tiled = v.streamed + num_seqs;
  v.of_seq = reinterpret_cast<StepRow*>(v.tiled + num_seqs);
  v.new_ids = reinterpret_cast<int32_t*>(v.of_seq + num_seqs);
  return v;
}

// a / b for a >= 0, b > 0 (a 64-bit division takes several times as long).
__host__ __device__ __forceinline__ int64_t step_div(int64_t a, int64_t b) {
  if (((uint64_t)a | (uint64_t)b) >> 32) return a / b;
  return (int64_t)((uint32_t)a / (uint32_t)b);
}

// Sum of floor((a i + b) / m) over i = 0 .. n - 1, for n, a, b >= 0 and m > 0.
// The whole multiples of m in a and b are summed in closed form; what is left
// counts lattice points under a line, which is the same sum with the axes
// exchanged: as many rounds as Euclid's algorithm takes on (a, m).
__host__ __device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t total = 0;
  while (n > 0) {
    const int64_t qa = step_div(a, m), qb = step_div(b, m);
    total += n * (n - 1) / 2 * qa + n * qb;
    a -= qa * m;
    b -= qb * m;
    const int64_t top = a * n + b;
    if (top < m) break;
    n = step_div(top, m);
    b = top - n * m;
    const int64_t t = a;
    a = m;
    m = t;
  }
  return total;
}

// A tiled sequence's new tokens are taken in query tiles of `tokens` each.
// Tile k sees the keys below seen + min(n_new, (k + 1) tokens): its key tiles;
// the line length of the query tiles before it; and that of all of them.
__host__ __device__ __forceinline__ int32_t step_key_tiles(int32_t seen, int32_t n_new,
                                                           int32_t tokens, int32_t k) {
  const int64_t end = (int64_t)(k + 1) * tokens;
  const int64_t keys = seen + (end < n_new ? end : (int64_t)n_new);
  return (int32_t)((keys + kStepTileKeys - 1) / kStepTileKeys);
}
__host__ __device__ __forceinline__ int64_t step_len_before(int32_t seen, int32_t tokens,
                                                            int32_t k) {
  // every tile before another one is whole
  return floor_sum(k, kStepTileKeys, tokens, (int64_t)seen + tokens + kStepTileKeys - 1) +
         (int64_t)k * kStepTileUnit;
}
__host__ __device__ __forceinline__ int64_t step_seq_len(int32_t seen, int32_t n_new,
                                                         int32_t tokens) {
  const int32_t tiles = (int32_t)(((int64_t)n_new + tokens - 1) / tokens);
  return step_len_before(seen, tokens, tiles - 1) +
         step_key_tiles(seen, n_new, tokens, tiles - 1) + kStepTileUnit;
}

// Drafted tokens: where a tiled sequence's units lie on the tile kernel's road.
//
// Query tiles of one sequence and KV head read the same keys, and one after the
// other on the line above they read them again from HBM: between two reads of a
// key lies what all CTAs read in the time of a unit (a tree of 64 tokens in groups
// of 4 behind 32768 keys: 260 MB for 137).  So two neighbouring query tiles are a
// pair, walked side by side by a pair of CTAs.  The road has one place for a step
// of both lanes: first, two to a place, the steps of units of one tile (over the
// prefix, and a sequence's last tile where their number is odd), then those of the
// pairs, as long as the second tile's.  A pair of CTAs takes an even cut of it;
// of the single units' steps in its part the first CTA walks the first half.
// (Entry 0 of the list holds the totals as lengths, the serial of the build that
// the trees were planned for as single_cum, and of the one whose paths were taken
// as pair_cum.)
struct __align__(16) StepLanes {
  int32_t single_cum, single_len;     // for one KV head, as StepSeq's
  int32_t pair_cum, pair_len;
};
static_assert(sizeof(StepLanes) == 16, "StepLanes is 4 int32");

// Pairs of a sequence, and their places and the steps of its other units, for one
// KV head.  Tiles of few keys are left single: what a unit reads is then still in
// the L2 when the next one does.
__host__ __device__ __forceinline__ int32_t step_pairs(int32_t seen, int32_t n_new,
                                                       int32_t tokens) {
  const int32_t tiles = (int32_t)(((int64_t)n_new + tokens - 1) / tokens);
  return step_key_tiles(seen, n_new, tokens, tiles - 1) >= kStepPairTiles ? tiles / 2 : 0;
}
__host__ __device__ __forceinline__ int32_t step_singles_len(int32_t seen, int32_t n_new,
                                                             int32_t tokens, int32_t pairs) {
  const int32_t tiles = (int32_t)(((int64_t)n_new + tokens - 1) / tokens);
  if (pairs == 0) return step_seq_len(seen, n_new, tokens);
  return tiles & 1 ? step_key_tiles(seen, n_new, tokens, tiles - 1) + kStepTileUnit : 0;
}
__host__ __device__ __forceinline__ int32_t step_pairs_len(int32_t seen, int32_t n_new,
                                                           int32_t tokens, int32_t pairs) {
  if (pairs == 0) return 0;
  // every pair before the last is whole
  return (int32_t)(floor_sum(pairs - 1, kStepTileKeys, 2 * tokens,
                             (int64_t)seen + 2 * tokens + kStepTileKeys - 1) +
                   step_key_tiles(seen, n_new, tokens, 2 * pairs - 1) +
                   (int64_t)pairs * kStepTileUnit);
}

// A unit's spills are every CTA's that follows, or every other one's.
constexpr int32_t kSpillsApart = 1 << 30;

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
  // drafted tokens (null: every row sees its sequence's earlier ones)
  const int32_t* place;         // [max_tokens]
  const uint4* ancestors;       // [max_tokens]
  const StepLanes* work;        // [num_seqs + 1]: totals, then the tiled sequences
};

// Work is cut evenly over the CTAs of a persistent grid.  A kernel's units lie
// on one line, one after the other, each as long as its key tiles and a fixed
// length for what it costs beside them (first the fixed length, then the
// tiles); with G' = min(grid, total), CTA c takes [start(c), start(c + 1)),
// start(c) = floor(c total / G').  A unit is so cut into segments of key tiles.
// The segment at a unit's first tile writes its result to the unit's own rows
// of the workspace; a segment that begins inside a unit can only be the first
// of its CTA, and goes to that CTA's spill rows: CTAs c + 1, c + 2, ... where
// CTA c holds the unit's first tile.
__host__ __device__ __forceinline__ int64_t step_cut(int64_t c, int64_t total, int64_t ctas) {
  return step_div(c * total, ctas);
}

// The units of the streaming kernel: (streamed sequence, KV head), the KV
// heads of a sequence in order; then, when the whole step has at most
// kStepPackedRows packed rows, the prefix as one more sequence.
// The units of the tile kernel: (KV head, query tile) over the prefix unless it
// is streamed; then (tiled sequence, KV head, query tile).
struct StepWork {
  int64_t stream_own, stream_total;
  int64_t tile_prefix, tile_total;
  int32_t rows, streamed;             // query rows; streamed sequences
  int32_t prefix_stream_tiles;        // 16-key tiles of the prefix, when streamed
  int32_t prefix_tile_steps;          // 128-key tiles of the prefix, when tiled
  int32_t prefix_rows;                // query tiles of a KV head over the prefix
};

// (Tiled even then, a step of one row of 32 heads in 8 groups takes 11.8 us behind
// 512 keys and 32.4 behind 32768, streamed 7.6 and 28.7; of 16 rows, one head
// per group, 24.2 and 21.5 behind 512 keys.)
__host__ __device__ __forceinline__ bool step_prefix_streamed(int32_t max_tokens, int32_t g) {
  return (int64_t)max_tokens * g <= kStepPackedRows;
}

#ifdef __CUDACC__
// Whether the step was built for what it is used with: else its lengths and
// lists would lead out of the tables.  kDraft: and whether its trees were planned for
// this build.  (Not asked of ds.place: that branch, untaken, cost a step without drafts
// 1 us: 512 rows behind 4096 keys 124.5 to 125.3 in a graph, 64 rows of 64 heads behind
// 15999 59.5 to 60.6.)
template <bool kDraft>
__device__ __forceinline__ bool step_matches(const DevStep& ds, const ShapeInfo& s,
                                             const StepPlan& plan) {
  static_assert(kPlanGroup == 5 && kPlanBlock == 6 && kPlanSeqs == 7 && kPlanTokens == 8 &&
                    kPlanMaxBlocks == 9, "the header's second and third vector");
  const int4 b = *reinterpret_cast<const int4*>(plan.header + 4);
  const int2 c = *reinterpret_cast<const int2*>(plan.header + 8);
  int32_t stale = 0;
  if constexpr (kDraft) stale = ds.work[0].single_cum ^ plan.header[kPlanSerial];
  // (no short cuts: all of it in one round trip)
  return ((b.y ^ s.g) | (b.z ^ s.B) | (b.w ^ ds.num_seqs) | (c.x ^ ds.max_tokens) |
          (c.y ^ ds.max_blocks) | stale) == 0;
}
// The step's rows; 0, and RBKV_ERR_INVALID in the status words, where it was
// built for something else.  (The tile and the streaming kernel leave the report
// to the join.)
template <bool kDraft>
__device__ __forceinline__ int32_t step_rows(const DevStep& ds, const ShapeInfo& s,
                                             const StepPlan& plan) {
  const int32_t rows = plan.header[kPlanRows];
  if (step_matches<kDraft>(ds, s, plan)) return rows;
  if (rows > 0 && threadIdx.x == 0) atomicCAS(ds.status, 0, kDevInvalid);
  return 0;
}

__device__ __forceinline__ StepWork step_work(const DevStep& ds, const ShapeInfo& s,
                                              const StepPlan& plan) {
  StepWork w;
  const int4 h = *reinterpret_cast<const int4*>(plan.header);
  const int32_t T = h.x;
  w.rows = T;
  w.streamed = h.y;
  const bool streamed = step_prefix_streamed(ds.max_tokens, s.g);
  const int32_t P = T > 0 ? ds.prefix_len : 0;
  w.prefix_stream_tiles = streamed ? (P + kStepStreamKeys - 1) / kStepStreamKeys : 0;
  w.prefix_tile_steps = streamed ? 0 : (int32_t)(((int64_t)P + kStepTileKeys - 1) / kStepTileKeys);
  const int32_t tokens = step_tile_tokens(s.g);
  w.prefix_rows = (T + tokens - 1) / tokens;
  w.stream_own = (int64_t)h.w * s.H_kv;
  w.stream_total = w.stream_own;
  if (w.prefix_stream_tiles)
    w.stream_total += (int64_t)(w.prefix_stream_tiles + kStepStreamUnit) * s.H_kv;
  w.tile_prefix = 0;
  if (w.prefix_tile_steps)
    w.tile_prefix = (int64_t)s.H_kv * w.prefix_rows * (w.prefix_tile_steps + kStepTileUnit);
  w.tile_total = w.tile_prefix + (int64_t)plan.header[kPlanTileLen] * s.H_kv;
  return w;
}
#endif

#ifdef __CUDACC__
// Drafted tokens: what the row of token `token` of a sequence sees of its own
// keys.  A row sees a run of keys from the first, up to key `last`, and of those
// behind it the keys seen + i with bit i of its ancestors: a row that follows all
// tokens before it (its depth is its index) sees them as one run, any other the
// tokens cached before the step.  (Sequences of more than kStepTreeTokens new
// tokens are chains, all runs.)
__device__ __forceinline__ bool draft_is_run(const DevStep& ds, int row, int seen, int token) {
  return ds.place[row] - seen == token;
}
// Words of the ancestors' set moved down by `by` bits (up, where negative).
__device__ __forceinline__ void draft_window(const uint4& set, int by, uint32_t (&w)[4]) {
  const uint32_t m[4] = {set.x, set.y, set.z, set.w};
  const int words = by >> 5, bits = by & 31;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      if (y == x + words) lo = m[y];
      if (y == x + words + 1) hi = m[y];
    }
    w[x] = __funnelshift_r(lo, hi, bits);
  }
}
// Bit i of a set (none outside it).
__device__ __forceinline__ bool draft_bit(const uint4& set, int i) {
  const uint32_t w = i < 64 ? (i < 32 ? set.x : set.y) : (i < 96 ? set.z : set.w);
  return (uint32_t)i < (uint32_t)kStepTreeTokens && (w >> (i & 31) & 1u);
}

// 0xffff over each of two bf16 that is an infinity or NaN.
//
// A row must not see the values of later tokens of its sequence, and in a
// matrix product a weight of 0 does not hide one that is not finite.  Where
// some rows of a unit see a key and others do not, the kernels look for such
// values, zero them in shared memory and add them as they are to the rows that
// see them (their weights are positive: the sums are what they would be).
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
         ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}
// Zeroes those of 8 bf16; true if there were any.
__device__ __forceinline__ bool zero_nonfinite(uint4* p) {
  const uint4 w = *p;
  const uint4 m = make_uint4(nonfinite2(w.x), nonfinite2(w.y), nonfinite2(w.z), nonfinite2(w.w));
  if (!(m.x | m.y | m.z | m.w)) return false;
  *p = make_uint4(w.x & ~m.x, w.y & ~m.y, w.z & ~m.z, w.w & ~m.w);
  return true;
}
#endif

// CTAs (or pipelines) whose spill rows hold the rest of a cut unit.
struct Spills {
  int32_t first, n;
};

// The workspace: fp32 partial outputs (head dim 128) and base-2 log-sum-exps,
// and what is to be joined.  The segment at a unit's first tile fills in the
// unit's Spills, at the unit's first row (a streamed prefix: row 0).
struct StepWorkspace {
  float *own_o, *pre_o;         // [max_tokens][H_q][128]
  float *own_lse, *pre_lse;     // [max_tokens][H_q]
  float *stream_o, *stream_lse; // spill rows [stream grid kStepPipes][kStepPackedRows]
  float *tile_o, *tile_lse;     // spill rows [tile grid][kStepTileRows]
  Spills *own_cut, *pre_cut;    // [max_tokens][H_kv]
  int32_t stream_grid, tile_grid;     // CTAs (the streaming kernel's: two per SM)
};

#ifdef __CUDACC__
// The streaming kernel's pipelines: kStepPipes in each of two CTAs per SM.
// Without tile work both CTAs of an SM run from the start and share its line
// evenly.  With it, the second one only fits once the tile kernel's CTA has
// left: the early CTAs take [0, cut) of the line and the late ones the rest,
// such that both end together.  Let x be the share of the streaming that the
// early ones do while the tile kernel runs; they do it at about 1.75 ns per
// 16-key group of the whole line (5.2 TB/s beside the tile kernel), which takes
// about 1.5 us per step then (1.05 alone) and 4 us to start.  What is left
// after that is shared evenly: the early ones' part is x + (1 - x) / 2.  (On 512
// sequences of 256 keys behind 4096 shared ones, with everything given to the
// early CTAs, the late ones idled for half of 130 us.)
struct StreamCuts {
  int64_t cut, total;       // the line
  int32_t early, late;      // pipelines of [0, cut) and of [cut, total)

  // where pipeline c's part begins
  __device__ __forceinline__ int64_t at(int32_t c) const {
    if (c < early) return step_cut(c, cut, early);
    return c < early + late ? cut + step_cut(c - early, total - cut, late) : total;
  }
  // the first pipeline whose part begins at or behind p (0 < p <= total)
  __device__ __forceinline__ int32_t first(int64_t p) const {
    if (p <= cut) return (int32_t)step_div(p * early + cut - 1, cut);
    return early + (int32_t)step_div((p - cut) * late + total - cut - 1, total - cut);
  }
};

__device__ __forceinline__ StreamCuts step_stream_cuts(const StepWorkspace& ws,
                                                       const StepWork& work) {
  StreamCuts c;
  const int64_t half = (int64_t)ws.stream_grid / 2 * kStepPipes;
  c.total = work.stream_total;
  c.cut = (c.total + 1) / 2;
  if (work.tile_total > 0) {
    const int64_t tile_ns = step_div(work.tile_total * 1500, ws.tile_grid) + 4000;
    const int64_t stream_ns = c.total * 7 / 4;
    const float part = 0.5f * ((float)tile_ns / (float)stream_ns);
    c.cut = tile_ns >= stream_ns ? c.total : c.total / 2 + (int64_t)((float)c.total * part);
  }
  c.early = (int32_t)(c.cut < half ? c.cut : half);
  c.late = (int32_t)(c.total - c.cut < half ? c.total - c.cut : half);
  return c;
}
#endif

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

// Drafted tokens (rbkv_draft.cu).
struct DraftArgs {
  int32_t num_seqs, max_blocks, max_tokens, num_blocks, block_size;
  const int32_t *q_start, *position, *slot, *table;
  int32_t *ctx, *free_words, *plan, *status;
  const int32_t *parent, *tokens, *chosen, *given;
  int32_t *place, *ancestors, *path, *accepted, *next_token, *work;
};
cudaError_t launch_draft_plan(const DraftArgs& a, cudaStream_t st);
cudaError_t launch_draft_accept(const DraftArgs& a, cudaStream_t st);
cudaError_t launch_draft_compact(const DraftArgs& a, const ShapeInfo& s, void* k_cache,
                                 void* v_cache, cudaStream_t st);

cudaError_t launch_step_build(const BuildArgs& a, cudaStream_t st);
cudaError_t launch_step_release(const BuildArgs& a, const int32_t* done, cudaStream_t st);
// CUDA-core attention of a step: every type and shape, its packed rows a few to
// a block and the keys of each shared by `splits` blocks (more than one: with
// a workspace and a second kernel).
constexpr int kStepGenericSplits = 32;
int step_generic_splits(const ShapeInfo& s, int32_t max_tokens, int32_t max_blocks,
                        int32_t prefix_len, int sms);
size_t step_generic_workspace(const ShapeInfo& s, int32_t max_tokens, int splits);
cudaError_t launch_step_generic(const DevStep& ds, const ShapeInfo& s, const void* q,
                                const void* k_cache, const void* v_cache, void* o,
                                void* workspace, int splits, int sms, cudaStream_t st);
// The fast path's three kernels.  The tile kernel, where there is one, is
// launched first and waits for the stream's previous kernel; the streaming
// kernel starts beside it and waits for it before ending, or is the `first`
// one itself; the combine waits for both.
cudaError_t launch_step_tile(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w,
                             const void* q, const void* k_cache, const void* v_cache, void* o,
                             cudaStream_t st);
cudaError_t launch_step_stream(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w,
                               const void* q, const void* k_cache, const void* v_cache, void* o,
                               bool first, cudaStream_t st);
cudaError_t launch_step_combine(const DevStep& ds, const ShapeInfo& s, const StepWorkspace& w,
                                void* o, cudaStream_t st);
}  // namespace rbkv
