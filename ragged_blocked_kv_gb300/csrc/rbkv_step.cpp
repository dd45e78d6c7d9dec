// Host side of a step whose metadata lives on the device: argument checks and
// launches.  Nothing here reads a device array; every count the kernels need
// comes from the tables' plan on the device.
#include <cmath>
#include <string>

#include "rbkv_step.h"

#include <cuda_runtime.h>

using namespace rbkv;

namespace {

rbkv_status fail(rbkv_status st, const char* msg) { return set_error(st, msg); }
rbkv_status invalid(const char* msg) { return fail(RBKV_ERR_INVALID, msg); }
rbkv_status cuda_fail(cudaError_t e, const char* what) {
  return fail(RBKV_ERR_CUDA, (std::string(what) + ": " + cudaGetErrorString(e)).c_str());
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

rbkv_status check_tables(const rbkv_config* c, const rbkv_step_tables* t) {
  rbkv_status st = check_config(c);
  if (st != RBKV_OK) return st;
  if (!t) return invalid("tables is NULL");
  if (t->num_seqs < 1 || t->max_blocks < 1 || t->max_tokens < 1)
    return invalid("num_seqs, max_blocks and max_tokens must be >= 1");
  if (c->num_blocks < 1) return invalid("a step needs a pool of at least one block");
  if (step_plan_ints(t->num_seqs, t->max_tokens) >= (int64_t)1 << 31)
    return invalid("num_seqs and max_tokens are too large for one plan");
  if (!t->block_table || !t->free_words || !t->q_start || !t->ctx || !t->position || !t->slot ||
      !t->plan || !t->status)
    return invalid("NULL table array");
  if (!aligned(t->block_table, 4) || !aligned(t->free_words, 4) || !aligned(t->q_start, 4) ||
      !aligned(t->ctx, 4) || !aligned(t->position, 4) || !aligned(t->slot, 4) ||
      !aligned(t->status, 4))
    return invalid("table arrays must be 4-byte aligned");
  if (!aligned(t->plan, 16)) return invalid("plan must be 16-byte aligned");
  return RBKV_OK;
}

// Whether the n int32 at p meet an array that a build writes, other than the
// one (of the same length) that they may be read from in place.
bool written_by_build(const rbkv_step_tables* t, int32_t num_blocks, const void* p, int64_t n,
                      const void* in_place) {
  if (p == in_place) return false;
  const int64_t S = t->num_seqs, T = t->max_tokens;
  return overlap(p, 4 * n, t->block_table, 4 * S * t->max_blocks) ||
         overlap(p, 4 * n, t->free_words, 4 * (((int64_t)num_blocks + 31) / 32)) ||
         overlap(p, 4 * n, t->q_start, 4 * (S + 1)) || overlap(p, 4 * n, t->ctx, 4 * S) ||
         overlap(p, 4 * n, t->position, 4 * T) || overlap(p, 4 * n, t->slot, 4 * T) ||
         overlap(p, 4 * n, t->plan, 4 * step_plan_ints(S, T)) ||
         overlap(p, 4 * n, t->status, 16);
}

BuildArgs build_args(const rbkv_config* c, const rbkv_step_tables* t) {
  BuildArgs a = {};
  a.num_seqs = t->num_seqs;
  a.max_blocks = t->max_blocks;
  a.max_tokens = t->max_tokens;
  a.num_blocks = c->num_blocks;
  a.block_size = c->block_size;
  a.group = c->num_heads_q / c->num_heads_kv;
  a.table_in = a.table = t->block_table;
  a.free_in = a.free_words = t->free_words;
  a.q_start = t->q_start;
  a.ctx = t->ctx;
  a.position = t->position;
  a.slot = t->slot;
  a.plan = t->plan;
  a.status = t->status;
  return a;
}

cudaError_t num_sms(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && *sms < 1) e = cudaErrorInvalidDevice;
  return e;
}

ShapeInfo shape(const rbkv_config* c) {
  ShapeInfo s;
  s.H_q = c->num_heads_q;
  s.H_kv = c->num_heads_kv;
  s.D = c->head_dim;
  s.B = c->block_size;
  s.g = c->num_heads_q / c->num_heads_kv;
  s.dtype = c->dtype;
  s.scale = (float)(1.0 / std::sqrt((double)c->head_dim));
  return s;
}

size_t workspace_of(const ShapeInfo& s, const rbkv_step_tables* t, int32_t prefix_len, int sms) {
  if (step_fast_supported(s)) return step_workspace(s, t->max_tokens, sms, nullptr, nullptr);
  const int splits = step_generic_splits(s, t->max_tokens, t->max_blocks, prefix_len, sms);
  return step_generic_workspace(s, t->max_tokens, splits);
}

}  // namespace

extern "C" {

int64_t rbkv_step_plan_ints(int32_t num_seqs, int32_t max_tokens) {
  if (num_seqs < 1 || max_tokens < 1) return 0;
  return step_plan_ints(num_seqs, max_tokens);
}

rbkv_status rbkv_step_build(const rbkv_config* cfg, const rbkv_step_tables* t,
                            const int32_t* seen, const int32_t* n_new,
                            const int32_t* table_in, const int32_t* free_in,
                            rbkv_stream stream) {
  NvtxRange nvtx_range("rbkv_step_build");
  rbkv_status st = check_tables(cfg, t);
  if (st != RBKV_OK) return st;
  if (!seen || !n_new) return invalid("seen and n_new must not be NULL");
  if (!aligned(seen, 4) || !aligned(n_new, 4) || !aligned(table_in, 4) || !aligned(free_in, 4))
    return invalid("arrays must be 4-byte aligned");
  BuildArgs a = build_args(cfg, t);
  a.seen = seen;
  a.n_new = n_new;
  if (table_in) a.table_in = table_in;
  if (free_in) a.free_in = free_in;
  const int64_t S = t->num_seqs, pool = cfg->num_blocks;
  if (written_by_build(t, cfg->num_blocks, seen, S, t->ctx) ||
      written_by_build(t, cfg->num_blocks, n_new, S, nullptr) ||
      written_by_build(t, cfg->num_blocks, a.table_in, S * t->max_blocks, t->block_table) ||
      written_by_build(t, cfg->num_blocks, a.free_in, (pool + 31) / 32, t->free_words))
    return invalid("an input overlaps an array that the step writes");
  if (seen == t->ctx && a.table_in != a.table)
    return invalid("seen may be the tables' ctx only when the block table is built in place");
  cudaError_t e = launch_step_build(a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "step build launch");
  note_launches(1);
  return RBKV_OK;
}

rbkv_status rbkv_step_release(const rbkv_config* cfg, const rbkv_step_tables* t,
                              const int32_t* done, rbkv_stream stream) {
  NvtxRange nvtx_range("rbkv_step_release");
  rbkv_status st = check_tables(cfg, t);
  if (st != RBKV_OK) return st;
  if (!done || !aligned(done, 4)) return invalid("done must be a 4-byte aligned array");
  const int64_t S = t->num_seqs;
  if (overlap(done, 4 * S, t->ctx, 4 * S) || overlap(done, 4 * S, t->status, 16) ||
      overlap(done, 4 * S, t->free_words, 4 * (((int64_t)cfg->num_blocks + 31) / 32)))
    return invalid("done overlaps an array that the release writes");
  cudaError_t e = launch_step_release(build_args(cfg, t), done, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "step release launch");
  note_launches(1);
  return RBKV_OK;
}

rbkv_status rbkv_step_append(const rbkv_config* cfg, const rbkv_step_tables* t,
                             const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                             rbkv_stream stream) {
  NvtxRange nvtx_range("rbkv_step_append");
  rbkv_status st = check_tables(cfg, t);
  if (st != RBKV_OK) return st;
  if (!k_new || !v_new || !k_cache || !v_cache) return invalid("NULL tensor");
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16))
    return invalid("tensors must be 16-byte aligned");
  const ShapeInfo s = shape(cfg);
  const int64_t vec = (int64_t)s.D * (s.dtype == RBKV_BF16 ? 2 : 4) / 16;
  if (2 * (int64_t)t->max_tokens * s.H_kv * vec >= (int64_t)1 << 31)
    return fail(RBKV_ERR_UNSUPPORTED, "max_tokens too large for one append");
  DevPass dp = {};
  dp.status = t->status;
  dp.slot = t->slot;
  dp.num_tokens = t->max_tokens;
  dp.num_blocks = cfg->num_blocks;
  dp.counts = t->plan + kPlanRows;
  dp.built_for[0] = t->plan + kPlanBlock;
  dp.built_for[1] = t->plan + kPlanTokens;
  cudaError_t e = launch_kv_append(dp, s, k_new, v_new, k_cache, v_cache, (cudaStream_t)stream,
                                   true);
  if (e != cudaSuccess) return cuda_fail(e, "step append launch");
  note_launches(1);
  return RBKV_OK;
}

size_t rbkv_step_workspace_bytes(const rbkv_config* cfg, const rbkv_step_tables* t,
                                 int32_t prefix_len) {
  if (check_tables(cfg, t) != RBKV_OK || prefix_len < 0 || prefix_len > 1 << 30) return 0;
  const ShapeInfo s = shape(cfg);
  int sms = 0;
  if (num_sms(&sms) != cudaSuccess) return 0;
  return workspace_of(s, t, prefix_len, sms);
}

rbkv_status rbkv_step_attention(const rbkv_config* cfg, const rbkv_step_tables* t, const void* q,
                                const void* k_cache, const void* v_cache,
                                const int32_t* prefix_table, int32_t prefix_len, void* o,
                                void* workspace, size_t workspace_bytes, rbkv_stream stream) {
  NvtxRange nvtx_range("rbkv_step_attention");
  rbkv_status st = check_tables(cfg, t);
  if (st != RBKV_OK) return st;
  if (!q || !k_cache || !v_cache || !o) return invalid("NULL tensor");
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16))
    return invalid("tensors must be 16-byte aligned");
  if (q == o) return invalid("o must not be q");
  if (prefix_len < 0 || prefix_len > 1 << 30)
    return invalid("prefix_len must be in [0, 2^30]");
  if (prefix_len > 0 && (!prefix_table || !aligned(prefix_table, 4)))
    return invalid("a prefix needs a 4-byte aligned block list");
  if (!aligned(workspace, 256)) return invalid("workspace must be 256-byte aligned");
  DevStep ds = {};
  ds.num_seqs = t->num_seqs;
  ds.max_blocks = t->max_blocks;
  ds.max_tokens = t->max_tokens;
  ds.num_blocks = cfg->num_blocks;
  ds.block_table = t->block_table;
  ds.q_start = t->q_start;
  ds.ctx = t->ctx;
  ds.plan = t->plan;
  ds.status = t->status;
  ds.prefix_table = prefix_table;
  ds.prefix_len = prefix_len;
  const ShapeInfo s = shape(cfg);
  const cudaStream_t cs = (cudaStream_t)stream;
  int sms = 0;
  cudaError_t e = num_sms(&sms);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const size_t need = workspace_of(s, t, prefix_len, sms);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(RBKV_ERR_WORKSPACE, "workspace missing or too small");
  const int64_t q_bytes =
      (int64_t)t->max_tokens * s.H_q * s.D * (s.dtype == RBKV_BF16 ? 2 : 4);
  if (overlap(q, q_bytes, o, q_bytes)) return invalid("o overlaps q");
  if (need > 0 && (overlap(workspace, (int64_t)need, q, q_bytes) ||
                   overlap(workspace, (int64_t)need, o, q_bytes)))
    return invalid("workspace overlaps q or o");
  if (!step_fast_supported(s)) {
    const int splits = step_generic_splits(s, t->max_tokens, t->max_blocks, prefix_len, sms);
    e = launch_step_generic(ds, s, q, k_cache, v_cache, o, workspace, splits, sms, cs);
    if (e == cudaSuccess) note_launches(splits > 1 ? 2 : 1);
  } else {
    StepWorkspace w;
    step_workspace(s, t->max_tokens, sms, workspace, &w);
    // a step of at most 16 packed rows has no work for the tile kernel
    const bool tiles = !step_prefix_streamed(t->max_tokens, s.g);
    if (tiles) e = launch_step_tile(ds, s, w, q, k_cache, v_cache, o, cs);
    if (e == cudaSuccess)
      e = launch_step_stream(ds, s, w, q, k_cache, v_cache, o, !tiles, cs);
    if (e == cudaSuccess) e = launch_step_combine(ds, s, w, o, cs);
    if (e == cudaSuccess) note_launches(tiles ? 3 : 2);
  }
  if (e != cudaSuccess) return cuda_fail(e, "step attention launch");
  return RBKV_OK;
}

rbkv_status rbkv_step_device_status(const rbkv_step_tables* t, rbkv_stream stream) {
  if (!t || !t->status) return invalid("tables or its status is NULL");
  return read_status_words(t->status, (cudaStream_t)stream);
}

}  // extern "C"
