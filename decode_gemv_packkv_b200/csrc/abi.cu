// C ABI of the PackKV decode path: argument checks, host-side counters and
// kernel launches.  Declarations and the contract of every call: include/packkv.h.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "packkv.h"

namespace {

using packkv::AttnArgs;
using packkv::EncodeArgs;
using packkv::GemvArgs;
using packkv::HeadsArgs;
using packkv::HeadsTensor;
using packkv::LengthPlan;
using packkv::PairPlan;
using packkv::RaggedAppendPlan;
using packkv::RaggedLengths;
using packkv::RaggedEncodePlan;
using packkv::RaggedPlan;
using packkv::RangePlan;
using packkv::WindowArgs;
using packkv::WindowPlan;

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

packkv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? PACKKV_OK : PACKKV_ERR_CUDA; }

constexpr uint64_t kMaxArenaBytes = 0xFFFFFFFEull * 16ull;  // offsets fit u32, 0xFFFFFFFF = invalid

packkv_status check_cache(const packkv_cache* c) {
  if (c == nullptr) return PACKKV_ERR_INVALID_ARG;
  const packkv_format& f = c->fmt;
  if (f.version != PACKKV_FORMAT_VERSION || f.block_tokens != PACKKV_BLOCK_TOKENS ||
      f.group_tokens != PACKKV_GROUP_TOKENS || f.head_dim != PACKKV_HEAD_DIM)
    return PACKKV_ERR_UNSUPPORTED;
  if (f.bits < 2 || f.bits > 4) return PACKKV_ERR_UNSUPPORTED;
  if (f.reorder_key > PACKKV_KEY_KV_SUM) return PACKKV_ERR_UNSUPPORTED;
  if (f.unit_mode > PACKKV_UNITS_WIDTH_ONLY) return PACKKV_ERR_UNSUPPORTED;
  if (c->batch < 1 || c->kv_heads < 1 || c->max_blocks < 1) return PACKKV_ERR_INVALID_ARG;
  if ((int64_t)c->batch * c->kv_heads > (1 << 24) || (int64_t)c->max_blocks > (1 << 24))
    return PACKKV_ERR_INVALID_ARG;
  if (c->n_blocks < 0 || c->n_blocks > c->max_blocks) return PACKKV_ERR_INVALID_ARG;
  if (c->tail_len < 0 || c->tail_len >= PACKKV_BLOCK_TOKENS) return PACKKV_ERR_INVALID_ARG;
  if (!aligned16(c->k_arena) || !aligned16(c->v_arena) || !aligned16(c->k_index) || !aligned16(c->v_index) ||
      !aligned16(c->k_tail) || !aligned16(c->v_tail) || !aligned16(c->ctrl))
    return PACKKV_ERR_INVALID_ARG;
  if (c->arena_bytes == 0 || (c->arena_bytes & 15u) != 0 || c->arena_bytes > kMaxArenaBytes)
    return PACKKV_ERR_INVALID_ARG;
  if ((c->seq_blocks == nullptr) != (c->seq_tail == nullptr)) return PACKKV_ERR_INVALID_ARG;
  if (c->block_table != nullptr && (reinterpret_cast<uintptr_t>(c->block_table) & 3u) != 0)
    return PACKKV_ERR_INVALID_ARG;
  if (c->seq_blocks != nullptr) {
    if (c->batch > PACKKV_RAGGED_MAX_BATCH) return PACKKV_ERR_UNSUPPORTED;
    if (c->n_blocks != 0 || c->tail_len != 0) return PACKKV_ERR_INVALID_ARG;
    for (int b = 0; b < c->batch; ++b)
      if (c->seq_blocks[b] < 0 || c->seq_blocks[b] > c->max_blocks || c->seq_tail[b] < 0 ||
          c->seq_tail[b] >= PACKKV_BLOCK_TOKENS)
        return PACKKV_ERR_INVALID_ARG;
  }
  return PACKKV_OK;
}

bool is_ragged(const packkv_cache* c) { return c->seq_blocks != nullptr; }

// Plans live in thread-local host storage: a launch copies its parameters when it is
// enqueued, so the storage is free again when the call returns.
RaggedPlan& plan_storage() {
  thread_local RaggedPlan p;
  return p;
}
RaggedEncodePlan& encode_plan_storage() {
  thread_local RaggedEncodePlan p;
  return p;
}
RaggedAppendPlan& append_plan_storage() {
  thread_local RaggedAppendPlan p;
  return p;
}

// As above for the plans of the block, head and window calls.
template <class Plan>
Plan& plan_of() {
  thread_local Plan p;
  return p;
}

// The flat item list of a ragged cache: per sequence its first item and tail; returns
// the item count and the longest sequence (tokens).
RaggedPlan& build_plan(const packkv_cache* c, long* n_items, int64_t* t_max) {
  RaggedPlan& p = plan_storage();
  long acc = 0;
  int64_t tm = 0;
  for (int b = 0; b < c->batch; ++b) {
    p.base[b] = (int32_t)acc;
    p.tail[b] = c->seq_tail[b];
    acc += (long)(c->seq_blocks[b] + (c->seq_tail[b] > 0 ? 1 : 0)) * c->kv_heads;
    const int64_t tb = (int64_t)c->seq_blocks[b] * PACKKV_BLOCK_TOKENS + c->seq_tail[b];
    tm = tb > tm ? tb : tm;
  }
  p.base[c->batch] = (int32_t)acc;
  *n_items = acc;
  *t_max = tm;
  return p;
}

// Tokens of the longest sequence (uniform: every sequence).
int64_t max_tokens(const packkv_cache* c) {
  if (!is_ragged(c)) return (int64_t)c->n_blocks * PACKKV_BLOCK_TOKENS + c->tail_len;
  int64_t tm = 0;
  for (int b = 0; b < c->batch; ++b) {
    const int64_t tb = (int64_t)c->seq_blocks[b] * PACKKV_BLOCK_TOKENS + c->seq_tail[b];
    tm = tb > tm ? tb : tm;
  }
  return tm;
}

EncodeArgs encode_args(const packkv_cache* c, const uint16_t* k, const uint16_t* v, int nb) {
  EncodeArgs a{};
  a.k = k;
  a.v = v;
  a.batch = c->batch;
  a.heads = c->kv_heads;
  a.nb = nb;
  a.n_old = c->n_blocks;
  a.max_blocks = c->max_blocks;
  a.bits = (int)c->fmt.bits;
  a.key_kind = (int)c->fmt.reorder_key;
  a.unit_mode = (int)c->fmt.unit_mode;
  a.k_index = c->k_index;
  a.v_index = c->v_index;
  a.k_arena = c->k_arena;
  a.v_arena = c->v_arena;
  a.arena_bytes = c->arena_bytes;
  a.perm = c->perm;
  a.ctrl = c->ctrl;
  a.block_table = c->block_table;
  a.ragged = false;
  return a;
}

// Query heads per kv head: 1, 2, 4 or 8 in one launch; 16, 32 or 64 (a wide group, or
// several queries per kv head, e.g. speculative decoding) in launches of 8 heads each.
bool group_ok(const packkv_cache* c, int32_t q_heads, int* group) {
  if (q_heads < 1 || q_heads % c->kv_heads != 0) return false;
  const int g = q_heads / c->kv_heads;
  *group = g;
  return g == 1 || g == 2 || g == 4 || g == 8 || g == 16 || g == 32 || g == 64;
}

constexpr int kMaxLaunchGroup = 8;  // query heads one launch serves
int launch_group(int g) { return g < kMaxLaunchGroup ? g : kMaxLaunchGroup; }

GemvArgs gemv_args(const packkv_cache* c, int group, const uint8_t* arena, const uint32_t* index,
                   const uint16_t* tail) {
  GemvArgs a{};
  a.arena = arena;
  a.index = index;
  a.tail = tail;
  a.batch = c->batch;
  a.kv_heads = c->kv_heads;
  a.group = launch_group(group);
  a.g_total = group;
  a.g_off = 0;
  a.max_blocks = c->max_blocks;
  a.n_blocks = c->n_blocks;
  a.tail_len = c->tail_len;
  a.bits = (int)c->fmt.bits;
  a.arena16 = c->arena_bytes / 16;
  a.ctrl = c->ctrl;
  a.items_per_bh = c->n_blocks + (c->tail_len > 0 ? 1 : 0);
  a.n_items = (long)c->batch * c->kv_heads * a.items_per_bh;
  a.block_table = c->block_table;
  a.ragged = is_ragged(c);
  return a;
}

// The ragged plan of a launch (nullptr for a uniform batch); sets a.n_items.
template <class A>
const RaggedPlan* launch_plan(const packkv_cache* c, A& a) {
  if (!is_ragged(c)) return nullptr;
  int64_t tm = 0;
  RaggedPlan& p = build_plan(c, &a.n_items, &tm);
  a.items_per_bh = 1;  // unused by ragged launches
  return &p;
}

int blocks_of(const packkv_cache* c, int b) { return is_ragged(c) ? c->seq_blocks[b] : c->n_blocks; }
int tail_of(const packkv_cache* c, int b) { return is_ragged(c) ? c->seq_tail[b] : c->tail_len; }

// Blocks and tail of every sequence; returns the blocks of the longest.
int fill_lengths(const packkv_cache* c, LengthPlan& p) {
  int most = 0;
  for (int b = 0; b < c->batch; ++b) {
    p.blocks[b] = blocks_of(c, b);
    p.tail[b] = (uint8_t)tail_of(c, b);
    most = p.blocks[b] > most ? p.blocks[b] : most;
  }
  return most;
}

// The permutation buffer of calls that read or move it (optional elsewhere, so
// check_cache does not look at it).
bool perm_ok(const packkv_cache* c) { return c->perm == nullptr || aligned16(c->perm); }

bool rope_ok(const packkv_rope* r) {
  return r->layout <= PACKKV_ROPE_INTERLEAVED && r->rot_dim <= PACKKV_HEAD_DIM && r->rot_dim % 2 == 0 &&
         std::isfinite(r->amplitude);
}

// Arguments of the head kernels from the call's; false: something is malformed.
bool heads_args(const packkv_rope* rope, const packkv_heads* in, HeadsArgs* a) {
  if (in == nullptr || (rope != nullptr && !rope_ok(rope))) return false;
  if (in->dtype != PACKKV_DTYPE_FP16 && in->dtype != PACKKV_DTYPE_BF16 && in->dtype != PACKKV_DTYPE_FP32) return false;
  const uintptr_t size = in->dtype == PACKKV_DTYPE_FP32 ? 4 : 2;
  if (std::isnan(in->eps)) return false;
  a->dtype = in->dtype;
  a->norm = in->eps >= 0.f;
  a->eps = a->norm ? in->eps : 0.f;
  if (!a->norm && (in->q_weight != nullptr || in->k_weight != nullptr)) return false;
  if (rope != nullptr) a->rope = *rope;  // else rot_dim 0: nothing turns
  const packkv_rows* rows[3] = {&in->q, &in->k, &in->v};
  const float* weight[3] = {in->q_weight, in->k_weight, nullptr};
  for (int i = 0; i < 3; ++i) {
    const int heads = i == 0 ? in->q_heads : in->kv_heads;
    if (reinterpret_cast<uintptr_t>(rows[i]->data) % size != 0 || reinterpret_cast<uintptr_t>(weight[i]) % 4 != 0)
      return false;
    if (rows[i]->data != nullptr && (heads < 1 || heads > (1 << 20))) return false;
    a->x[i] = HeadsTensor{rows[i]->data, rows[i]->batch_stride, rows[i]->token_stride, rows[i]->head_stride,
                          heads, weight[i], nullptr};
  }
  if ((in->q.data == nullptr) != (in->q_heads == 0) || (in->k.data == nullptr) != (in->v.data == nullptr)) return false;
  return in->q.data != nullptr || in->k.data != nullptr;
}

}  // namespace

extern "C" {

uint32_t packkv_abi_version(void) { return PACKKV_ABI_VERSION; }

size_t packkv_cache_struct_size(void) { return sizeof(packkv_cache); }

const char* packkv_status_string(packkv_status s) {
  switch (s) {
    case PACKKV_OK: return "ok";
    case PACKKV_ERR_INVALID_ARG: return "invalid argument";
    case PACKKV_ERR_UNSUPPORTED: return "unsupported";
    case PACKKV_ERR_CAPACITY: return "capacity exceeded";
    case PACKKV_ERR_CUDA: return "CUDA error";
    case PACKKV_ERR_DEVICE: return "device-detected error";
  }
  return "unknown status";
}

size_t packkv_record_bytes_max(uint32_t bits) {
  if (bits < 2 || bits > 4) return 0;
  return (size_t)packkv::raw_record_bytes((int)bits);
}

size_t packkv_workspace_bytes(const packkv_cache* cache, int32_t q_heads) {
  if (check_cache(cache) != PACKKV_OK) return 0;
  int g = 0;
  if (!group_ok(cache, q_heads, &g)) return 0;
  return packkv::pv_workspace_bytes(cache->batch, cache->kv_heads, launch_group(g));
}

packkv_status packkv_cache_check(const packkv_cache* cache) { return check_cache(cache); }

packkv_status packkv_cache_reset(packkv_cache* cache, void* stream) {
  const packkv_status st = check_cache(cache);
  if (st != PACKKV_OK) return st;
  const cudaError_t e = cudaMemsetAsync(cache->ctrl, 0, 4 * sizeof(uint64_t), as_stream(stream));
  if (e != cudaSuccess) return PACKKV_ERR_CUDA;
  cache->n_blocks = 0;
  cache->tail_len = 0;
  if (is_ragged(cache))
    for (int b = 0; b < cache->batch; ++b) cache->seq_blocks[b] = cache->seq_tail[b] = 0;
  return PACKKV_OK;
}

packkv_status packkv_encode_block(packkv_cache* cache, const uint16_t* k, const uint16_t* v, int32_t n_blocks,
                                  void* stream) {
  const packkv_status st = check_cache(cache);
  if (st != PACKKV_OK) return st;
  if (n_blocks < 0) return PACKKV_ERR_INVALID_ARG;
  if (!is_ragged(cache) && cache->tail_len != 0) return PACKKV_ERR_INVALID_ARG;
  if (n_blocks == 0) return PACKKV_OK;
  if (!aligned16(k) || !aligned16(v)) return PACKKV_ERR_INVALID_ARG;
  if ((int64_t)cache->batch * cache->kv_heads * n_blocks > 0x7fffffffLL) return PACKKV_ERR_INVALID_ARG;
  if (!is_ragged(cache)) {
    if ((int64_t)cache->n_blocks + n_blocks > cache->max_blocks) return PACKKV_ERR_CAPACITY;
    const cudaError_t e = packkv::launch_encode(encode_args(cache, k, v, n_blocks), nullptr, as_stream(stream));
    if (e != cudaSuccess) return PACKKV_ERR_CUDA;
    cache->n_blocks += n_blocks;
    return PACKKV_OK;
  }
  for (int b = 0; b < cache->batch; ++b) {
    if (cache->seq_tail[b] != 0) return PACKKV_ERR_INVALID_ARG;
    if ((int64_t)cache->seq_blocks[b] + n_blocks > cache->max_blocks) return PACKKV_ERR_CAPACITY;
  }
  RaggedEncodePlan& plan = encode_plan_storage();
  for (int b = 0; b < cache->batch; ++b) {
    plan.seq[b] = b;
    plan.first_block[b] = cache->seq_blocks[b];
  }
  EncodeArgs a = encode_args(cache, k, v, n_blocks);
  a.ragged = true;
  const cudaError_t e = packkv::launch_encode(a, &plan, as_stream(stream));
  if (e != cudaSuccess) return PACKKV_ERR_CUDA;
  for (int b = 0; b < cache->batch; ++b) cache->seq_blocks[b] += n_blocks;
  return PACKKV_OK;
}

// One token for the sequences with active[b] (all if active is NULL) of a ragged cache.
packkv_status append_ragged(packkv_cache* cache, const uint16_t* k, const uint16_t* v, const uint8_t* active,
                            cudaStream_t stream) {
  RaggedAppendPlan& ap = append_plan_storage();
  RaggedEncodePlan& ep = encode_plan_storage();
  int n_done = 0;
  for (int b = 0; b < cache->batch; ++b) {
    const bool on = active == nullptr || active[b] != 0;
    ap.pos[b] = on ? cache->seq_tail[b] : -1;
    if (on && cache->seq_tail[b] + 1 == PACKKV_BLOCK_TOKENS) {
      if (cache->seq_blocks[b] >= cache->max_blocks) return PACKKV_ERR_CAPACITY;
      ep.seq[n_done] = b;
      ep.first_block[n_done] = cache->seq_blocks[b];
      ++n_done;
    }
  }
  cudaError_t e = packkv::launch_append_ragged(k, v, cache->k_tail, cache->v_tail, cache->batch, cache->kv_heads,
                                               ap, stream);
  if (e != cudaSuccess) return PACKKV_ERR_CUDA;
  if (n_done > 0) {
    EncodeArgs a = encode_args(cache, cache->k_tail, cache->v_tail, 1);
    a.batch = n_done;
    a.ragged = true;
    e = packkv::launch_encode(a, &ep, stream);
    if (e != cudaSuccess) return PACKKV_ERR_CUDA;
  }
  for (int b = 0; b < cache->batch; ++b) {
    if (ap.pos[b] < 0) continue;
    if (cache->seq_tail[b] + 1 == PACKKV_BLOCK_TOKENS) {
      cache->seq_blocks[b] += 1;
      cache->seq_tail[b] = 0;
    } else {
      cache->seq_tail[b] += 1;
    }
  }
  return PACKKV_OK;
}

packkv_status packkv_append_token(packkv_cache* cache, const uint16_t* k, const uint16_t* v, void* stream) {
  const packkv_status st = check_cache(cache);
  if (st != PACKKV_OK) return st;
  if (!aligned16(k) || !aligned16(v)) return PACKKV_ERR_INVALID_ARG;
  if (is_ragged(cache)) return append_ragged(cache, k, v, nullptr, as_stream(stream));
  const bool completes = cache->tail_len + 1 == PACKKV_BLOCK_TOKENS;
  if (completes && cache->n_blocks >= cache->max_blocks) return PACKKV_ERR_CAPACITY;
  cudaError_t e = packkv::launch_append(k, v, cache->k_tail, cache->v_tail, cache->batch * cache->kv_heads,
                                        cache->tail_len, as_stream(stream));
  if (e != cudaSuccess) return PACKKV_ERR_CUDA;
  if (!completes) {
    cache->tail_len += 1;
    return PACKKV_OK;
  }
  e = packkv::launch_encode(encode_args(cache, cache->k_tail, cache->v_tail, 1), nullptr, as_stream(stream));
  if (e != cudaSuccess) return PACKKV_ERR_CUDA;
  cache->n_blocks += 1;
  cache->tail_len = 0;
  return PACKKV_OK;
}

packkv_status packkv_append_token_masked(packkv_cache* cache, const uint16_t* k, const uint16_t* v,
                                         const uint8_t* active, void* stream) {
  const packkv_status st = check_cache(cache);
  if (st != PACKKV_OK) return st;
  if (!is_ragged(cache)) return PACKKV_ERR_UNSUPPORTED;
  if (!aligned16(k) || !aligned16(v) || active == nullptr) return PACKKV_ERR_INVALID_ARG;
  return append_ragged(cache, k, v, active, as_stream(stream));
}

packkv_status packkv_qk_gemv(const packkv_cache* cache, const uint16_t* q, int32_t q_heads, float scale,
                             float* scores, int64_t ld_scores, void* ws, size_t ws_bytes, void* stream) {
  (void)ws;
  (void)ws_bytes;
  const packkv_status st = check_cache(cache);
  if (st != PACKKV_OK) return st;
  int g = 0;
  if (q_heads < 1 || q_heads % cache->kv_heads != 0) return PACKKV_ERR_INVALID_ARG;
  if (!group_ok(cache, q_heads, &g)) return PACKKV_ERR_UNSUPPORTED;
  const int64_t T = max_tokens(cache);
  if (!aligned16(q) || !aligned16(scores) || ld_scores < T || ld_scores % 4 != 0) return PACKKV_ERR_INVALID_ARG;
  if (T == 0) return PACKKV_OK;
  GemvArgs a = gemv_args(cache, g, cache->k_arena, cache->k_index, cache->k_tail);
  const RaggedPlan* plan = launch_plan(cache, a);
  a.q = q;
  a.scores = scores;
  a.ld = ld_scores;
  a.scale = scale;
  for (a.g_off = 0; a.g_off < g; a.g_off += a.group) {
    const cudaError_t e = packkv::launch_qk(a, plan, as_stream(stream));
    if (e != cudaSuccess) return PACKKV_ERR_CUDA;
  }
  return PACKKV_OK;
}

packkv_status packkv_pv_gemv(const packkv_cache* cache, const float* p, int64_t ld_p, int32_t q_heads, float* out,
                             void* ws, size_t ws_bytes, void* stream) {
  const packkv_status st = check_cache(cache);
  if (st != PACKKV_OK) return st;
  int g = 0;
  if (q_heads < 1 || q_heads % cache->kv_heads != 0) return PACKKV_ERR_INVALID_ARG;
  if (!group_ok(cache, q_heads, &g)) return PACKKV_ERR_UNSUPPORTED;
  const int64_t T = max_tokens(cache);
  if (!aligned16(p) || !aligned16(out) || ld_p < T || ld_p % 4 != 0) return PACKKV_ERR_INVALID_ARG;
  if (T == 0) {
    const size_t bytes = (size_t)cache->batch * q_heads * PACKKV_HEAD_DIM * sizeof(float);
    return cuda_status(cudaMemsetAsync(out, 0, bytes, as_stream(stream)));
  }
  const size_t need = packkv::pv_workspace_bytes(cache->batch, cache->kv_heads, launch_group(g));
  if (!aligned16(ws) || ws_bytes < need) return PACKKV_ERR_INVALID_ARG;
  GemvArgs a = gemv_args(cache, g, cache->v_arena, cache->v_index, cache->v_tail);
  const RaggedPlan* plan = launch_plan(cache, a);
  a.p = p;
  a.ld = ld_p;
  a.out = out;
  a.partials = reinterpret_cast<float*>(ws);
  for (a.g_off = 0; a.g_off < g; a.g_off += a.group) {  // launches of one stream: ws is reused in turn
    const cudaError_t e = packkv::launch_pv(a, plan, as_stream(stream));
    if (e != cudaSuccess) return PACKKV_ERR_CUDA;
  }
  return PACKKV_OK;
}

size_t packkv_attention_workspace_bytes(const packkv_cache* cache, int32_t q_heads) {
  if (check_cache(cache) != PACKKV_OK) return 0;
  int g = 0;
  if (!group_ok(cache, q_heads, &g)) return 0;
  return packkv::attention_workspace_bytes(cache->batch, cache->kv_heads, launch_group(g));
}

packkv_status packkv_attention_decode(const packkv_cache* cache, const uint16_t* q, int32_t q_heads, float scale,
                                      float* out, void* ws, size_t ws_bytes, void* stream) {
  const packkv_status st = check_cache(cache);
  if (st != PACKKV_OK) return st;
  int g = 0;
  if (q_heads < 1 || q_heads % cache->kv_heads != 0) return PACKKV_ERR_INVALID_ARG;
  if (!group_ok(cache, q_heads, &g)) return PACKKV_ERR_UNSUPPORTED;
  const int64_t T = max_tokens(cache);
  if ((T == 0 && !is_ragged(cache)) || !aligned16(q) || !aligned16(out)) return PACKKV_ERR_INVALID_ARG;
  const size_t need = packkv::attention_workspace_bytes(cache->batch, cache->kv_heads, launch_group(g));
  if (!aligned16(ws) || ws_bytes < need) return PACKKV_ERR_INVALID_ARG;
  AttnArgs a{};
  a.k_arena = cache->k_arena;
  a.v_arena = cache->v_arena;
  a.k_index = cache->k_index;
  a.v_index = cache->v_index;
  a.k_tail = cache->k_tail;
  a.v_tail = cache->v_tail;
  a.batch = cache->batch;
  a.kv_heads = cache->kv_heads;
  a.group = launch_group(g);
  a.g_total = g;
  a.max_blocks = cache->max_blocks;
  a.n_blocks = cache->n_blocks;
  a.tail_len = cache->tail_len;
  a.bits = (int)cache->fmt.bits;
  a.arena16 = cache->arena_bytes / 16;
  a.ctrl = cache->ctrl;
  a.items_per_bh = cache->n_blocks + (cache->tail_len > 0 ? 1 : 0);
  a.n_items = (long)cache->batch * cache->kv_heads * a.items_per_bh;
  a.block_table = cache->block_table;
  a.ragged = is_ragged(cache);
  const RaggedPlan* plan = launch_plan(cache, a);
  a.q = q;
  a.scale = scale;
  a.out = out;
  a.partials = reinterpret_cast<float*>(ws);
  for (a.g_off = 0; a.g_off < g; a.g_off += a.group) {
    const cudaError_t e = packkv::launch_attention(a, plan, as_stream(stream));
    if (e != cudaSuccess) return PACKKV_ERR_CUDA;
  }
  return PACKKV_OK;
}

packkv_status packkv_rope_init(packkv_rope* rope, uint32_t rot_dim, uint32_t layout, double theta, int32_t scaling,
                               double factor, double original_tokens, double low, double high, float amplitude) {
  if (rope == nullptr || rot_dim > PACKKV_HEAD_DIM || rot_dim % 2 != 0 || layout > PACKKV_ROPE_INTERLEAVED)
    return PACKKV_ERR_INVALID_ARG;
  if (scaling < PACKKV_ROPE_SCALE_NONE || scaling > PACKKV_ROPE_SCALE_PARTS) return PACKKV_ERR_INVALID_ARG;
  if (!(theta > 1.0) || !std::isfinite(theta) || !std::isfinite(amplitude)) return PACKKV_ERR_INVALID_ARG;
  if (scaling != PACKKV_ROPE_SCALE_NONE && (!(factor > 0.0) || !std::isfinite(factor))) return PACKKV_ERR_INVALID_ARG;
  if (scaling == PACKKV_ROPE_SCALE_PARTS &&
      (!(original_tokens > 0.0) || !std::isfinite(original_tokens) || !std::isfinite(low) || !std::isfinite(high) ||
       !(high > low)))
    return PACKKV_ERR_INVALID_ARG;
  packkv_rope r{};
  r.layout = layout;
  r.rot_dim = rot_dim;
  r.amplitude = amplitude;
  const long double two_pi = 6.283185307179586476925286766559L, d = (long double)rot_dim;
  long double base = (long double)theta;
  if (scaling == PACKKV_ROPE_SCALE_BASE && rot_dim > 2) base *= powl((long double)factor, d / (d - 2.0L));
  for (uint32_t i = 0; i < rot_dim / 2; ++i) {
    long double f = powl(base, -2.0L * (long double)i / d);
    if (scaling == PACKKV_ROPE_SCALE_LINEAR) f /= (long double)factor;
    if (scaling == PACKKV_ROPE_SCALE_PARTS) {
      const long double turns = (long double)original_tokens * f / two_pi;
      long double keep = (turns - (long double)low) / ((long double)high - (long double)low);
      keep = keep < 0.0L ? 0.0L : (keep > 1.0L ? 1.0L : keep);
      f = keep * f + (1.0L - keep) * f / (long double)factor;
    }
    if (!(f > 0.0L) || f > two_pi / 2.0L) return PACKKV_ERR_INVALID_ARG;
    r.turn[i] = (uint64_t)(f / two_pi * 18446744073709551616.0L + 0.5L);  // at most 2^63
  }
  *rope = r;
  return PACKKV_OK;
}

packkv_status packkv_norm_rope(const packkv_rope* rope, const packkv_heads* in, int32_t batch, int32_t tokens,
                               const int32_t* positions, int64_t first, uint16_t* q_out, uint16_t* k_out,
                               uint16_t* v_out, void* stream) {
  HeadsArgs a{};
  if (!heads_args(rope, in, &a) || batch < 0 || tokens < 0) return PACKKV_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(positions) % 4 != 0) return PACKKV_ERR_INVALID_ARG;
  uint16_t* outs[3] = {q_out, k_out, v_out};
  for (int i = 0; i < 3; ++i) {
    if (a.x[i].data != nullptr && !aligned16(outs[i])) return PACKKV_ERR_INVALID_ARG;
    a.x[i].out = outs[i];
  }
  if ((int64_t)batch * tokens > 0x7fffffffLL) return PACKKV_ERR_INVALID_ARG;
  if (batch == 0 || tokens == 0) return PACKKV_OK;
  a.batch = batch;
  a.tokens = tokens;
  a.positions = positions;
  a.first = first;
  return cuda_status(packkv::launch_prompt_heads(a, as_stream(stream)));
}

packkv_status packkv_append_norm_rope(packkv_cache* cache, const packkv_rope* rope, const packkv_heads* in,
                                      const uint8_t* active, uint16_t* q_out, void* stream) {
  const packkv_status st = check_cache(cache);
  if (st != PACKKV_OK) return st;
  HeadsArgs a{};
  if (!heads_args(rope, in, &a) || in->k.data == nullptr || in->kv_heads != cache->kv_heads ||
      (in->q.data != nullptr && !aligned16(q_out)))
    return PACKKV_ERR_INVALID_ARG;
  if (active != nullptr && !is_ragged(cache)) return PACKKV_ERR_UNSUPPORTED;
  a.batch = cache->batch;
  a.tokens = 1;
  a.x[0].out = q_out;
  a.x[1].out = cache->k_tail;
  a.x[2].out = cache->v_tail;
  cudaStream_t s = as_stream(stream);
  if (!is_ragged(cache)) {
    const bool completes = cache->tail_len + 1 == PACKKV_BLOCK_TOKENS;
    if (completes && cache->n_blocks >= cache->max_blocks) return PACKKV_ERR_CAPACITY;
    const uint32_t held = (uint32_t)cache->n_blocks * PACKKV_BLOCK_TOKENS + (uint32_t)cache->tail_len;
    if (packkv::launch_append_heads(a, held, nullptr, s) != cudaSuccess) return PACKKV_ERR_CUDA;
    if (!completes) {
      cache->tail_len += 1;
      return PACKKV_OK;
    }
    if (packkv::launch_encode(encode_args(cache, cache->k_tail, cache->v_tail, 1), nullptr, s) != cudaSuccess)
      return PACKKV_ERR_CUDA;
    cache->n_blocks += 1;
    cache->tail_len = 0;
    return PACKKV_OK;
  }
  RaggedLengths& lp = plan_of<RaggedLengths>();
  RaggedEncodePlan& ep = encode_plan_storage();
  int n_on = 0, n_done = 0;
  for (int b = 0; b < cache->batch; ++b) {
    const bool on = active == nullptr || active[b] != 0;
    lp.tokens[b] = on ? (uint32_t)cache->seq_blocks[b] * PACKKV_BLOCK_TOKENS + (uint32_t)cache->seq_tail[b]
                      : 0xFFFFFFFFu;
    n_on += on;
    if (on && cache->seq_tail[b] + 1 == PACKKV_BLOCK_TOKENS) {
      if (cache->seq_blocks[b] >= cache->max_blocks) return PACKKV_ERR_CAPACITY;
      ep.seq[n_done] = b;
      ep.first_block[n_done] = cache->seq_blocks[b];
      ++n_done;
    }
  }
  if (n_on == 0) return PACKKV_OK;
  if (packkv::launch_append_heads(a, 0, &lp, s) != cudaSuccess) return PACKKV_ERR_CUDA;
  if (n_done > 0) {
    EncodeArgs e = encode_args(cache, cache->k_tail, cache->v_tail, 1);
    e.batch = n_done;
    e.ragged = true;
    if (packkv::launch_encode(e, &ep, s) != cudaSuccess) return PACKKV_ERR_CUDA;
  }
  for (int b = 0; b < cache->batch; ++b) {
    if (lp.tokens[b] == 0xFFFFFFFFu) continue;
    if (cache->seq_tail[b] + 1 == PACKKV_BLOCK_TOKENS) {
      cache->seq_blocks[b] += 1;
      cache->seq_tail[b] = 0;
    } else {
      cache->seq_tail[b] += 1;
    }
  }
  return PACKKV_OK;
}

size_t packkv_attention_window_workspace_bytes(const packkv_cache* cache, int32_t q_heads) {
  if (check_cache(cache) != PACKKV_OK) return 0;
  int g = 0;
  if (!group_ok(cache, q_heads, &g)) return 0;
  return packkv::window_workspace_bytes(cache->batch, cache->kv_heads, g);
}

packkv_status packkv_attention_window(const packkv_cache* cache, const uint16_t* q, int32_t q_heads, int32_t queries,
                                      int32_t window, int32_t sinks, float scale, float* out, void* ws,
                                      size_t ws_bytes, void* stream) {
  const packkv_status st = check_cache(cache);
  if (st != PACKKV_OK) return st;
  int rows = 0;
  if (q_heads < 1 || q_heads % cache->kv_heads != 0) return PACKKV_ERR_INVALID_ARG;
  if (!group_ok(cache, q_heads, &rows)) return PACKKV_ERR_UNSUPPORTED;
  if (queries < 1 || rows % queries != 0 || window < 1 || sinks < 0) return PACKKV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !perm_ok(cache)) return PACKKV_ERR_INVALID_ARG;
  if (cache->perm == nullptr && cache->fmt.reorder_key != PACKKV_KEY_IDENTITY) return PACKKV_ERR_INVALID_ARG;
  const size_t need = packkv::window_workspace_bytes(cache->batch, cache->kv_heads, rows);
  if (need > 0 && (!aligned16(ws) || ws_bytes < need)) return PACKKV_ERR_INVALID_ARG;
  WindowArgs a{};
  a.k_arena = cache->k_arena;
  a.v_arena = cache->v_arena;
  a.k_index = cache->k_index;
  a.v_index = cache->v_index;
  a.k_tail = cache->k_tail;
  a.v_tail = cache->v_tail;
  a.perm = cache->perm;
  a.block_table = cache->block_table;
  a.ctrl = cache->ctrl;
  a.arena16 = cache->arena_bytes / 16;
  a.batch = cache->batch;
  a.kv_heads = cache->kv_heads;
  a.max_blocks = cache->max_blocks;
  a.bits = (int)cache->fmt.bits;
  a.rows = rows;
  a.queries = queries;
  a.group = rows / queries;
  a.window = window;
  a.sinks = sinks;
  a.n_blocks = cache->n_blocks;
  a.tail_len = cache->tail_len;
  a.q = q;
  a.scale = scale;
  a.out = out;
  a.partials = reinterpret_cast<float*>(ws);
  if (!is_ragged(cache)) {
    if (!packkv::window_countable(a, nullptr)) return PACKKV_ERR_UNSUPPORTED;
    return cuda_status(packkv::launch_window(a, nullptr, as_stream(stream)));
  }
  WindowPlan& plan = plan_of<WindowPlan>();
  for (int b = 0; b < cache->batch; ++b) {
    plan.blocks[b] = cache->seq_blocks[b];
    plan.tail[b] = (uint8_t)cache->seq_tail[b];
  }
  if (!packkv::window_countable(a, &plan)) return PACKKV_ERR_UNSUPPORTED;
  return cuda_status(packkv::launch_window(a, &plan, as_stream(stream)));
}

packkv_status packkv_fork_sequences(packkv_cache* cache, const int32_t* src, const int32_t* dst, int32_t n,
                                    void* stream) {
  const packkv_status st = check_cache(cache);
  if (st != PACKKV_OK) return st;
  if (cache->batch > PACKKV_RAGGED_MAX_BATCH) return PACKKV_ERR_UNSUPPORTED;
  if (n < 0 || n > cache->batch || !perm_ok(cache)) return PACKKV_ERR_INVALID_ARG;
  if (n == 0) return PACKKV_OK;
  if (src == nullptr || dst == nullptr) return PACKKV_ERR_INVALID_ARG;
  uint8_t role[PACKKV_RAGGED_MAX_BATCH] = {};  // 1: a src, 2: a dst
  for (int i = 0; i < n; ++i) {
    if (src[i] < 0 || src[i] >= cache->batch || dst[i] < 0 || dst[i] >= cache->batch) return PACKKV_ERR_INVALID_ARG;
    role[src[i]] = 1;
  }
  PairPlan& plan = plan_of<PairPlan>();
  for (int i = 0; i < n; ++i) {
    if (role[dst[i]] != 0) return PACKKV_ERR_INVALID_ARG;
    role[dst[i]] = 2;
    plan.src[i] = (int16_t)src[i];
    plan.dst[i] = (int16_t)dst[i];
    plan.blocks[i] = blocks_of(cache, src[i]);
    plan.tail[i] = (uint8_t)tail_of(cache, src[i]);
  }
  if (packkv::launch_fork(*cache, plan, n, as_stream(stream)) != cudaSuccess) return PACKKV_ERR_CUDA;
  if (is_ragged(cache)) {
    for (int i = 0; i < n; ++i) {
      cache->seq_blocks[dst[i]] = cache->seq_blocks[src[i]];
      cache->seq_tail[dst[i]] = cache->seq_tail[src[i]];
    }
  }
  return PACKKV_OK;
}

packkv_status packkv_free_blocks(packkv_cache* cache, const int32_t* first, const int32_t* count, void* stream) {
  const packkv_status st = check_cache(cache);
  if (st != PACKKV_OK) return st;
  if (cache->batch > PACKKV_RAGGED_MAX_BATCH) return PACKKV_ERR_UNSUPPORTED;
  if (first == nullptr || count == nullptr) return PACKKV_ERR_INVALID_ARG;
  RangePlan& plan = plan_of<RangePlan>();
  int most = 0;
  for (int b = 0; b < cache->batch; ++b) {
    if (count[b] < 0 || (count[b] > 0 && (first[b] < 0 || (int64_t)first[b] + count[b] > blocks_of(cache, b))))
      return PACKKV_ERR_INVALID_ARG;
    plan.first[b] = count[b] > 0 ? first[b] : 0;
    plan.count[b] = count[b];
    most = count[b] > most ? count[b] : most;
  }
  if (most == 0) return PACKKV_OK;
  return cuda_status(packkv::launch_free(*cache, plan, most, as_stream(stream)));
}

size_t packkv_compact_workspace_bytes(const packkv_cache* src) {
  if (check_cache(src) != PACKKV_OK) return 0;
  const int64_t entries = (int64_t)src->batch * src->kv_heads * src->max_blocks;
  if (entries > 0x7fffffffLL) return 0;
  return packkv::compact_workspace_bytes(entries, src->arena_bytes / 16);
}

packkv_status packkv_compact(packkv_cache* dst, const packkv_cache* src, void* ws, size_t ws_bytes, void* stream) {
  packkv_status st = check_cache(src);
  if (st == PACKKV_OK) st = check_cache(dst);
  if (st != PACKKV_OK) return st;
  if (src->batch > PACKKV_RAGGED_MAX_BATCH) return PACKKV_ERR_UNSUPPORTED;
  if (std::memcmp(&dst->fmt, &src->fmt, sizeof(packkv_format)) != 0 || dst->batch != src->batch ||
      dst->kv_heads != src->kv_heads || is_ragged(dst) != is_ragged(src))
    return PACKKV_ERR_INVALID_ARG;
  if (is_ragged(src) && dst->seq_blocks == src->seq_blocks) return PACKKV_ERR_INVALID_ARG;
  if (dst->perm != nullptr && src->perm == nullptr) return PACKKV_ERR_INVALID_ARG;
  if (!perm_ok(dst) || !perm_ok(src)) return PACKKV_ERR_INVALID_ARG;
  // no buffer of dst may overlap one of src
  const uint64_t rows = (uint64_t)src->batch * src->kv_heads;
  struct Range {
    const void* at;
    uint64_t bytes;
  };
  auto ranges = [&](const packkv_cache* c, Range (&r)[8]) {
    const uint64_t index = rows * c->max_blocks * 8, tail = rows * 128 * 128 * 2;
    r[0] = {c->k_arena, c->arena_bytes};
    r[1] = {c->v_arena, c->arena_bytes};
    r[2] = {c->k_index, index};
    r[3] = {c->v_index, index};
    r[4] = {c->k_tail, tail};
    r[5] = {c->v_tail, tail};
    r[6] = {c->ctrl, 32};
    r[7] = {c->perm, c->perm != nullptr ? rows * c->max_blocks * 128 : 0};
  };
  Range rd[8], rs[8];
  ranges(dst, rd);
  ranges(src, rs);
  for (const Range& x : rd)
    for (const Range& y : rs) {
      const uintptr_t x0 = reinterpret_cast<uintptr_t>(x.at), y0 = reinterpret_cast<uintptr_t>(y.at);
      if (x.bytes != 0 && y.bytes != 0 && x0 < y0 + y.bytes && y0 < x0 + x.bytes) return PACKKV_ERR_INVALID_ARG;
    }
  LengthPlan& plan = plan_of<LengthPlan>();
  const int most = fill_lengths(src, plan);
  if (most > dst->max_blocks) return PACKKV_ERR_CAPACITY;
  const size_t need = packkv_compact_workspace_bytes(src);
  if (need == 0) return PACKKV_ERR_UNSUPPORTED;
  if (!aligned16(ws) || ws_bytes < need) return PACKKV_ERR_INVALID_ARG;
  if (packkv::launch_compact(*dst, *src, plan, most, ws, as_stream(stream)) != cudaSuccess) return PACKKV_ERR_CUDA;
  if (is_ragged(src)) {
    for (int b = 0; b < src->batch; ++b) {
      dst->seq_blocks[b] = src->seq_blocks[b];
      dst->seq_tail[b] = src->seq_tail[b];
    }
  } else {
    dst->n_blocks = src->n_blocks;
    dst->tail_len = src->tail_len;
  }
  return PACKKV_OK;
}

packkv_status packkv_get_status(const packkv_cache* cache, void* stream, uint32_t* bits_out) {
  const packkv_status st = check_cache(cache);
  if (st != PACKKV_OK) return st;
  uint64_t bits = 0;
  cudaError_t e = cudaMemcpyAsync(&bits, cache->ctrl + packkv::kCtrlStatus, sizeof(bits), cudaMemcpyDeviceToHost,
                                  as_stream(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(as_stream(stream));
  if (e != cudaSuccess) return PACKKV_ERR_CUDA;
  if (bits_out) *bits_out = (uint32_t)bits;
  if (bits == 0) return PACKKV_OK;
  e = cudaMemsetAsync(cache->ctrl + packkv::kCtrlStatus, 0, sizeof(uint64_t), as_stream(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(as_stream(stream));
  if (e != cudaSuccess) return PACKKV_ERR_CUDA;
  return (bits & PACKKV_DEV_CAPACITY) ? PACKKV_ERR_CAPACITY : PACKKV_ERR_DEVICE;
}

}  // extern "C"
