// Internal launch interface between the C ABI (abi.cu) and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "packkv.h"

namespace packkv {

// Ragged batches (sequences of their own lengths) are described to the kernels by value,
// in the launch's parameter space: per sequence b, base[b] = its first item in the flat
// (sequence, head, item) list and tail[b] = its tail tokens (items of b: base[b+1] -
// base[b] = kv_heads * (blocks + (tail > 0))).  At most kMaxRaggedBatch sequences.
constexpr int kMaxRaggedBatch = PACKKV_RAGGED_MAX_BATCH;
struct RaggedPlan {
  int32_t base[kMaxRaggedBatch + 1];
  int32_t tail[kMaxRaggedBatch];
};
// The sequences an encode call touches, in order, and the logical block each starts at.
struct RaggedEncodePlan {
  int32_t seq[kMaxRaggedBatch];
  int32_t first_block[kMaxRaggedBatch];
};
// The tail position each sequence appends at (-1: the sequence takes no token).
struct RaggedAppendPlan {
  int32_t pos[kMaxRaggedBatch];
};

struct EncodeArgs {
  const uint16_t* k;  // [batch][heads][nb*128][128] fp16
  const uint16_t* v;
  int batch, heads, nb, n_old, max_blocks, bits, key_kind;
  int unit_mode;  // PACKKV_UNITS_*: unit base = smallest code, or 0
  uint32_t* k_index;
  uint32_t* v_index;
  uint8_t* k_arena;
  uint8_t* v_arena;
  uint64_t arena_bytes;
  uint8_t* perm;  // optional
  uint64_t* ctrl;
  // ragged calls: `batch` sequences of the plan (seq[s], first_block[s]); k, v rows are
  // (seq[s] * heads + h) * nb + i; block_table (optional, device) maps logical blocks
  const int32_t* block_table;
  bool ragged;
};

cudaError_t launch_encode(const EncodeArgs& a, const RaggedEncodePlan* plan, cudaStream_t stream);
cudaError_t launch_append(const uint16_t* k, const uint16_t* v, uint16_t* k_tail, uint16_t* v_tail, int n_bh,
                          int pos, cudaStream_t stream);
// Ragged append: sequence b's token goes to tail position plan.pos[b] (none if negative).
cudaError_t launch_append_ragged(const uint16_t* k, const uint16_t* v, uint16_t* k_tail, uint16_t* v_tail,
                                 int batch, int heads, const RaggedAppendPlan& plan, cudaStream_t stream);
size_t encode_smem_bytes();

// One decode GEMV over the packed cache (q·Kᵀ or p·V).
struct GemvArgs {
  const uint8_t* arena;
  const uint32_t* index;  // [batch][kv_heads][max_blocks][2]
  const uint16_t* tail;   // [batch][kv_heads][128][128] fp16
  int batch, kv_heads, group, max_blocks, n_blocks, tail_len, bits;
  int g_total, g_off;     // query heads per kv head, and the first one this launch serves
  uint64_t arena16;       // arena_bytes / 16
  uint64_t* ctrl;
  long n_items;           // batch*kv_heads*items_per_bh
  int items_per_bh;       // n_blocks + (tail_len > 0)
  int n_warps;            // logical warps sharing the items
  const int32_t* block_table;  // optional: physical block of (sequence, logical block)
  bool ragged;            // sequences of their own lengths (RaggedPlan passed with the launch)
  // q·Kᵀ
  const uint16_t* q;      // [batch][q_heads][128]
  float* scores;          // row (b, hq) at (b*q_heads + hq) * ld
  long ld;
  float scale;
  // p·V
  const float* p;         // row (b, hq) at (b*q_heads + hq) * ld
  float* out;             // [batch][q_heads][128]
  float* partials;        // [n_warps + batch*kv_heads][group][128]
};

cudaError_t launch_qk(GemvArgs a, const RaggedPlan* plan, cudaStream_t stream);
cudaError_t launch_pv(GemvArgs a, const RaggedPlan* plan, cudaStream_t stream);

// Logical warps used by the GEMVs on the current device (an upper bound used
// for workspace sizing), and the workspace layout of p·V.
int gemv_max_warps();
size_t pv_workspace_bytes(int batch, int kv_heads, int group);
// Workspace bytes the launch of `a` by launch_pv would use (n_warps chosen as launch_pv does).
cudaError_t pv_launch_workspace_bytes(const GemvArgs& a, size_t* bytes);

// Fused decode attention over the packed cache: out = softmax(scale * q·Kᵀ) · V.
struct AttnArgs {
  const uint8_t* k_arena;
  const uint8_t* v_arena;
  const uint32_t* k_index;  // [batch][kv_heads][max_blocks][2]
  const uint32_t* v_index;
  const uint16_t* k_tail;   // [batch][kv_heads][128][128] fp16
  const uint16_t* v_tail;
  int batch, kv_heads, group, max_blocks, n_blocks, tail_len, bits;
  int g_total, g_off;       // query heads per kv head, and the first one this launch serves
  uint64_t arena16;         // arena_bytes / 16
  uint64_t* ctrl;
  long n_items;             // batch*kv_heads*items_per_bh
  int items_per_bh;         // n_blocks + (tail_len > 0)
  int n_warps;              // logical warps sharing the items
  const int32_t* block_table;  // optional: physical block of (sequence, logical block)
  bool ragged;              // sequences of their own lengths (RaggedPlan passed with the launch)
  const uint16_t* q;        // [batch][q_heads][128]
  float scale;
  float* out;               // [batch][q_heads][128]
  float* partials;          // [n_warps + batch*kv_heads][group][132]: sums [128], max, sum of exp
};

cudaError_t launch_attention(AttnArgs a, const RaggedPlan* plan, cudaStream_t stream);
size_t attention_workspace_bytes(int batch, int kv_heads, int group);

// Norm and rotation of query and key heads, values cast beside them (rope.cu).
struct HeadsTensor {
  const void* data;  // NULL: absent
  int64_t batch_stride, token_stride, head_stride;  // elements
  int heads;
  const float* weight;  // [128] or NULL
  uint16_t* out;        // [batch][heads][tokens][128]; appends: k and v tails [batch][heads][128][128]
};
struct HeadsArgs {
  HeadsTensor x[3];  // q, k, v
  int dtype;         // PACKKV_DTYPE_*
  int batch, tokens;
  int tile;          // tokens of a CTA (set by the launch)
  bool norm;
  float eps;
  const int32_t* positions;  // [batch][tokens] or NULL (first + t)
  int64_t first;
  packkv_rope rope;
};
// Tokens each sequence of a ragged batch holds (0xFFFFFFFF: it takes no token).
template <int N>
struct RaggedLengthsT {
  uint32_t tokens[N];
};
using RaggedLengths = RaggedLengthsT<kMaxRaggedBatch>;
cudaError_t launch_prompt_heads(const HeadsArgs& a, cudaStream_t stream);
// `tokens` held by every sequence, or the lengths of a ragged batch.
cudaError_t launch_append_heads(const HeadsArgs& a, uint32_t tokens, const RaggedLengths* lengths,
                                cudaStream_t stream);

// The blocks of a cache (blocks.cu).  Per-sequence arguments travel by value, like those
// above; calls of at most kSmallBatch sequences (or pairs) take plans of that size, because
// a launch copies its parameters (16 KB of them took the call from 2.3 to 3.9 us).
constexpr int kSmallBatch = 64;
template <int N>
struct PairPlanT {  // sequence dst[i] becomes src[i], which holds blocks[i] blocks and tail[i] tail tokens
  int16_t src[N], dst[N];
  int32_t blocks[N];
  uint8_t tail[N];
};
template <int N>
struct RangePlanT {  // logical blocks [first, first + count) of every sequence
  int32_t first[N], count[N];
};
template <int N>
struct LengthPlanT {  // what every sequence holds
  int32_t blocks[N];
  uint8_t tail[N];
};
using PairPlan = PairPlanT<kMaxRaggedBatch>;
using RangePlan = RangePlanT<kMaxRaggedBatch>;
using LengthPlan = LengthPlanT<kMaxRaggedBatch>;
cudaError_t launch_fork(const packkv_cache& c, const PairPlan& plan, int n, cudaStream_t stream);
cudaError_t launch_free(const packkv_cache& c, const RangePlan& plan, int most, cudaStream_t stream);
size_t compact_workspace_bytes(int64_t entries, uint64_t arena16);
// most: blocks of the longest sequence
cudaError_t launch_compact(const packkv_cache& dst, const packkv_cache& src, const LengthPlan& plan, int most, void* ws,
                           cudaStream_t stream);

// Decode attention with a sliding window and first tokens that stay visible (window.cu).
struct WindowArgs {
  const uint8_t* k_arena;
  const uint8_t* v_arena;
  const uint32_t* k_index;
  const uint32_t* v_index;
  const uint16_t* k_tail;
  const uint16_t* v_tail;
  const uint8_t* perm;      // NULL: slot = token
  const int32_t* block_table;
  uint64_t* ctrl;
  uint64_t arena16;
  int batch, kv_heads, max_blocks, bits;
  int rows;                 // query rows per kv head: queries * group
  int group, queries, window, sinks;
  int n_blocks, tail_len;   // uniform batches
  int most_items;           // items of the longest row (set by launch_window, with the next two)
  long n_items;             // items of all (row, chunk)s
  int n_parts;              // warps sharing them (the even split)
  const uint16_t* q;        // [batch][kv_heads][rows][128]
  float scale;
  float* out;
  float* partials;
};
template <int N>
struct WindowPlanT {  // ragged batches: what every sequence holds, and its rows' first item
  int32_t blocks[N];
  int32_t base[N + 1];  // items of the (row, chunk)s of the sequences before
  uint8_t tail[N];
};
using WindowPlan = WindowPlanT<kMaxRaggedBatch>;
size_t window_workspace_bytes(int batch, int kv_heads, int rows);
// Whether the items of all rows can be counted in 31 bits.
bool window_countable(const WindowArgs& a, const WindowPlan* plan);
// plan: blocks and tail of every sequence filled in (ragged batches), or NULL
cudaError_t launch_window(WindowArgs a, const WindowPlan* plan, cudaStream_t stream);

}  // namespace packkv
