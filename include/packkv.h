/*
 * packkv.h — C ABI of the PackKV decode path for NVIDIA B200 (sm_100a).
 *
 * The operations follow the PackKV paper page ("PackKV: Reducing KV Cache
 * Memory Footprint through LLM-Aware Lossy Compression"):
 *   - abstract: a KV cache compressed so that it stays compatible with its
 *     dynamic growth during decoding, and decompression fused into the
 *     matrix-vector products;
 *   - Figure 1: each query dots every K vector, softmax, weighted sum of V;
 *   - Figure 2 and the TL;DR: quantize, reorder the quantized vectors (K and V
 *     bound together), bit-pack the integer codes along the channel direction;
 *     decompression inside the matrix-vector multiply, no write-back;
 *   - Figure 5: token-wise and channel-wise quantization granularity.
 * Every parameter the pages leave open is fixed by the packed-cache format, version 1.
 *
 * Conventions for every call:
 *   - Pointers named "device" are CUDA device pointers; all must be 16-byte
 *     aligned.  fp16 data is passed as uint16_t (IEEE binary16 bits).
 *   - The library never allocates, frees or synchronises memory, except
 *     packkv_get_status, which synchronises `stream` to read the status word.
 *     The caller owns every buffer.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  All work is
 *     stream-ordered; host-side counters in packkv_cache are updated by the
 *     calls at enqueue time.
 *   - Errors found on the host are returned before anything is launched, and
 *     nothing is written.  Errors found on the device (arena full, non-finite
 *     input, corrupt index entry, a wait that gave up) set sticky bits in the
 *     cache's status word; packkv_get_status reads and clears them.  A block
 *     holding a NaN or Inf is still encoded, but its records are unspecified.
 *   - Thread safety: calls on one cache must be serialised by the caller.
 */
#ifndef PACKKV_H
#define PACKKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PACKKV_ABI_VERSION 3u
#define PACKKV_FORMAT_VERSION 1u
#define PACKKV_BLOCK_TOKENS 128
#define PACKKV_GROUP_TOKENS 32
#define PACKKV_HEAD_DIM 128
#define PACKKV_RAGGED_MAX_BATCH 2048  /* sequences of a ragged batch (see packkv_cache) */

typedef enum {
  PACKKV_OK = 0,
  PACKKV_ERR_INVALID_ARG = 1,  /* bad pointer, alignment, shape or counter */
  PACKKV_ERR_UNSUPPORTED = 2,  /* valid but not implemented (e.g. q_heads/kv_heads = 3) */
  PACKKV_ERR_CAPACITY = 3,     /* cache block table full (host) or arena full (device) */
  PACKKV_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed */
  PACKKV_ERR_DEVICE = 5        /* device-detected error other than capacity */
} packkv_status;

/* Sticky device status bits (packkv_get_status). */
#define PACKKV_DEV_CAPACITY 0x1u   /* an encode did not fit in an arena; its blocks are invalid */
#define PACKKV_DEV_NONFINITE 0x2u  /* an encoded block held a NaN or Inf */
#define PACKKV_DEV_BAD_RECORD 0x4u /* a GEMV met an invalid index entry; its outputs are NaN/skipped */
#define PACKKV_DEV_TIMEOUT 0x8u    /* a kernel's bounded wait on an async copy gave up */

/* Reorder keys (packed-cache format v1, section 2). */
#define PACKKV_KEY_IDENTITY 0u
#define PACKKV_KEY_K_SUM 1u
#define PACKKV_KEY_KV_SUM 2u

/* How the encoder sizes a pack unit (packed-cache format v1, section 3; the PackKV
 * paper page, Figure 3: quantized codes concentrate on few values).  Both give format
 * v1 units (meta byte = base | width << 4) that every decode path reads alike:
 *   FOR:        frame of reference, base = the unit's smallest code, width = bit length
 *               of (largest - smallest);
 *   WIDTH_ONLY: base = 0, width = bit length of the largest code (for the ablation). */
#define PACKKV_UNITS_FOR 0u
#define PACKKV_UNITS_WIDTH_ONLY 1u

typedef struct {
  uint32_t version;      /* PACKKV_FORMAT_VERSION */
  uint32_t bits;         /* code width: 2, 3 or 4 */
  uint32_t block_tokens; /* 128 */
  uint32_t group_tokens; /* 32 */
  uint32_t head_dim;     /* 128 */
  uint32_t reorder_key;  /* PACKKV_KEY_* */
  uint32_t unit_mode;    /* PACKKV_UNITS_*: encoder only */
} packkv_format;

/*
 * The packed cache of one attention layer: plain data, every pointer owned by
 * the caller.  Zero ctrl[0..3] and set n_blocks = tail_len = 0 before first
 * use (packkv_cache_reset does both).
 *
 * Ragged batches and paged blocks (the visualisation page, "Read the caveat":
 * paging and multi-request scheduling).  With seq_blocks and seq_tail set, each
 * sequence b has its own length: seq_blocks[b] packed blocks and seq_tail[b]
 * (0..127) tail tokens.  Both are HOST arrays of `batch` int32 that the calls
 * read and advance at enqueue time, as they do n_blocks and tail_len for a
 * uniform batch (which must then stay 0); batch <= PACKKV_RAGGED_MAX_BATCH.
 * Scores and probabilities of sequence b are its first seq_blocks[b]*128 +
 * seq_tail[b] row entries; a sequence without tokens gets zero outputs.
 * With block_table set (uniform or ragged), logical block j of sequence b is the
 * physical block p = block_table[b*max_blocks + j] (device int32), whose records
 * the index entries at (p / max_blocks, head, p % max_blocks) name: sequences may
 * share blocks (a common prompt) and need not own contiguous index rows.  The
 * blocks an encode or append call creates must map to distinct physical blocks.
 */
typedef struct {
  packkv_format fmt;
  int32_t batch;       /* sequences */
  int32_t kv_heads;    /* KV heads per sequence */
  int32_t max_blocks;  /* block-table capacity per (sequence, head) */
  int32_t n_blocks;    /* host counter: packed blocks per (sequence, head), uniform over the batch */
  int32_t tail_len;    /* host counter: tokens in the uncompressed tail, 0..127 */
  int32_t reserved0;
  uint8_t* k_arena;    /* device, arena_bytes: K records (packed-cache format v1, section 4) */
  uint8_t* v_arena;    /* device, arena_bytes: V records */
  uint64_t arena_bytes;/* capacity of EACH arena; multiple of 16, at most 2^36 */
  uint32_t* k_index;   /* device u32 [batch][kv_heads][max_blocks][2] = {offset16, length16} */
  uint32_t* v_index;   /* device, same shape */
  uint16_t* k_tail;    /* device fp16 [batch][kv_heads][128][128], arrival order */
  uint16_t* v_tail;    /* device fp16, same shape */
  uint64_t* ctrl;      /* device u64[4]: K arena end (16-B units), V arena end, status bits, scratch */
  uint8_t* perm;       /* device, optional (NULL): u8 [batch][kv_heads][max_blocks][128],
                          perm[slot] = token index within the block (at the physical block) */
  int32_t* seq_blocks; /* host, optional (NULL = uniform batch): [batch] packed blocks per sequence */
  int32_t* seq_tail;   /* host, with seq_blocks: [batch] tail tokens per sequence */
  const int32_t* block_table; /* device, optional (NULL): [batch][max_blocks] physical blocks */
} packkv_cache;

/* ABI version and sizeof(packkv_cache), for bindings to check their mirror. */
uint32_t packkv_abi_version(void);
size_t packkv_cache_struct_size(void);
const char* packkv_status_string(packkv_status s);

/* Largest record of one block for `bits` (the raw record: 528 + 2048*bits bytes).
 * Returns 0 for unsupported bits. */
size_t packkv_record_bytes_max(uint32_t bits);

/* Workspace bytes packkv_pv_gemv needs for any n_blocks <= cache->max_blocks
 * with `q_heads` query heads (split-K partials).  packkv_qk_gemv needs none. */
size_t packkv_workspace_bytes(const packkv_cache* cache, int32_t q_heads);

/* Validates the struct (host-side checks only).  Nothing is launched. */
packkv_status packkv_cache_check(const packkv_cache* cache);

/* Zeroes ctrl[0..3] on `stream` and sets n_blocks = tail_len = 0. */
packkv_status packkv_cache_reset(packkv_cache* cache, void* stream);

/*
 * Encode n_blocks full blocks per (sequence, head) and append them to the cache
 * (quantize, joint token reorder, channel-direction bit-packing: packed-cache format v1,
 * sections 1-4; paper page Figures 2 and 5).
 *   k, v: device fp16 [batch][kv_heads][n_blocks*128][128], row-major.
 * Pack units are sized as cache->fmt.unit_mode says (PACKKV_UNITS_*).
 * Records go to the arenas in ascending (sequence, head, block) order.
 * Requires tail_len == 0 and n_blocks + cache->n_blocks <= max_blocks
 * (else PACKKV_ERR_INVALID_ARG / PACKKV_ERR_CAPACITY, nothing launched).
 * On success cache->n_blocks += n_blocks.  If an arena overflows on the device,
 * PACKKV_DEV_CAPACITY is set, the arena ends do not move and every new index
 * entry is marked invalid; records that fitted may have been written into the
 * free space past the old arena end.  One pass over the input: the records'
 * arena offsets come from a decoupled look-back over the new index entries
 * (which the call clears first) and ctrl[3] counts the call's blocks.
 * n_blocks == 0 is a no-op.
 * Ragged batch: every sequence gets n_blocks blocks after its own seq_blocks[b]
 * (every seq_tail[b] must be 0); seq_blocks[b] += n_blocks.
 */
packkv_status packkv_encode_block(packkv_cache* cache, const uint16_t* k, const uint16_t* v,
                                  int32_t n_blocks, void* stream);

/*
 * Append one token per (sequence, head) to the uncompressed tail (the cache's
 * dynamic growth, paper abstract).  k, v: device fp16 [batch][kv_heads][128].
 * When the tail reaches 128 tokens it is encoded as one block (as
 * packkv_encode_block) and tail_len returns to 0.
 * PACKKV_ERR_CAPACITY if the tail is full-to-be and the block table is full.
 * Ragged batch: every sequence appends at its own seq_tail[b]; the sequences whose
 * tail completes are encoded (in ascending order) into their next block.
 */
packkv_status packkv_append_token(packkv_cache* cache, const uint16_t* k, const uint16_t* v,
                                  void* stream);

/*
 * Ragged batch only: as packkv_append_token for the sequences with active[b] != 0
 * (host uint8 [batch]); the others take no token (k, v rows of those are not read).
 * This is how sequences of one batch come to differ in length (a request that
 * joins later, or one that has finished).  PACKKV_ERR_UNSUPPORTED for a uniform
 * batch.
 */
packkv_status packkv_append_token_masked(packkv_cache* cache, const uint16_t* k, const uint16_t* v,
                                         const uint8_t* active, void* stream);

/*
 * scores[b][hq][i] = scale * sum_c q[b][hq][c] * k_hat[b][hq/G][i][c]  (fp32 accumulate)
 * over the packed blocks in storage order, then the tail in arrival order
 * (packed-cache format v1, sections 6-7; paper page Figure 1, Figure 2 fused decompression).
 *   q:      device fp16 [batch][q_heads][128]; q_heads = G * kv_heads, G in {1,2,4,8,16,32,64}.
 *           G > 8 runs as G/8 launches of 8 query heads (the cache is read G/8 times).
 *           Several queries per kv head in one step (speculative decoding) are such a
 *           group: the S queries of the G heads of kv head h are rows h*S*G .. +S*G-1.
 *   scores: device fp32, row (b, hq) starts at (b*q_heads + hq) * ld_scores;
 *           ld_scores >= T = n_blocks*128 + tail_len (ragged: the longest sequence),
 *           multiple of 4.
 *   ws, ws_bytes: unused (may be NULL / 0).
 * The decompressed K is never written to memory.  T == 0 is a no-op.
 */
packkv_status packkv_qk_gemv(const packkv_cache* cache, const uint16_t* q, int32_t q_heads,
                             float scale, float* scores, int64_t ld_scores, void* ws,
                             size_t ws_bytes, void* stream);

/*
 * out[b][hq][c] = sum_i p[b][hq][i] * v_hat[b][hq/G][i][c]  (fp32 accumulate)
 * with p in the same storage order as the scores.
 *   p:   device fp32, row (b, hq) at (b*q_heads + hq) * ld_p, ld_p >= T, multiple of 4.
 *   out: device fp32 [batch][q_heads][128].
 *   ws:  device, ws_bytes >= packkv_workspace_bytes(cache, q_heads): split-K
 *        partial sums over the sequence (no initialisation needed).  A second
 *        kernel adds them in a fixed order, so results are deterministic on a
 *        given GPU.  Two calls sharing one ws must not overlap in time.
 * With T == 0, out is set to zero.
 */
packkv_status packkv_pv_gemv(const packkv_cache* cache, const float* p, int64_t ld_p,
                             int32_t q_heads, float* out, void* ws, size_t ws_bytes, void* stream);

/*
 * p·V without a caller-provided workspace.  (The PackKV pages have no
 * counterpart: this is a calling convention, not part of the method.)
 * For callers that cannot allocate device memory: runtimes that reserve all
 * device memory at start-up and forbid later allocations, hosts without a
 * device allocator to pass in, or decode loops that must not call cudaMalloc
 * because it synchronises the device.
 * Same arguments and result as packkv_pv_gemv minus ws/ws_bytes.  The split-K
 * partials live in a static device array of PACKKV_PV_NOALLOC_SCRATCH_BYTES
 * (8 MiB) that every GPU loading the library holds until the process exits;
 * the call allocates nothing.  It needs
 *     (W + batch*kv_heads) * G * 512 bytes,
 * W = the warps it launches = min(batch*kv_heads*items per pair, resident warps
 * of the p·V kernel: SMs x CTAs per SM x 4); e.g. on a B200 with 4-bit records
 * and G = 4 (2 CTAs per SM, W = 1184 once the cache has that many items) about
 * 2900 (sequence, kv head) pairs fit.  A call that needs more returns
 * PACKKV_ERR_CAPACITY without launching anything.
 * The first call on a device looks up the array's device address (a one-time
 * set-up, cached per device).
 * The cached address belongs to the device's current context: after a
 * cudaDeviceReset in the same process this entry point must not be used again.
 * All calls share the one array, and it keeps the last call's partials: calls
 * that overlap in time on the GPU race.  Nothing in it needs clearing (every
 * partial is written before it is read).  With T == 0, out is set to zero.
 * A ragged cache, one with a block table, or G above 8: PACKKV_ERR_UNSUPPORTED.
 */
#define PACKKV_PV_NOALLOC_SCRATCH_BYTES (8u << 20)
packkv_status packkv_pv_gemv_noalloc(const packkv_cache* cache, const float* p, int64_t ld_p,
                                     int32_t q_heads, float* out, void* stream);

/*
 * Decode attention over the packed cache in one pass (paper page, Figure 1: the
 * scores, the softmax and the weighted sum of values; Figure 2: decompression
 * inside the products):
 *   out[b][hq][c] = sum_i softmax_i(scale * q[b][hq]·k_hat[b][hq/G][i]) * v_hat[b][hq/G][i][c]
 * over every packed block and the tail.  The scores and probabilities never
 * reach global memory; the softmax is computed online (a running maximum and
 * sum of exponentials per warp), split over the sequence and merged with the
 * log-sum-exp rule by a second kernel in a fixed order (deterministic).
 *   q:   device fp16 [batch][q_heads][128]; q_heads = G * kv_heads, G in {1,2,4,8,16,32,64}
 *        (as for packkv_qk_gemv).
 *   out: device fp32 [batch][q_heads][128].
 *   ws:  device, ws_bytes >= packkv_attention_workspace_bytes(cache, q_heads)
 *        (no initialisation needed; two calls sharing ws must not overlap in time).
 * T == 0 (nothing to attend to) is PACKKV_ERR_INVALID_ARG for a uniform batch; in a
 * ragged batch a sequence without tokens gets zero outputs.  A block whose K or V
 * index entry is invalid sets PACKKV_DEV_BAD_RECORD and its tokens are left out of the
 * softmax.
 */
size_t packkv_attention_workspace_bytes(const packkv_cache* cache, int32_t q_heads);
packkv_status packkv_attention_decode(const packkv_cache* cache, const uint16_t* q, int32_t q_heads,
                                      float scale, float* out, void* ws, size_t ws_bytes, void* stream);

/*
 * ---- Preparing the heads: norm and position rotation --------------------------------
 * What a decoder layer does to its query and key heads before they meet the cache
 * (the PackKV pages start behind it, at the cached K and V).  In fp32, rounded to fp16
 * once at the end:
 *   y_c  = x_c * rsqrt(mean_c x_c^2 + eps) * w_c           (if eps >= 0, else y = x)
 *   pairs (a, b) of the first rot_dim channels:
 *   (a, b) -> amplitude * (a cos t - b sin t, b cos t + a sin t),  t = position * frequency
 * Channels from rot_dim on pass unrotated (and without the amplitude).
 */
#define PACKKV_DTYPE_FP16 0
#define PACKKV_DTYPE_BF16 1
#define PACKKV_DTYPE_FP32 2

#define PACKKV_ROPE_HALF 0u         /* pair i = channels (i, i + rot_dim/2) */
#define PACKKV_ROPE_INTERLEAVED 1u  /* pair i = channels (2i, 2i + 1) */

/* How the frequencies f_i = theta^(-2i/rot_dim) are scaled for contexts longer than the
 * trained ones: LINEAR f/factor; BASE theta * factor^(rot_dim/(rot_dim-2)) in theta's
 * place (rot_dim > 2); PARTS k f + (1-k) f/factor with k = clamp((n - low)/(high - low), 0, 1)
 * and n = original_tokens * f / 2pi, the turns a pair makes within the trained length.  The
 * ramp is linear in the turns (low and high are turns, typically 1 and 32, or 1 and 4).  A
 * ramp over the pair's number between two rounded borders, or a factor per pair, is none of
 * these: fill turn[] (below) with those frequencies instead. */
#define PACKKV_ROPE_SCALE_NONE 0
#define PACKKV_ROPE_SCALE_LINEAR 1
#define PACKKV_ROPE_SCALE_BASE 2
#define PACKKV_ROPE_SCALE_PARTS 3

/* A rotation, as packkv_rope_init lays it down.  turn[i] is pair i's frequency as a
 * fraction of a turn per position, times 2^64: position * turn[i] (mod 2^64) is the
 * angle to within position * 2^-65 turns, however far the position. */
typedef struct {
  uint32_t layout;    /* PACKKV_ROPE_HALF / _INTERLEAVED */
  uint32_t rot_dim;   /* rotated channels: even, 0..128 */
  float amplitude;    /* factor on cos and sin */
  uint32_t reserved0;
  uint64_t turn[64];
} packkv_rope;

/* Fills *rope.  PACKKV_ERR_INVALID_ARG (and *rope unchanged) for an odd or too large
 * rot_dim, an unknown layout or scaling, theta <= 1, factor <= 0, a non-finite amplitude,
 * and for PARTS original_tokens <= 0 or high <= low.  Frequencies that do not lie in
 * (0, pi] per position are refused too. */
packkv_status packkv_rope_init(packkv_rope* rope, uint32_t rot_dim, uint32_t layout, double theta,
                               int32_t scaling, double factor, double original_tokens, double low,
                               double high, float amplitude);

/* Heads of 128 channels as a projection leaves them: element (b, t, h, c) of a tensor is
 * data[b*batch_stride + t*token_stride + h*head_stride + c] (strides in elements, any
 * sign; head_stride 128 and token_stride (q_heads + 2*kv_heads)*128 for one fused
 * projection).  data: device, aligned to its element; 16-byte aligned data and strides
 * take the wide loads. */
typedef struct {
  const void* data;
  int64_t batch_stride, token_stride, head_stride;
} packkv_rows;

typedef struct {
  int32_t dtype;      /* PACKKV_DTYPE_*, of q, k and v */
  int32_t q_heads;    /* 0: no q (q.data NULL) */
  int32_t kv_heads;
  float eps;          /* of the norm; negative: no norm */
  packkv_rows q, k, v;    /* k and v: both or neither (NULL data) for packkv_norm_rope */
  const float* q_weight;  /* device fp32 [128] (4-byte aligned) or NULL (ones); without a norm NULL */
  const float* k_weight;
} packkv_heads;

/*
 * Norm and rotation of q and k, v cast, from token-major rows to the layouts the cache
 * calls take: q_out, k_out, v_out device fp16 [batch][heads][tokens][128] (k_out and
 * v_out feed packkv_encode_block).  rope NULL: no rotation.  The position of token t of
 * sequence b is positions[b*tokens + t] (device int32, any order, negative ones turn
 * back) or, with positions NULL, first + t.  Values beyond the fp16 range become
 * infinities.  Outputs must not overlap the inputs.  batch or tokens 0 is a no-op.
 */
packkv_status packkv_norm_rope(const packkv_rope* rope, const packkv_heads* in, int32_t batch, int32_t tokens,
                               const int32_t* positions, int64_t first, uint16_t* q_out, uint16_t* k_out,
                               uint16_t* v_out, void* stream);

/*
 * One new token per sequence, prepared and appended in one launch: as packkv_norm_rope
 * for in's single token (token_stride is not used; in->kv_heads = cache->kv_heads), at
 * the position the cache gives it (the tokens its sequence holds before the call), with
 * k and v written to the cache's tails and q to q_out (device fp16 [batch][q_heads][128],
 * the q of the attention calls).  Then as packkv_append_token: tails that reach 128
 * tokens are encoded, the counters advance.  active (host uint8 [batch], ragged caches
 * only) selects the sequences as in packkv_append_token_masked; NULL: all.  q_out rows
 * of sequences that take no token are left as they were.
 */
packkv_status packkv_append_norm_rope(packkv_cache* cache, const packkv_rope* rope, const packkv_heads* in,
                                      const uint8_t* active, uint16_t* q_out, void* stream);

/*
 * Decode attention over the packed cache with a sliding window and first tokens that
 * stay visible.  `queries` query positions per sequence, the last ones the cache holds
 * (their k and v are appended before the call): query s of sequence b, 0 <= s < queries,
 * is at position p = T_b - queries + s and sees the tokens i with
 *   i <= p  and  (i > p - window  or  i < sinks).
 *   out[b][r][c] = sum_i softmax_i(scale * q[b][r]·k_hat[i]) * v_hat[i][c] over those i.
 *   q:   device fp16 [batch][q_heads][128]; q_heads = kv_heads * queries * G; row
 *        (h*queries + s)*G + g is query head g of kv head h at position s.
 *        queries * G in {1,2,4,8,16,32,64}.
 *   out: device fp32 [batch][q_heads][128].  A row that sees no token (or only tokens of
 *        score -inf) is zero; a row whose q holds an infinity or NaN and that sees one is NaN.
 * window >= 1 (window >= T_b: all tokens up to p), sinks >= 0.  Blocks that no query
 * sees are not read: they may have been freed.  The tokens inside a block are reordered,
 * so a block that is seen in part is masked through cache->perm, which must be set
 * unless reorder_key is PACKKV_KEY_IDENTITY (PACKKV_ERR_INVALID_ARG).  A seen block whose
 * K or V index entry is invalid or freed sets PACKKV_DEV_BAD_RECORD and its tokens are
 * left out of the softmax.  A compressed record whose contents do not fit its length sets
 * the bit too; in K its tokens are left out, in V (read behind the softmax) the outputs of
 * the rows that see it are unspecified.  More than 2^31 - 1 seen (block, query row) pairs
 * in one call are PACKKV_ERR_UNSUPPORTED.  ws as for packkv_attention_decode
 * (packkv_attention_window_workspace_bytes); results do not depend on the launch's
 * timing.
 */
size_t packkv_attention_window_workspace_bytes(const packkv_cache* cache, int32_t q_heads);
packkv_status packkv_attention_window(const packkv_cache* cache, const uint16_t* q, int32_t q_heads,
                                      int32_t queries, int32_t window, int32_t sinks, float scale, float* out,
                                      void* ws, size_t ws_bytes, void* stream);

/*
 * ---- The cache's blocks --------------------------------------------------------------
 * Records are never rewritten, so two index entries may name one record: a sequence is
 * forked by copying entries, blocks are given up by marking entries, and the room of
 * records that no entry names is taken back by copying the live ones.  Batches of more
 * than PACKKV_RAGGED_MAX_BATCH sequences are PACKKV_ERR_UNSUPPORTED in all three calls.
 */

/*
 * Sequence dst[i] becomes a copy of sequence src[i], i < n (host arrays): its first
 * blocks' index entries (at the physical blocks the block table gives dst[i], which no
 * other sequence may share), permutations, tail tokens and counters.  No record moves.
 * Every dst at most once and none of them a src, all in range (PACKKV_ERR_INVALID_ARG).
 * One src may have several dst.  What dst held is forgotten.
 */
packkv_status packkv_fork_sequences(packkv_cache* cache, const int32_t* src, const int32_t* dst, int32_t n,
                                    void* stream);

/*
 * Gives up the logical blocks first[b] .. first[b] + count[b] - 1 of every sequence b
 * (host int32 [batch]; count 0: none) for all heads: their index entries become
 * {0xFFFFFFFF, 0}.  Counters and positions stay, so a window that has moved on reads
 * as before; a call that reads a freed block treats it as an invalid entry
 * (PACKKV_DEV_BAD_RECORD).  A physical block that another sequence shares through the
 * block table is given up for it too.  0 <= first, first + count <= the sequence's
 * blocks (PACKKV_ERR_INVALID_ARG, nothing launched).  A sequence that is done: free its
 * blocks, then set its counters to 0.
 */
packkv_status packkv_free_blocks(packkv_cache* cache, const int32_t* first, const int32_t* count, void* stream);

/*
 * Copies what src's sequences hold into dst, records packed from the start of dst's
 * arenas in (sequence, head, block) order of their first entry, a record that several
 * entries name once.  dst: a cache of the same format, batch and kv_heads whose buffers
 * src does not use, with max_blocks >= src's blocks; both ragged or both uniform; a
 * block table may belong to either (dst's gives blocks that src holds apart distinct
 * physical blocks).  Freed entries stay freed; dst->perm (if set, src->perm must be)
 * and the tails up to each length are copied; dst's arena ends and counters are set.
 * The rest of dst is left as it was.  If the records do not fit dst's arenas,
 * PACKKV_DEV_CAPACITY is set in dst, its ends are 0 and every copied entry is invalid;
 * an invalid entry of src sets PACKKV_DEV_BAD_RECORD in dst and is copied as freed.
 *   ws: device, 16-byte aligned, ws_bytes >= packkv_compact_workspace_bytes(src); no
 *       initialisation needed; calls that share it must not overlap in time.
 */
size_t packkv_compact_workspace_bytes(const packkv_cache* src);
packkv_status packkv_compact(packkv_cache* dst, const packkv_cache* src, void* ws, size_t ws_bytes, void* stream);

/* Synchronises `stream`, returns PACKKV_OK if no device status bit is set,
 * else PACKKV_ERR_CAPACITY (capacity bit set) or PACKKV_ERR_DEVICE; stores
 * the bits in *bits_out (if not NULL) and clears them. */
packkv_status packkv_get_status(const packkv_cache* cache, void* stream, uint32_t* bits_out);

#ifdef __cplusplus
}
#endif

#endif /* PACKKV_H */
