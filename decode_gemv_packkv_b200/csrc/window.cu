// Decode attention over the packed cache with a sliding window and first tokens that
// stay visible (sinks), for one or several query positions per sequence.
//
//   out[r] = sum_i w_i v_i,  w = softmax over the visible i of scale * q[r]·k_i
//   query s at p = T - queries + s sees i <= p with i > p - window or i < sinks.
//
// Items of a (sequence, kv head) row: the blocks that hold first tokens, the blocks from
// the first query's window on, and the tail in pieces of 32 tokens.  A block that every
// query sees whole needs no mask; any other is masked slot by slot through the block's
// permutation.  Records go through the int8 tensor-core decode of the other products
// (decode.cuh), with four digits; the running maximum and sum of the softmax and the value
// sums are fp32, and neither scores nor probabilities reach global memory.
//
// Bound: latencies.  16 x 32 heads over 33 blocks of 3 bits (226 MB) take 56 us, 4.0 TB/s,
// 0.62 of a plain copy's rate, with issue slots 55 %, DRAM 53 % and the tensor pipe 33 % busy:
// an item is 1690 instructions of a warp in a row, between which it waits for its one stage
// (K, then V) and for its own products, and sixteen warps per SM do not cover that.
// Compressed records take about four times the instructions.  For few rows it is the latency
// of one item: 8 kv heads x 4 rows over 512 tokens take 6.8 us.
// A kernel with one CTA per record, its codes unpacked for the 5th-generation tensor cores,
// was slower in both: every item became a chain of barriers, products and tensor-memory
// reads (114 and 9.8 us).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstring>
#include <type_traits>

#include "decode.cuh"

namespace packkv {

namespace {

namespace cg = cooperative_groups;

constexpr int kWinWarps = 4;
constexpr int kTailPiece = 32;
constexpr int kMaxRanks = 8;  // CTAs of a cluster
constexpr float kWinLog2e = 1.4426950408889634f;
constexpr float kMinusInf = -__builtin_huge_valf();
// Four digits of q' and p' (decode.cuh): over a long window the values average out, and
// three digits' score error (2^-22 of the largest q') showed as 1.7e-5 of the output.
constexpr int kWinDigits = 4;
constexpr int kPartFloats = 132;  // per (slot, query row) of the workspace: 128 sums, maximum, sum of exp, pad

// The items of a row that holds nb blocks and tl tail tokens.
struct ItemList {
  int front;  // blocks [0, front) hold first tokens
  int from;   // then blocks [from, nb)
  int nb, tl;
  int n;      // items in all
};

__host__ __device__ inline ItemList item_list(int queries, int window, int sinks, int nb, int tl) {
  ItemList x;
  x.nb = nb;
  x.tl = tl;
  const long long first = (long long)nb * 128 + tl - queries - (long long)window + 1;  // oldest token a window holds
  const long long s = ((long long)sinks + 127) / 128;
  x.front = (int)(s < nb ? s : nb);
  x.from = first > 0 ? (int)(first / 128) : 0;
  if (x.from < x.front) x.from = x.front;
  if (x.from > nb) x.from = nb;
  x.n = x.front + (nb - x.from) + (tl + kTailPiece - 1) / kTailPiece;
  return x;
}

// The four parameters of this lane (channels or slots 4*lane ..) at `at` of a record.
__device__ __forceinline__ float4 param4(const unsigned char* st, int at, int lane) {
  const uint2 v = *reinterpret_cast<const uint2*>(st + at + 8 * lane);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
  return make_float4(x.x, x.y, y.x, y.y);
}

template <class Plan>
constexpr bool kRagged = !std::is_same<Plan, NoPlan>::value;

// A place in the list of all items: (sequence, kv head, chunk of query rows), item.
struct ItemCursor {
  int b, h, chunk, i;
  ItemList items;  // of the sequence

  // Index of this (row, chunk): row of q and out / G, workspace slot.
  __device__ long row(const WindowArgs& a, int chunks) const { return ((long)b * a.kv_heads + h) * chunks + chunk; }
  __device__ int block() const { return i < items.front ? i : items.from + (i - items.front); }  // >= nb: a piece of the tail
};

__device__ __forceinline__ ItemList row_list(const WindowArgs& a, const NoPlan&, int) {
  return item_list(a.queries, a.window, a.sinks, a.n_blocks, a.tail_len);
}
template <int N>
__device__ __forceinline__ ItemList row_list(const WindowArgs& a, const WindowPlanT<N>& p, int b) {
  return item_list(a.queries, a.window, a.sinks, p.blocks[b], p.tail[b]);
}

// The cursor at item x of the whole list.
template <class Plan>
__device__ __forceinline__ ItemCursor item_at(const WindowArgs& a, const Plan& p, int chunks, long x) {
  ItemCursor c;
  const int rpc = a.kv_heads * chunks;  // (row, chunk)s of a sequence
  if constexpr (kRagged<Plan>) {
    int lo = 0, hi = a.batch;  // the last sequence whose first item is <= x has items
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.base[mid] <= x) lo = mid; else hi = mid;
    }
    c.b = lo;
    x -= p.base[lo];
    c.items = row_list(a, p, lo);
  } else {
    c.items = row_list(a, p, 0);
    const long per = (long)rpc * c.items.n;
    c.b = (int)(x / per);
    x -= c.b * per;
  }
  const int r = (int)(x / c.items.n);
  c.i = (int)(x - (long)r * c.items.n);
  c.h = r / chunks;
  c.chunk = r - c.h * chunks;
  return c;
}
template <class Plan>
__device__ __forceinline__ void item_next(const WindowArgs& a, const Plan& p, int chunks, ItemCursor& c) {
  if (++c.i < c.items.n) return;
  c.i = 0;
  if (++c.chunk < chunks) return;
  c.chunk = 0;
  if (++c.h < a.kv_heads) return;
  c.h = 0;
  ++c.b;
  if constexpr (kRagged<Plan>) {  // the next sequence that has items
    while (c.b < a.batch && p.base[c.b + 1] == p.base[c.b]) ++c.b;
    if (c.b < a.batch) c.items = row_list(a, p, c.b);
  }
}

// Where the index entry and the permutation of a row's logical block j are (-1: the block
// table names no block).
__device__ __forceinline__ long entry_of(const WindowArgs& a, int b, int h, int j) {
  if (a.block_table == nullptr) return ((long)b * a.kv_heads + h) * a.max_blocks + j;
  const int p = a.block_table[(size_t)b * a.max_blocks + j];
  if (p < 0 || (long)p >= (long)a.batch * a.max_blocks) return -1;
  return ((long)(p / a.max_blocks) * a.kv_heads + h) * a.max_blocks + p % a.max_blocks;
}

// {kind, checked} of an index entry.
template <int BITS>
__device__ __forceinline__ int entry_kind(const WindowArgs& a, uint2 e) {
  constexpr uint32_t raw = (uint32_t)raw_record_bytes(BITS);
  const bool valid = e.x != 0xFFFFFFFFu && e.y >= 1040 / 16 && e.y <= raw / 16 && (uint64_t)e.x + e.y <= a.arena16;
  return !valid ? kKindInvalid : (e.y == raw / 16 ? kKindRaw : kKindPacked);
}

// What a query row sees of the 128 (or fewer) tokens from pos0 on, as bounds on the offset
// r from pos0: lo < r <= hi, or r < first.
struct Seen {
  int lo, hi, first;
  __device__ bool operator()(int r) const { return r <= hi && (r > lo || r < first); }
};
__device__ __forceinline__ int clamp_offset(long long x) { return (int)(x < -1 ? -1 : (x > 128 ? 128 : x)); }
__device__ __forceinline__ Seen seen_of(long long p, long long pos0, int window, int sinks) {
  return {clamp_offset(p - window - pos0), clamp_offset(p - pos0), clamp_offset(sinks - pos0)};
}

// Blocks that every query of a row sees whole: from <= j <= to, or j <= sink with j <= to.
struct WholeBlocks {
  int from, to, sink;
  __device__ bool operator()(int j) const { return j <= to && (j >= from || j <= sink); }
};
__device__ __forceinline__ WholeBlocks whole_blocks(const WindowArgs& a, const ItemList& x) {
  const long long T = (long long)x.nb * 128 + x.tl, p0 = T - a.queries;
  const long long lo = T - 1 - a.window;  // the last query sees from lo + 1 on
  WholeBlocks w;
  w.from = lo < 0 ? 0 : (int)(lo / 128 + 1);
  w.to = p0 < 127 ? -1 : (int)((p0 - 127) / 128);  // 128 j + 127 <= p0
  w.sink = a.sinks / 128 - 1;
  return w;
}

// Two fp16 of a query, infinities made NaN: the digits cannot carry an infinity, and scores
// of -inf alone would look like a row that sees nothing; a NaN reaches every score (through
// the records' min term, through the tail's products).
__device__ __forceinline__ uint32_t inf_to_nan(uint32_t w) {
  return w | ((((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u) >> 6);  // exponent all ones: the top mantissa bit
}

// Scores of a staged K record into sc; false: the record failed its checks.
template <int BITS, int G>
__device__ __forceinline__ bool record_scores(unsigned char* st, int kind_len, uint32_t* tab, const float (&qr)[G][4],
                                              float* sc, float scale, int lane) {
  constexpr int NT = I8Layout<G>::kNT;
  const float4 mn = param4(st, kParamOffset, lane), sl = param4(st, kParamOffset + 256, lane);
  float cst[G], qv[G][4], invf[G];
#pragma unroll
  for (int hd = 0; hd < G; ++hd) {
    cst[hd] = warp_sum(fmaf(qr[hd][3], mn.w, fmaf(qr[hd][2], mn.z, fmaf(qr[hd][1], mn.y, qr[hd][0] * mn.x))));
    qv[hd][0] = qr[hd][0] * sl.x;
    qv[hd][1] = qr[hd][1] * sl.y;
    qv[hd][2] = qr[hd][2] * sl.z;
    qv[hd][3] = qr[hd][3] * sl.w;
  }
  build_i8tab<G, NT, kWinDigits>(tab, qv, invf, lane);
  __syncwarp();
  if ((kind_len & 0xFF) == kKindRaw) {
    qk_i8<BITS, G, kWinDigits>(st, tab, cst, invf, sc, 128, scale, lane);
    return true;
  }
  return qk_packed_tc<BITS, G, kWinDigits>(st, (uint32_t)(kind_len >> 8) * 16u, tab, qv, cst, invf, sc, 128, scale, lane);
}

// Adds the staged V record's values weighted by pr (slots 4*lane + i) into the accumulators
// (raw) or the channel sums (compressed) and the min terms; false: failed its checks.
template <int BITS, int G>
__device__ __forceinline__ bool record_values(unsigned char* st, int kind_len, uint32_t* tab, const float (&pr)[G][4],
                                              float (&acc_lo)[I8Layout<G>::kNH][8],
                                              float (&acc_hi)[I8Layout<G>::kNH][8], float* sacc, float (&mp)[G],
                                              int lane) {
  constexpr int NT = I8Layout<G>::kNT;
  const float4 mn = param4(st, kParamOffset, lane), sl = param4(st, kParamOffset + 256, lane);
  float pv[G][4], add[G], invf[G];
#pragma unroll
  for (int hd = 0; hd < G; ++hd) {
    add[hd] = fmaf(pr[hd][3], mn.w, fmaf(pr[hd][2], mn.z, fmaf(pr[hd][1], mn.y, pr[hd][0] * mn.x)));
    pv[hd][0] = pr[hd][0] * sl.x;
    pv[hd][1] = pr[hd][1] * sl.y;
    pv[hd][2] = pr[hd][2] * sl.z;
    pv[hd][3] = pr[hd][3] * sl.w;
  }
  build_i8tab<G, NT, kWinDigits>(tab, pv, invf, lane);
  __syncwarp();
  if ((kind_len & 0xFF) == kKindRaw)
    pv_i8<BITS, G, kWinDigits>(st, tab, invf, acc_lo, acc_hi, lane);
  else if (!pv_packed_nat<BITS, G, kWinDigits>(st, (uint32_t)(kind_len >> 8) * 16u, tab, invf, sacc, lane))
    return false;
#pragma unroll
  for (int hd = 0; hd < G; ++hd) mp[hd] += add[hd];
  return true;
}

// m16n8k16, fp16 operands, fp32 accumulators.
__device__ __forceinline__ void hmma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Scaled scores of n <= 32 tail tokens into sc[head*128 + t].  The contraction's channel
// order is free: lane (g, t) takes channels 32 kk + 8t .. +7 of its token (A) and of its
// head (B) with one 16-byte load each, two k-steps per load.  Exact products, fp32 sums.
template <int G>
__device__ __forceinline__ void tail_scores32(const uint16_t* tail, const uint16_t* q, int n, float scale, float* sc,
                                              int lane) {
  const int g = lane >> 2, t = lane & 3;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 qb[4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) {
    qb[kk] = g < G ? *reinterpret_cast<const uint4*>(q + (size_t)g * 128 + 32 * kk + 8 * t) : zero;
    qb[kk] = make_uint4(inf_to_nan(qb[kk].x), inf_to_nan(qb[kk].y), inf_to_nan(qb[kk].z), inf_to_nan(qb[kk].w));
  }
#pragma unroll
  for (int tile = 0; tile < 2; ++tile) {
    if (16 * tile >= n) break;
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    const int r0 = 16 * tile + g, r1 = r0 + 8;
    uint4 x[4], y[4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      x[kk] = r0 < n ? *reinterpret_cast<const uint4*>(tail + (size_t)r0 * 128 + 32 * kk + 8 * t) : zero;
      y[kk] = r1 < n ? *reinterpret_cast<const uint4*>(tail + (size_t)r1 * 128 + 32 * kk + 8 * t) : zero;
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      hmma16816(d, x[kk].x, y[kk].x, x[kk].y, y[kk].y, qb[kk].x, qb[kk].y);
      hmma16816(d, x[kk].z, y[kk].z, x[kk].w, y[kk].w, qb[kk].z, qb[kk].w);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int head = 2 * t + (i & 1), tok = (i & 2) ? r1 : r0;
      if (head < G) sc[head * 128 + tok] = scale * d[i];
    }
  }
}

// Adds sum_t p[head][t] v[t][c] over n <= 32 tail tokens into the channel sums (p: fp32 in
// sc[head*128 + t], zero from n to 31).  p <= 1 = hi + lo/4096 with fp16 hi, lo: rows g
// of the A tile carry hi, rows g + 8 lo, so one product sums both.  Column m of n-tile j is
// channel 16m + 8x + j: lane (g, t) reads 8 channels of its tokens per half x.  With an
// infinity or NaN among the values the tokens are added one by one, those of zero weight
// (masked ones) left out, so that it does not spread.
// (On the CUDA cores, a token or four channels per lane, 16 x 32 heads over 1024 tokens with
// a tail of 118 took 39.0 us, this way 29.2.)
template <int G>
__device__ __forceinline__ void tail_values32(const uint16_t* tail, const float* sc, int n, float* sacc, int lane) {
  const int g = lane >> 2, t = lane & 3;
  uint32_t a[2][4];  // per token tile: rows g (hi) k 2t, 2t+1 | rows g + 8 (lo) | both again for k + 8
#pragma unroll
  for (int tile = 0; tile < 2; ++tile)
#pragma unroll
    for (int kh = 0; kh < 2; ++kh) {
      const int k = 16 * tile + 2 * t + 8 * kh;
      const float p0 = g < G ? sc[g * 128 + k] : 0.f, p1 = g < G ? sc[g * 128 + k + 1] : 0.f;
      const __half2 hi = __floats2half2_rn(p0, p1);
      const float2 hf = __half22float2(hi);
      const __half2 lo = __floats2half2_rn((p0 - hf.x) * 4096.f, (p1 - hf.y) * 4096.f);
      a[tile][2 * kh] = *reinterpret_cast<const uint32_t*>(&hi);
      a[tile][2 * kh + 1] = *reinterpret_cast<const uint32_t*>(&lo);
    }
#pragma unroll 1
  for (int x = 0; x < 2; ++x) {
    uint4 v[2][4];  // tokens 2t, 2t+1, 2t+8, 2t+9 of each tile
    uint32_t ones = 0u;
#pragma unroll
    for (int tile = 0; tile < 2; ++tile)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tok = 16 * tile + 2 * t + (i & 1) + 8 * (i >> 1);
        v[tile][i] = tok < n ? *reinterpret_cast<const uint4*>(tail + (size_t)tok * 128 + 16 * g + 8 * x)
                             : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
    for (int tile = 0; tile < 2; ++tile)
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // an exponent of all ones in either half
        const uint32_t w[4] = {v[tile][i].x, v[tile][i].y, v[tile][i].z, v[tile][i].w};
#pragma unroll
        for (int y = 0; y < 4; ++y) ones |= ((w[y] & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
      }
    if (__any_sync(0xffffffffu, ones != 0u)) {  // these 64 channels (16m + 8x + j) one by one
#pragma unroll 1
      for (int hd = 0; hd < G; ++hd)
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          const int c = 16 * (lane >> 2) + 8 * x + 2 * (lane & 3) + k;
          float sum = sacc[hd * 128 + c];
          for (int tok = 0; tok < n; ++tok) {
            const float p = sc[hd * 128 + tok];
            if (p != 0.f) sum = fmaf(p, half_bits_to_float(tail[(size_t)tok * 128 + c]), sum);
          }
          sacc[hd * 128 + c] = sum;
        }
      continue;
    }
    float d[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
#pragma unroll
    for (int tile = 0; tile < 2; ++tile)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4& q4 = v[tile][i];
          w[i] = j < 2 ? q4.x : (j < 4 ? q4.y : (j < 6 ? q4.z : q4.w));
        }
        const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
        hmma16816(d[j], a[tile][0], a[tile][1], a[tile][2], a[tile][3], __byte_perm(w[0], w[1], sel),
                  __byte_perm(w[2], w[3], sel));
      }
    if (g < G) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)  // columns 2t, 2t + 1; their lo parts sit in rows g + 8
          sacc[g * 128 + 16 * (2 * t + i) + 8 * x + j] += fmaf(d[j][2 + i], 1.f / 4096.f, d[j][i]);
    }
  }
  __syncwarp();
}

// ---- the kernel --------------------------------------------------------------------
// A warp takes an item at a time.  Two ways to share the items out:
//  * even split (kEven): the items of all (row, chunk)s in one list, an equal contiguous
//    part for every warp the device holds.  A warp stages an item's K record, then its V
//    record in the same stage (half the shared memory, so more warps per SM), and at each
//    (row, chunk) border writes its sums to the workspace; window_merge_kernel joins them.
//  * a cluster per (row, chunk): its warps take the items in turn, K and V records in
//    flight together, and the sums are joined through (distributed) shared memory: one
//    launch, for calls with few items.
// Both join in a fixed order, so results do not depend on timing.
template <int BITS, int G, bool kEven>
struct WinCfg {
  using C = Cfg<BITS, G, false>;
  static constexpr int kStage = C::kStageRec;
  static constexpr int kStages = kEven ? 1 : 2;
  static constexpr int kTableBytes = (C::kI8Tab + 15) / 16 * 16;
  static constexpr int kFixed = kStages * kStage + kTableBytes + 1024 * G;
  static constexpr int kWarpSmem = (kFixed + 16 + 127) / 128 * 128;
};

// Warp-private shared memory: [K stage][V stage][table][scores][sums][2 mbarriers].
template <int BITS, int G, bool kEven>
struct WinMem {
  using W = WinCfg<BITS, G, kEven>;
  unsigned char* base;
  __device__ unsigned char* stage(int v) const { return base + (kEven ? 0 : v) * W::kStage; }
  __device__ uint32_t* table() const { return reinterpret_cast<uint32_t*>(base + W::kStages * W::kStage); }
  __device__ float* scores() const {
    return reinterpret_cast<float*>(base + W::kStages * W::kStage + W::kTableBytes);
  }
  __device__ float* sums() const { return scores() + 128 * G; }
  __device__ uint64_t* bar(int v) const { return reinterpret_cast<uint64_t*>(base + W::kFixed) + v; }
};

// Resident CTAs per SM the register budget of the even split is sized for.  Single rows, 16 x
// 32 heads, the last 4096 of 4500 tokens: four CTAs 56.7 / 59.3 / 44.3 us (4 / 3 / 2 bits),
// five (96 registers, some spilled) 61.7 / 65.6 / 45.8, six 69 / 72 / 54.  2 bits took five
// when four took 47.4, before the tail's pieces went to the tensor cores.
constexpr int win_ctas(int bits, int g, bool even) { return !even ? 0 : (g == 1 ? (bits == 2 ? 5 : 4) : (g == 2 ? 4 : 3)); }

template <int BITS, int G, bool kEven, class Plan>
__global__ void __launch_bounds__(kWinWarps * 32, win_ctas(BITS, G, kEven))
    window_kernel(const WindowArgs a, const __grid_constant__ Plan plan) {
  using W = WinCfg<BITS, G, kEven>;
  using L = I8Layout<G>;
  constexpr int NH = L::kNH;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float wmax[kWinWarps][G], wsum[kWinWarps][G], cmax[G], csum[G];  // cluster form
  if constexpr (kEven) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunks = a.rows / G;
  const WinMem<BITS, G, kEven> m{smem + warp * W::kWarpSmem};

  // this warp's items
  ItemCursor cc;
  int n_mine, step = 1, ranks = 1, rank = 0;
  const int part = blockIdx.x * kWinWarps + warp;  // of the even split
  if constexpr (kEven) {
    if (part >= a.n_parts) return;
    const long lo = (long)((long long)a.n_items * part / a.n_parts);
    n_mine = (int)((long)((long long)a.n_items * (part + 1) / a.n_parts) - lo);
    cc = item_at(a, plan, chunks, lo);
  } else {
    cg::cluster_group cluster = cg::this_cluster();
    ranks = (int)cluster.num_blocks();
    rank = (int)cluster.block_rank();
    step = ranks * kWinWarps;
    const int rc = blockIdx.x / ranks, r = rc / chunks;
    cc.chunk = rc - r * chunks;
    cc.b = r / a.kv_heads;
    cc.h = r - cc.b * a.kv_heads;
    cc.items = row_list(a, plan, cc.b);
    cc.i = warp * ranks + rank;  // neighbours in the list on different SMs
    n_mine = cc.i < cc.items.n ? (cc.items.n - cc.i + step - 1) / step : 0;
  }
  auto next = [&](ItemCursor& c) {
    if constexpr (kEven) item_next(a, plan, chunks, c);
    else c.i += step;
  };
  // lanes 0 and 1 load an item's K and V entry
  auto load_entry = [&](const ItemCursor& c) {
    uint2 e = make_uint2(0u, 0u);
    const int j = c.block();
    if (lane < 2 && j < c.items.nb) {
      const long at = entry_of(a, c.b, c.h, j);
      e = at < 0 ? make_uint2(0xFFFFFFFFu, 0u)
                 : *reinterpret_cast<const uint2*>((lane == 0 ? a.k_index : a.v_index) + at * 2);
    }
    return e;
  };
  // lane v issues its record (K: 0, V: 1)
  auto issue = [&](int v, bool tail, uint2 e) {
    if (lane == v) {
      const int kind = tail ? kKindTail : entry_kind<BITS>(a, e);
      fence_async_smem();
      if (kind == kKindRaw || kind == kKindPacked) {
        mbar_arrive_expect_tx(m.bar(v), e.y * 16u);
        bulk_g2s(m.stage(v), (v ? a.v_arena : a.k_arena) + (uint64_t)e.x * 16, e.y * 16u, m.bar(v));
      } else {
        mbar_arrive(m.bar(v));
      }
    }
    __syncwarp();
  };
  uint2 ent = make_uint2(0u, 0u);
  if (n_mine > 0) ent = load_entry(cc);
  if (lane == 0) {
    mbar_init(m.bar(0), 1);
    mbar_init(m.bar(1), 1);
    fence_mbar_init();
  }
  __syncwarp();
  if (n_mine > 0) {
    issue(0, cc.block() >= cc.items.nb, ent);
    if (!kEven) issue(1, cc.block() >= cc.items.nb, ent);
  }

  float qr[G][4], mrun[G], lrun[G], mp[G];
  float acc_lo[NH][8], acc_hi[NH][8];
#pragma unroll
  for (int hd = 0; hd < G; ++hd) {
    mrun[hd] = kMinusInf;
    lrun[hd] = 0.f;
    mp[hd] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < NH; ++j)
#pragma unroll
    for (int T8 = 0; T8 < 8; ++T8) acc_lo[j][T8] = acc_hi[j][T8] = 0.f;
  float* sacc = m.sums();
  float* sc = m.scores();
  zero_sums<G>(sacc, lane);
  __syncwarp();
  const int g = lane >> 2, t = lane & 3;
  // the tensor-core accumulators and min terms into the channel sums; l over the warp
  auto collect = [&]() {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NH; ++j) {
      float* row = sacc + L::head(j, t) * 128 + g;
#pragma unroll
      for (int T8 = 0; T8 < 8; ++T8) {
        if (L::owns(j, t)) {
          row[16 * T8] += acc_lo[j][T8];
          row[16 * T8 + 8] += acc_hi[j][T8];
        }
        acc_lo[j][T8] = acc_hi[j][T8] = 0.f;
      }
    }
    __syncwarp();
#pragma unroll
    for (int hd = 0; hd < G; ++hd) {
      const float mn = warp_sum(mp[hd]);
      lrun[hd] = warp_sum(lrun[hd]);
      float4* row = reinterpret_cast<float4*>(sacc + hd * 128) + lane;
      float4 s = *row;
      s.x += mn;
      s.y += mn;
      s.z += mn;
      s.w += mn;
      *row = s;
      mp[hd] = 0.f;
    }
  };
  bool fresh = true;  // the next item begins a (row, chunk)
  long slot = 0;      // of the current one
  const uint16_t* qrow = nullptr;
  WholeBlocks whole_of{0, -1, -1};
  uint32_t phase = 0u;
#pragma unroll 1
  for (int x = 0; x < n_mine; ++x, phase ^= 1u) {
    if (fresh) {
      fresh = false;
      slot = cc.row(a, chunks);
      qrow = a.q + (size_t)slot * G * 128;
      whole_of = whole_blocks(a, cc.items);
#pragma unroll
      for (int hd = 0; hd < G; ++hd) {
        uint2 v = *reinterpret_cast<const uint2*>(qrow + hd * 128 + 4 * lane);
        v.x = inf_to_nan(v.x);
        v.y = inf_to_nan(v.y);
        const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
        const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
        qr[hd][0] = u.x;
        qr[hd][1] = u.y;
        qr[hd][2] = w.x;
        qr[hd][3] = w.y;
      }
    }
    const int j = cc.block();
    const bool tail = j >= cc.items.nb;
    const int piece = tail ? j - cc.items.nb : 0;
    const int n_tok = tail ? min(kTailPiece, cc.items.tl - piece * kTailPiece) : 128;
    const size_t tail_at = (((size_t)cc.b * a.kv_heads + cc.h) * 128 + piece * kTailPiece) * 128;
    const bool whole = !tail && whole_of(j);
    uint32_t slots = 0x03020100u + 0x04040404u * (uint32_t)lane;  // this lane's four slots' tokens
    if (!tail && !whole && a.perm != nullptr) {
      const long at = entry_of(a, cc.b, cc.h, j);
      if (at >= 0)  // asked for now, needed behind the scores
        asm volatile("ld.global.u32 %0, [%1];" : "=r"(slots) : "l"(a.perm + at * 128 + 4 * lane));
    }
    ItemCursor nc = cc;
    next(nc);
    const uint2 ent_next = x + 1 < n_mine ? load_entry(nc) : make_uint2(0u, 0u);
    const bool tail_next = nc.block() >= nc.items.nb;
    const int len_k = (int)__shfl_sync(0xffffffffu, ent.y, 0), len_v = (int)__shfl_sync(0xffffffffu, ent.y, 1);
    const int kind_of_lane = entry_kind<BITS>(a, ent);
    const int kind_k = __shfl_sync(0xffffffffu, kind_of_lane, 0), kind_v = __shfl_sync(0xffffffffu, kind_of_lane, 1);

    // ---- scores ----
    if (!mbar_wait_bounded(m.bar(0), phase, a.ctrl)) {  // never landed (status set)
      if (!kEven) mbar_wait_bounded(m.bar(1), phase, a.ctrl);
      break;
    }
    bool ok = true;
    if (tail) {
      tail_scores32<G>(a.k_tail + tail_at, qrow, n_tok, a.scale, sc, lane);
    } else if (kind_k == kKindInvalid || kind_v == kKindInvalid) {
      ok = false;  // before the softmax: neither the sums nor the maximum know the block
    } else {
      ok = record_scores<BITS, G>(m.stage(0), kind_k | (len_k << 8), m.table(), qr, sc, a.scale, lane);
    }
    __syncwarp();
    if (kEven) issue(1, tail, ent);
    else if (x + 1 < n_mine) issue(0, tail_next, ent_next);

    // ---- masks and the running softmax ----
    float pr[G][4];
#pragma unroll
    for (int hd = 0; hd < G; ++hd) {
      const float4 s4 = *reinterpret_cast<const float4*>(sc + hd * 128 + 4 * lane);
      float sv[4] = {s4.x, s4.y, s4.z, s4.w};
      if (!ok) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sv[i] = kMinusInf;
      } else if (!whole) {
        const long long pos0 = tail ? (long long)cc.items.nb * 128 + piece * kTailPiece : (long long)j * 128;
        const long long p0 = (long long)cc.items.nb * 128 + cc.items.tl - a.queries;
        const Seen see = seen_of(p0 + (cc.chunk * G + hd) / a.group, pos0, a.window, a.sinks);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (int)((slots >> (8 * i)) & 0xFFu);
          if (!see(r) || r >= n_tok) sv[i] = kMinusInf;
        }
      }
      const float bm = warp_max(fmaxf(fmaxf(sv[0], sv[1]), fmaxf(sv[2], sv[3])));
      const float m_new = fmaxf(mrun[hd], bm);
      float ps = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pr[hd][i] = sv[i] == kMinusInf ? 0.f : exp2f((sv[i] - m_new) * kWinLog2e);
        ps += pr[hd][i];
      }
      if (m_new > mrun[hd]) {  // warp-uniform: rescale what was summed under the old maximum
        if (mrun[hd] != kMinusInf) {
          const float alpha = exp2f((mrun[hd] - m_new) * kWinLog2e);
          lrun[hd] *= alpha;
          mp[hd] *= alpha;
          float4* row = reinterpret_cast<float4*>(sacc + hd * 128) + lane;
          const float4 r4 = *row;
          *row = make_float4(r4.x * alpha, r4.y * alpha, r4.z * alpha, r4.w * alpha);
#pragma unroll
          for (int jn = 0; jn < NH; ++jn) {
            if (L::head(jn, t) == hd) {
#pragma unroll
              for (int T8 = 0; T8 < 8; ++T8) {
                acc_lo[jn][T8] *= alpha;
                acc_hi[jn][T8] *= alpha;
              }
            }
          }
        }
        mrun[hd] = m_new;
      }
      lrun[hd] += ps;  // of this lane's slots; summed over the warp by collect()
    }

    // ---- values ----
    if (!mbar_wait_bounded(m.bar(1), phase, a.ctrl)) {
      if (!kEven && x + 1 < n_mine) mbar_wait_bounded(m.bar(0), phase ^ 1u, a.ctrl);
      break;
    }
    if (tail) {
      __syncwarp();
#pragma unroll
      for (int hd = 0; hd < G; ++hd)
        *reinterpret_cast<float4*>(sc + hd * 128 + 4 * lane) = make_float4(pr[hd][0], pr[hd][1], pr[hd][2], pr[hd][3]);
      __syncwarp();
      tail_values32<G>(a.v_tail + tail_at, sc, n_tok, sacc, lane);
    } else if (ok) {
      ok = record_values<BITS, G>(m.stage(1), kind_v | (len_v << 8), m.table(), pr, acc_lo, acc_hi, sacc, mp, lane);
    }
    if (!ok && lane == 0) set_status(a.ctrl, PACKKV_DEV_BAD_RECORD);
    __syncwarp();
    if (x + 1 < n_mine) issue(kEven ? 0 : 1, tail_next, ent_next);
    cc = nc;
    ent = ent_next;
    if constexpr (kEven) {
      fresh = cc.i == 0 || x + 1 == n_mine;
      if (fresh) {  // the (row, chunk) is done here: its sums to slot part + row
        collect();
        float* out = a.partials + (size_t)(part + slot) * G * kPartFloats;
#pragma unroll
        for (int hd = 0; hd < G; ++hd) {
          __stcg(reinterpret_cast<float4*>(out + hd * kPartFloats) + lane,
                 reinterpret_cast<const float4*>(sacc + hd * 128)[lane]);
          if (lane == 0)
            __stcg(reinterpret_cast<float2*>(out + hd * kPartFloats + 128), make_float2(mrun[hd], lrun[hd]));
          mrun[hd] = kMinusInf;
          lrun[hd] = 0.f;
        }
        __syncwarp();
        zero_sums<G>(sacc, lane);
        __syncwarp();
      }
    }
  }

  if constexpr (!kEven) {
    // this warp's sums, then the CTA's, then the cluster's
    collect();
#pragma unroll
    for (int hd = 0; hd < G; ++hd) {
      if (lane == 0) {
        wmax[warp][hd] = mrun[hd];
        wsum[warp][hd] = lrun[hd];
      }
    }
    __syncthreads();
    float* cta = WinMem<BITS, G, kEven>{smem}.scores();  // [G][128], free now
    for (int o = threadIdx.x; o < G * 128; o += kWinWarps * 32) {
      const int hd = o >> 7;
      float M = wmax[0][hd];
#pragma unroll
      for (int w = 1; w < kWinWarps; ++w) M = fmaxf(M, wmax[w][hd]);
      float s = 0.f, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWinWarps; ++w) {
        const float e = wsum[w][hd] == 0.f ? 0.f : exp2f((wmax[w][hd] - M) * kWinLog2e);
        if (e != 0.f) s = fmaf(WinMem<BITS, G, kEven>{smem + w * W::kWarpSmem}.sums()[o], e, s);
        l = fmaf(wsum[w][hd], e, l);
      }
      cta[o] = s;
      if ((o & 127) == 0) {
        cmax[hd] = M;
        csum[hd] = l;
      }
    }
    cg::cluster_group cluster = cg::this_cluster();
    if (ranks > 1) cluster.sync(); else __syncthreads();
    float* orow = a.out + (size_t)(blockIdx.x / ranks) * G * 128;
    for (int o = rank * kWinWarps * 32 + threadIdx.x; o < G * 128; o += ranks * kWinWarps * 32) {
      const int hd = o >> 7;
      float mr[kMaxRanks], lr[kMaxRanks], y[kMaxRanks];  // all ranks' loads in flight
#pragma unroll
      for (int r = 0; r < kMaxRanks; ++r) {
        mr[r] = kMinusInf;
        lr[r] = y[r] = 0.f;
        if (r < ranks) {
          mr[r] = *cluster.map_shared_rank(&cmax[hd], r);
          lr[r] = *cluster.map_shared_rank(&csum[hd], r);
          y[r] = *cluster.map_shared_rank(&cta[o], r);
        }
      }
      float M = mr[0];
#pragma unroll
      for (int r = 1; r < kMaxRanks; ++r) M = fmaxf(M, mr[r]);
      float s = 0.f, l = 0.f;
#pragma unroll
      for (int r = 0; r < kMaxRanks; ++r) {
        const float e = lr[r] == 0.f ? 0.f : exp2f((mr[r] - M) * kWinLog2e);
        if (e != 0.f) s = fmaf(y[r], e, s);
        l = fmaf(lr[r], e, l);
      }
      orow[o] = l == 0.f ? 0.f : s / l;  // a row that sees nothing is zero; a NaN stays one
    }
    if (ranks > 1) cluster.sync();  // no CTA leaves while another reads its sums
  }
}

// Joins the slots of every output row with the log-sum-exp rule in a fixed order: one CTA
// of four warps per row, warp i takes slots w0 + i, w0 + i + 4, ...
template <class Plan>
__global__ void __launch_bounds__(128) window_merge_kernel(const WindowArgs a, int group, const __grid_constant__ Plan plan) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float4 wsum[4][32];
  __shared__ float2 wml[4];
  const int chunks = a.rows / group, rpc = a.kv_heads * chunks;
  const long row = blockIdx.x;  // of out
  const long bhc = row / group;
  const int hd = (int)(row - bhc * group), b = (int)(bhc / rpc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ItemList items = row_list(a, plan, b);
  float4* out = reinterpret_cast<float4*>(a.out + row * 128) + lane;
  if (items.n == 0) {  // a sequence without tokens
    if (warp == 0) *out = make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  long first;
  if constexpr (kRagged<Plan>)
    first = plan.base[b] + (bhc - (long)b * rpc) * items.n;
  else
    first = bhc * items.n;
  // warp whose range [w*N/W, (w+1)*N/W) holds an item
  auto warp_of = [&](long item) { return (long)(((long long)(item + 1) * a.n_parts + a.n_items - 1) / a.n_items) - 1; };
  const long w0 = warp_of(first), w1 = warp_of(first + items.n - 1);
  const float* base = a.partials + hd * kPartFloats;
  const size_t stride = (size_t)group * kPartFloats;
  float M = kMinusInf, l = 0.f;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (long w = w0 + warp; w <= w1; w += 4) {
    const float* p = base + (w + bhc) * stride;
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(p + 128));
    const float4 y = __ldcg(reinterpret_cast<const float4*>(p) + lane);
    const float m = fmaxf(M, ml.x);
    const float eo = M == kMinusInf ? 0.f : exp2f((M - m) * kWinLog2e);
    const float en = ml.y == 0.f ? 0.f : exp2f((ml.x - m) * kWinLog2e);  // 0 sum: nothing was seen
    if (en != 0.f) {
      s.x = fmaf(y.x, en, s.x * eo);
      s.y = fmaf(y.y, en, s.y * eo);
      s.z = fmaf(y.z, en, s.z * eo);
      s.w = fmaf(y.w, en, s.w * eo);
      l = fmaf(ml.y, en, l * eo);
      M = m;
    } else if (ml.y != ml.y) {
      l = ml.y;
    }
  }
  wsum[warp][lane] = s;
  if (lane == 0) wml[warp] = make_float2(M, l);
  __syncthreads();
  if (warp != 0) return;
  float top = kMinusInf;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = fmaxf(top, wml[i].x);
  float L = 0.f;
  s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 ml = wml[i];
    const float e = ml.y == 0.f ? 0.f : exp2f((ml.x - top) * kWinLog2e);
    const float4 y = wsum[i][lane];
    if (e != 0.f) {
      s.x = fmaf(y.x, e, s.x);
      s.y = fmaf(y.y, e, s.y);
      s.z = fmaf(y.z, e, s.z);
      s.w = fmaf(y.w, e, s.w);
    }
    L = fmaf(ml.y, e, L);
  }
  *out = L == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(s.x / L, s.y / L, s.z / L, s.w / L);
}

struct WinKernel {
  const void* fn;
  int smem;
  std::atomic<int>* ctas;  // [kMaxDevices]: CTAs of the kernel a device holds (0: not asked yet)
};

constexpr int kMaxDevices = 64;

template <int BITS, int G, bool kEven, class Plan>
WinKernel win_kernel() {
  static std::atomic<int> ctas[kMaxDevices];
  return {reinterpret_cast<const void*>(&window_kernel<BITS, G, kEven, Plan>),
          kWinWarps * WinCfg<BITS, G, kEven>::kWarpSmem, ctas};
}

// bits 2..4, g 1, 2 or 4.
template <class Plan>
WinKernel win_select(int bits, int g, bool even) {
#define PACKKV_WCASE(B, GG) \
  if (bits == B && g == GG) return even ? win_kernel<B, GG, true, Plan>() : win_kernel<B, GG, false, Plan>();
  PACKKV_WCASE(4, 1) PACKKV_WCASE(4, 2) PACKKV_WCASE(4, 4)
  PACKKV_WCASE(3, 1) PACKKV_WCASE(3, 2) PACKKV_WCASE(3, 4)
  PACKKV_WCASE(2, 1) PACKKV_WCASE(2, 2)
#undef PACKKV_WCASE
  return even ? win_kernel<2, 4, true, Plan>() : win_kernel<2, 4, false, Plan>();
}

// CTAs of the kernel that the current device holds; raises its shared memory limit there
// the first time.
cudaError_t win_configure(const WinKernel& k, int dev, int* ctas) {
  if (dev < kMaxDevices && (*ctas = k.ctas[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  int sms = 0, per_sm = 0;
  cudaError_t e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k.fn, kWinWarps * 32, (size_t)k.smem);
  if (e != cudaSuccess) return e;
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  *ctas = sms * per_sm;
  if (dev < kMaxDevices) k.ctas[dev].store(*ctas, std::memory_order_relaxed);
  return cudaSuccess;
}

// Warps that an even split may have (workspace slots): at most 32 per SM.
int max_parts() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms * 32;
}

template <class Plan>
cudaError_t even_split(WindowArgs a, const Plan& plan, int g, const WinKernel& k, int warps, cudaStream_t stream) {
  a.n_parts = warps < max_parts() ? warps : max_parts();
  if (a.n_items < a.n_parts) a.n_parts = (int)a.n_items;
  void* args[] = {&a, const_cast<Plan*>(&plan)};
  cudaError_t e = cudaLaunchKernel(k.fn, dim3((unsigned)((a.n_parts + kWinWarps - 1) / kWinWarps)),
                                   dim3(kWinWarps * 32), args, (size_t)k.smem, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3((unsigned)((long)a.batch * a.kv_heads * a.rows));
  cfg.blockDim = dim3(128);
  return cudaLaunchKernelEx(&cfg, &window_merge_kernel<Plan>, a, g, plan);
}

template <class Plan>
cudaError_t clusters(WindowArgs a, const Plan& plan, int g, const WinKernel& k, int ctas, cudaStream_t stream) {
  const long row_chunks = (long)a.batch * a.kv_heads * (a.rows / g);
  int ranks = 1;
  while (ranks < kMaxRanks && ranks * kWinWarps < a.most_items && row_chunks * ranks * 2 <= ctas) ranks *= 2;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3((unsigned)(row_chunks * ranks));
  cfg.blockDim = dim3(kWinWarps * 32);
  cfg.dynamicSmemBytes = (size_t)k.smem;
  void* args[] = {&a, const_cast<Plan*>(&plan)};
  return cudaLaunchKernelExC(&cfg, k.fn, args);
}

// Items of one kv head over all sequences, and of the longest row.
template <class Plan>
long items_per_head(const WindowArgs& a, const Plan* plan, int* most) {
  if constexpr (kRagged<Plan>) {
    long sum = 0;
    *most = 0;
    for (int b = 0; b < a.batch; ++b) {
      const int n = item_list(a.queries, a.window, a.sinks, plan->blocks[b], plan->tail[b]).n;
      if (n > *most) *most = n;
      sum += n;
    }
    return sum;
  } else {
    *most = item_list(a.queries, a.window, a.sinks, a.n_blocks, a.tail_len).n;
    return (long)a.batch * *most;
  }
}

// Query rows of a chunk (1, 2 or 4) and the form.  A record's codes are read and masked
// once per chunk, so larger chunks do less work in all; smaller ones spread it over more
// warps.  Measured (us, E the even split, C clusters, digits the chunk's rows; uncompressed
// records, and in brackets compressed ones):
//   8 kv heads x 4 rows, 5 blocks:        C1 6.9  C2 8.2  C4 10.3  E1 10.6
//   2 kv heads x 8 rows, 36 blocks:       C1 10.1 C2 11.4 E1 12.9  E2 13.1 (30 32 25 24)
//   8 kv heads x 8 rows, 36 blocks:       C2 12.6 C1 13.6 E2 14.6  E4 15.9 (36 46 28 28)
//   32 kv heads x 2 rows, 18 blocks:      C2 8.6  C1 10.6 E2 11.5          (21 31 22)
//   2 x 32 kv heads x 4 rows, 18 blocks:  E2 15.1 E4 15.5 C2 16.1  C4 16.8 (35 30 52 42)
//   16 x 8 kv heads x 4 rows, 33 blocks:  E2 28.7 E4 29.7 C4 32.7  E1 40.6 (124 87 102 210)
// so, for uncompressed records: single rows while they give every scheduler of the device at most one item, pairs
// while they fill at most half of the warps it holds, both in clusters; else four rows (or
// what there is), in clusters while those items fill at most half of the warps.  The host does
// not know which records are compressed (index entries are on the device), so caches of
// compressed ones follow the same rule and lose where the brackets differ: 30 against 24 us in
// the second line, 36 against 28 in the third.
template <class Plan>
cudaError_t launch_window_p(WindowArgs a, Plan& plan, cudaStream_t stream) {
  const long per_head = items_per_head(a, &plan, &a.most_items);
  auto items = [&](int g) { return per_head * a.kv_heads * (a.rows / g); };
  int sms = 0, dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int g = a.rows < 4 ? a.rows : 4, ctas = 0;
  bool cluster = false;
  if (items(1) <= 4L * sms) {
    g = 1;
    cluster = true;
  } else if (a.rows >= 2) {
    e = win_configure(win_select<Plan>(a.bits, 2, true), dev, &ctas);
    if (e != cudaSuccess) return e;
    if (2 * items(2) <= (long)ctas * kWinWarps) {
      g = 2;
      cluster = true;
    }
  }
  const WinKernel even = win_select<Plan>(a.bits, g, true);
  e = win_configure(even, dev, &ctas);
  if (e != cudaSuccess) return e;
  cluster = cluster || 2 * items(g) <= (long)ctas * kWinWarps;
  a.n_items = items(g);
  if constexpr (kRagged<Plan>) {
    long at = 0;
    for (int b = 0; b < a.batch; ++b) {
      plan.base[b] = (int32_t)at;
      at += (long)item_list(a.queries, a.window, a.sinks, plan.blocks[b], plan.tail[b]).n * a.kv_heads * (a.rows / g);
    }
    plan.base[a.batch] = (int32_t)at;
  }
  if (!cluster) return even_split(a, plan, g, even, ctas * kWinWarps, stream);
  const WinKernel k = win_select<Plan>(a.bits, g, false);
  e = win_configure(k, dev, &ctas);
  if (e != cudaSuccess) return e;
  return clusters(a, plan, g, k, ctas, stream);
}

}  // namespace

bool window_countable(const WindowArgs& a, const WindowPlan* plan) {
  int most = 0;
  const NoPlan none;
  const long per_head = plan ? items_per_head(a, plan, &most) : items_per_head(a, &none, &most);
  return per_head <= 0x7fffffffL / ((long)a.kv_heads * a.rows);
}

size_t window_workspace_bytes(int batch, int kv_heads, int rows) {
  // (parts + (row, chunk)s) slots of a chunk's rows: at most this for any chunk
  return ((size_t)max_parts() * (rows < 4 ? rows : 4) + (size_t)batch * kv_heads * rows) * kPartFloats * sizeof(float);
}

cudaError_t launch_window(WindowArgs a, const WindowPlan* plan, cudaStream_t stream) {
  if (plan != nullptr && a.batch > kSmallBatch) {
    thread_local WindowPlan p;
    std::memcpy(p.blocks, plan->blocks, sizeof(int32_t) * a.batch);
    std::memcpy(p.tail, plan->tail, a.batch);
    return launch_window_p(a, p, stream);
  }
  if (plan != nullptr) {
    WindowPlanT<kSmallBatch> p;
    std::memcpy(p.blocks, plan->blocks, sizeof(int32_t) * a.batch);
    std::memcpy(p.tail, plan->tail, a.batch);
    return launch_window_p(a, p, stream);
  }
  NoPlan none;
  return launch_window_p(a, none, stream);
}

}  // namespace packkv
