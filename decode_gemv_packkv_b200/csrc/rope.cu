// Norm of the query and key heads with the position rotation in the same pass, values
// cast beside them, and the single-token form that appends to the cache's tails.
//
// Per head of 128 channels, fp32: y_c = x_c * rsqrt(mean x^2 + eps) * w_c, then each
// rotated pair (a, b) -> amplitude * (a cos t - b sin t, b cos t + a sin t), one rounding
// to fp16.  The angle of pair i at a position is position * turn[i] in 2^-64 turns, a
// wrapping 64-bit product: exact modulo whole turns however far the position, so the
// fp32 sine and cosine see an argument in [-1, 1) half turns that is off by 2^-25.
//
// Bound: HBM bytes (each input and output element once).  A prompt of 4 x 4096 tokens with
// 32 + 8 heads in bf16 (403 MB) takes 69.6 us, 5.8 TB/s; a plain copy runs at 6.56.  What
// brought it there: a half-warp keeps one token, so that its cosines, sines and weights
// stay in registers over all heads (93 -> 81 us), four rows in flight, each loaded again as
// soon as it is converted (-> 75), and registers for six CTAs per SM instead of eight (-> 70;
// 55.7e6 warp instructions at 64 registers, 39.3e6 at 71).
// A half-warp takes one head at a time; lane l has channels A..A+3 and B..B+3, chosen so
// that both members of each pair sit in one lane (no shuffles for the rotation): half layout
// A = 4l, B = rot/2 + 4l (the unrotated rest packed behind), interleaved A = 4l, B = 64 + 4l.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace packkv {

namespace {

constexpr int kThreads = 128;
constexpr int kRowSlots = kThreads / 16;     // heads side by side in a CTA
constexpr int kTokTile = kRowSlots;          // most tokens of a CTA: one per half-warp
constexpr int kDepth = 4;                    // rows a half-warp has in flight
// Resident CTAs per SM that the registers are sized for (4 x 4096 tokens; 16-bit rows: six 70,
// eight 75, five 77 us; swapping ones: five 85, six 89; fp32 rows: five 116, four 129, six 124).
constexpr int heads_ctas(int size, bool wide, bool swap) { return !wide ? 1 : (size == 2 && !swap ? 6 : 5); }

template <class T>
struct Vec4;  // four consecutive elements
template <>
struct Vec4<__half> {
  using Raw = uint2;
  __device__ static float4 widen(const uint2& r) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
};
template <>
struct Vec4<__nv_bfloat16> {
  using Raw = uint2;
  __device__ static float4 widen(const uint2& r) {
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xFFFF0000u));
  }
};
template <>
struct Vec4<float> {
  using Raw = uint4;
  __device__ static float4 widen(const uint4& r) {
    return make_float4(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w));
  }
};

__device__ __forceinline__ float widen1(__half x) { return __half2float(x); }
__device__ __forceinline__ float widen1(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen1(float x) { return x; }

__device__ __forceinline__ uint2 half4(const float (&y)[4]) {
  const __half2 a = __floats2half2_rn(y[0], y[1]), b = __floats2half2_rn(y[2], y[3]);
  uint2 r;
  r.x = *reinterpret_cast<const uint32_t*>(&a);
  r.y = *reinterpret_cast<const uint32_t*>(&b);
  return r;
}

// The channels of a lane and how its pairs turn.  Wide (vector accesses): ca + i and
// cb + i, i < 4.  Narrow (unaligned rows): element i at channels ca_i and cb_i.  Half
// layouts whose rot_dim is no multiple of 8 cannot have both members of every pair at
// aligned places of one lane: they swap members through shared memory (kSwap).
struct LaneMap {
  int ca[4], cb[4];
  int pa[4], pb[4];  // pair of element i of A and of B
};

// Layout of lane l (0..15).  half: (A_i, B_i) is pair pa[i]; interleaved: (A_0, A_1),
// (A_2, A_3), (B_0, B_1), (B_2, B_3) are pairs.
template <bool kHalf, bool kWide, bool kSwap>
__device__ __forceinline__ LaneMap lane_map(int rot, int l) {
  LaneMap m;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kSwap) {
      m.ca[i] = 4 * l + i;
      m.cb[i] = 64 + 4 * l + i;
      m.pa[i] = m.ca[i] < rot / 2 ? m.ca[i] : m.ca[i] - rot / 2;
      m.pb[i] = m.cb[i] < rot / 2 ? m.cb[i] : m.cb[i] - rot / 2;
    } else if constexpr (!kHalf) {
      m.ca[i] = 4 * l + i;
      m.cb[i] = 64 + 4 * l + i;
      m.pa[i] = 2 * l + (i >> 1);
      m.pb[i] = 32 + 2 * l + (i >> 1);
    } else if constexpr (kWide) {  // rot a multiple of 8
      const bool turned = 8 * l < rot;
      m.ca[i] = (turned ? 4 * l : rot + 8 * (l - rot / 8)) + i;
      m.cb[i] = (turned ? rot / 2 + 4 * l : rot + 8 * (l - rot / 8) + 4) + i;
      m.pa[i] = m.pb[i] = 4 * l + i;
    } else {
      const int p = l + 16 * i;  // pair p < rot/2, or the (p - rot/2)-th two unrotated channels
      const bool turned = 2 * p < rot;
      m.ca[i] = turned ? p : 2 * p;
      m.cb[i] = turned ? p + rot / 2 : 2 * p + 1;
      m.pa[i] = m.pb[i] = p;
    }
  }
  return m;
}

struct HeadRow {
  float a[4], b[4];
};

template <class T, bool kWide>
struct RowLoad {  // the loads of a row, before the conversion
  typename Vec4<T>::Raw ra, rb;
  __device__ void clear() { ra = rb = typename Vec4<T>::Raw{}; }
  __device__ void issue(const T* p, const LaneMap& m) {
    ra = __ldcs(reinterpret_cast<const typename Vec4<T>::Raw*>(p + m.ca[0]));
    rb = __ldcs(reinterpret_cast<const typename Vec4<T>::Raw*>(p + m.cb[0]));
  }
  __device__ HeadRow get() const {
    const float4 x = Vec4<T>::widen(ra), y = Vec4<T>::widen(rb);
    return {{x.x, x.y, x.z, x.w}, {y.x, y.y, y.z, y.w}};
  }
};
template <class T>
struct RowLoad<T, false> {
  T ra[4], rb[4];
  __device__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) ra[i] = rb[i] = T(0.f);
  }
  __device__ void issue(const T* p, const LaneMap& m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ra[i] = p[m.ca[i]];
      rb[i] = p[m.cb[i]];
    }
  }
  __device__ HeadRow get() const {
    HeadRow r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.a[i] = widen1(ra[i]);
      r.b[i] = widen1(rb[i]);
    }
    return r;
  }
};

template <bool kHalf, bool kWide>
__device__ __forceinline__ void store_row(uint16_t* dst, const HeadRow& r, const LaneMap& m) {
  if constexpr (kWide || !kHalf) {  // channels ca[0]..+3, cb[0]..+3; outputs are 16-byte aligned
    *reinterpret_cast<uint2*>(dst + m.ca[0]) = half4(r.a);
    *reinterpret_cast<uint2*>(dst + m.cb[0]) = half4(r.b);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dst[m.ca[i]] = __half_as_ushort(__float2half_rn(r.a[i]));
      dst[m.cb[i]] = __half_as_ushort(__float2half_rn(r.b[i]));
    }
  }
}

// What one token does to this lane's channels, the norm's weights folded in: element i of
// A and B (half layout, a pair) or neighbours (interleaved).
//   half:        a' = a ca + b sa,  b' = b cb + a sb   with (wa cos, -wb sin, wb cos, wa sin)
//   interleaved: x' = x c + y s for both members: A in (ca, sa), B in (cb, sb)
// Pairs that are not turned hold (w, 0), and their rows must not read the s terms (an
// infinity would spoil its neighbour).
struct Turn {
  float2 ca[2], sa[2], cb[2], sb[2];
  uint32_t on;  // half: bit i (pair i); interleaved: bits 0, 1 (A), 2, 3 (B); swapped: a bit per channel
};

template <bool kHalf, bool kWide, bool kSwap>
__device__ __forceinline__ Turn lane_turn(const float2* cs, const HeadRow& w, const float* weight, const LaneMap& m,
                                          int rot) {
  Turn u;
  u.on = 0u;
  if constexpr (kSwap) {  // x' = x c + y s with the other member y of the pair, weights folded in
    float* c[2] = {&u.ca[0].x, &u.cb[0].x};
    float* z[2] = {&u.sa[0].x, &u.sb[0].x};
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ch = k ? m.cb[i] : m.ca[i], pair = k ? m.pb[i] : m.pa[i];
        c[k][i] = k ? w.b[i] : w.a[i];
        z[k][i] = 0.f;
        if (ch < rot) {
          const float2 t = cs[pair];
          const bool first = ch < rot / 2;
          const float wy = weight ? weight[first ? ch + rot / 2 : ch - rot / 2] : 1.f;
          c[k][i] *= t.x;
          z[k][i] = (first ? -t.y : t.y) * wy;
          u.on |= 1u << (4 * k + i);
        }
      }
    return u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float ca = w.a[i], sa = 0.f, cb = w.b[i], sb = 0.f;
    if constexpr (kHalf) {
      if (2 * m.pa[i] < rot) {
        const float2 z = cs[m.pa[i]];
        ca = w.a[i] * z.x;
        sa = -w.b[i] * z.y;
        cb = w.b[i] * z.x;
        sb = w.a[i] * z.y;
        u.on |= 1u << i;
      }
    } else {
      const float sign = (i & 1) ? 1.f : -1.f;  // x' = x cos - y sin, y' = y cos + x sin
      if (2 * m.pa[i] < rot) {
        const float2 z = cs[m.pa[i]];
        ca = w.a[i] * z.x;
        sa = sign * w.a[i ^ 1] * z.y;
        u.on |= 1u << (i >> 1);
      }
      if (2 * m.pb[i] < rot) {
        const float2 z = cs[m.pb[i]];
        cb = w.b[i] * z.x;
        sb = sign * w.b[i ^ 1] * z.y;
        u.on |= 4u << (i >> 1);
      }
    }
    float2 *pca = &u.ca[i >> 1], *psa = &u.sa[i >> 1], *pcb = &u.cb[i >> 1], *psb = &u.sb[i >> 1];
    if (i & 1) {
      pca->y = ca, psa->y = sa, pcb->y = cb, psb->y = sb;
    } else {
      pca->x = ca, psa->x = sa, pcb->x = cb, psb->x = sb;
    }
  }
  return u;
}

// Place of channel c in a half-warp's swap row: a word of padding per 32, so that lanes four
// channels apart meet different banks.
__device__ __forceinline__ int swap_at(int c) { return c + (c >> 5); }
constexpr int kSwapRow = 133;  // 131 words used; a half-warp has two rows: its neighbour lies 10 banks on

// Norm and rotation of one row.  swap (kSwap): the half-warp's swap row.
template <bool kHalf, bool kWide, bool kSwap>
__device__ __forceinline__ void turn_row(HeadRow& r, bool norm, float eps, const Turn& u, const LaneMap& m, int half,
                                         float* swap) {
  float2 a[2] = {{r.a[0], r.a[1]}, {r.a[2], r.a[3]}}, b[2] = {{r.b[0], r.b[1]}, {r.b[2], r.b[3]}};
  if (norm) {
    float2 s2 = __fmul2_rn(a[0], a[0]);
    s2 = __ffma2_rn(a[1], a[1], s2);
    s2 = __ffma2_rn(b[0], b[0], s2);
    s2 = __ffma2_rn(b[1], b[1], s2);
    float ss = s2.x + s2.y;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);  // within the half-warp
    const float f = rsqrtf(fmaf(ss, 1.f / 128.f, eps));
    const float2 f2 = make_float2(f, f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = __fmul2_rn(a[i], f2);
      b[i] = __fmul2_rn(b[i], f2);
    }
  }
  if constexpr (kSwap) {
    const float v[2][4] = {{a[0].x, a[0].y, a[1].x, a[1].y}, {b[0].x, b[0].y, b[1].x, b[1].y}};
    const float c[2][4] = {{u.ca[0].x, u.ca[0].y, u.ca[1].x, u.ca[1].y}, {u.cb[0].x, u.cb[0].y, u.cb[1].x, u.cb[1].y}};
    const float z[2][4] = {{u.sa[0].x, u.sa[0].y, u.sa[1].x, u.sa[1].y}, {u.sb[0].x, u.sb[0].y, u.sb[1].x, u.sb[1].y}};
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) swap[swap_at(k ? m.cb[i] : m.ca[i])] = v[k][i];
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ch = k ? m.cb[i] : m.ca[i];
        float x = v[k][i] * c[k][i];
        if (u.on & (1u << (4 * k + i))) x = fmaf(swap[swap_at(ch < half ? ch + half : ch - half)], z[k][i], x);
        if (k) r.b[i] = x;
        else r.a[i] = x;
      }
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float2 x = __fmul2_rn(a[i], u.ca[i]), y = __fmul2_rn(b[i], u.cb[i]);
    if constexpr (kHalf && kWide) {
      if (u.on) {  // the lane's pairs turn all or none
        x = __ffma2_rn(b[i], u.sa[i], x);
        y = __ffma2_rn(a[i], u.sb[i], y);
      }
    } else if constexpr (kHalf) {
      if (u.on & (1u << (2 * i))) {
        x.x = fmaf(b[i].x, u.sa[i].x, x.x);
        y.x = fmaf(a[i].x, u.sb[i].x, y.x);
      }
      if (u.on & (2u << (2 * i))) {
        x.y = fmaf(b[i].y, u.sa[i].y, x.y);
        y.y = fmaf(a[i].y, u.sb[i].y, y.y);
      }
    } else {
      if (u.on & (1u << i)) x = __ffma2_rn(make_float2(a[i].y, a[i].x), u.sa[i], x);
      if (u.on & (4u << i)) y = __ffma2_rn(make_float2(b[i].y, b[i].x), u.sb[i], y);
    }
    r.a[2 * i] = x.x;
    r.a[2 * i + 1] = x.y;
    r.b[2 * i] = y.x;
    r.b[2 * i + 1] = y.y;
  }
}

// Where a token goes.  Prompts: token t of sequence b at positions[b*T + t] (or first +
// t), outputs [b][head][t].  Appends: one token per sequence at the length the plan (or
// the uniform length) gives, k and v at that slot of the tails.
struct PromptPlan {};

template <class Plan>
constexpr bool is_append = !std::is_same<Plan, PromptPlan>::value;

struct UniformLength {
  uint32_t tokens;
};

// Tokens sequence b holds (kNoToken: it takes none).
constexpr uint32_t kNoToken = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t length_of(const UniformLength& p, int) { return p.tokens; }
template <int N>
__device__ __forceinline__ uint32_t length_of(const RaggedLengthsT<N>& p, int b) {
  return p.tokens[b];
}

template <class T, bool kHalf, bool kWide, bool kSwap, class Plan>
__global__ void __launch_bounds__(kThreads, heads_ctas(sizeof(T), kWide, kSwap)) heads_kernel(const HeadsArgs a, const __grid_constant__ Plan plan) {
  __shared__ float2 table[kTokTile][64];
  const int tiles = is_append<Plan> ? 1 : (a.tokens + a.tile - 1) / a.tile;
  const int b = blockIdx.x / tiles;
  const int t0 = (blockIdx.x - b * tiles) * a.tile;
  const int nt = is_append<Plan> ? 1 : min(a.tile, a.tokens - t0);
  const int rot = (int)a.rope.rot_dim;
  uint32_t held = 0;
  if constexpr (is_append<Plan>) {
    held = length_of(plan, b);
    if (held == kNoToken) return;
  }
  for (int i = threadIdx.x; i < nt * 64; i += kThreads) {
    const int p = i & 63, t = i >> 6;
    if (2 * p < rot) {
      long long pos;
      if constexpr (is_append<Plan>)
        pos = held;
      else
        pos = a.positions ? (long long)a.positions[(size_t)b * a.tokens + t0 + t] : a.first + t0 + t;
      // signed turns in [-1/2, 1/2) as 64-bit fractions -> half turns
      const long long turns = (long long)((unsigned long long)pos * a.rope.turn[p]);
      float s, c;
      sincospif((float)turns * 1.0842021724855044e-19f, &s, &c);  // 2^-63
      table[t][p] = make_float2(c * a.rope.amplitude, s * a.rope.amplitude);
    }
  }
  const int l = threadIdx.x & 15;
  const LaneMap m = lane_map<kHalf, kWide, kSwap>(rot, l);
  // two swap rows per half-warp in turn: one barrier per row is enough
  __shared__ float swap_rows[kSwap ? kRowSlots : 1][2][kSwap ? kSwapRow : 1];
  int swap_row = 0;
  __syncthreads();
  // half-warp `slot` takes one token of the tile and every `step`-th head, so its token's
  // cosines, sines and the weights stay in registers
  const int slot = threadIdx.x >> 4;
  const int lt = nt > 1 ? 32 - __clz(nt - 1) : 0;  // log2 of the token slots
  const int ti = slot & ((1 << lt) - 1), h0 = slot >> lt, step = kRowSlots >> lt;
  const int t = min(ti, nt - 1);
  const bool mine = ti < nt;
#pragma unroll 1
  for (int which = 0; which < 3; ++which) {  // q, k, v
    const HeadsTensor& x = a.x[which];
    if (x.data == nullptr) continue;
    const bool norm = a.norm && which < 2;
    HeadRow w = {{1.f, 1.f, 1.f, 1.f}, {1.f, 1.f, 1.f, 1.f}};
    if (norm && x.weight != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w.a[i] = x.weight[m.ca[i]];
        w.b[i] = x.weight[m.cb[i]];
      }
    }
    const Turn u = lane_turn<kHalf, kWide, kSwap>(table[t], w, norm ? x.weight : nullptr, m, which < 2 ? rot : 0);
    const T* src = reinterpret_cast<const T*>(x.data) + b * x.batch_stride + (t0 + t) * x.token_stride;
    uint16_t* dst = x.out;
    size_t pitch;  // between heads of the output
    if (!is_append<Plan> || which == 0) {
      pitch = (size_t)a.tokens * kHeadDim;
      dst += ((size_t)b * x.heads * a.tokens + t0 + t) * kHeadDim;
    } else {
      pitch = (size_t)kBlockTokens * kHeadDim;
      dst += ((size_t)b * x.heads * kBlockTokens + (held & (kBlockTokens - 1))) * kHeadDim;
    }
    // kDepth rows in flight: a row's registers are loaded again as soon as it is converted.
    // Whole warps stay in the loop (the norm's shuffles); heads past the end are not loaded.
    src += h0 * x.head_stride;
    dst += h0 * pitch;
    const int64_t src_step = step * x.head_stride;
    const size_t dst_step = step * pitch;
    int left = x.heads - h0;  // heads from this half-warp's next load on
    RowLoad<T, kWide> in[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      in[d].clear();
      if (left > 0) in[d].issue(src, m);
      left -= step;
      src += src_step;
    }
    for (int hb = 0; hb < x.heads; hb += kDepth * step) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (d > 0 && hb + d * step >= x.heads) break;  // CTA-uniform
        HeadRow y = in[d].get();
        if (left > 0) in[d].issue(src, m);
        if (which < 2) {
          turn_row<kHalf, kWide, kSwap>(y, norm, a.eps, u, m, rot / 2, swap_rows[kSwap ? slot : 0][swap_row]);
          if (kSwap) swap_row ^= 1;
        }
        if (mine && left > -kDepth * step) store_row<kHalf, kWide>(dst, y, m);
        left -= step;
        src += src_step;
        dst += dst_step;
      }
    }
  }
}

template <class T, bool kHalf, bool kWide, bool kSwap, class Plan>
cudaError_t launch_heads_t(const HeadsArgs& a, const Plan& plan, cudaStream_t stream) {
  const long tiles = is_append<Plan> ? 1 : (a.tokens + (long)a.tile - 1) / a.tile;
  heads_kernel<T, kHalf, kWide, kSwap, Plan><<<(unsigned)(tiles * a.batch), kThreads, 0, stream>>>(a, plan);
  return cudaGetLastError();
}

// Vector accesses need four consecutive elements aligned to their size everywhere.
bool wide_ok(const HeadsArgs& a) {
  const int bytes = a.dtype == PACKKV_DTYPE_FP32 ? 16 : 8;
  for (const HeadsTensor& x : a.x) {
    if (x.data == nullptr) continue;
    if (reinterpret_cast<uintptr_t>(x.data) % bytes != 0) return false;
    if (x.batch_stride % 4 != 0 || x.token_stride % 4 != 0 || x.head_stride % 4 != 0) return false;
  }
  return true;
}

template <class T, class Plan>
cudaError_t launch_heads_d(const HeadsArgs& a, const Plan& plan, cudaStream_t stream) {
  const bool half = a.rope.layout == PACKKV_ROPE_HALF;
  if (!wide_ok(a))
    return half ? launch_heads_t<T, true, false, false, Plan>(a, plan, stream)
                : launch_heads_t<T, false, false, false, Plan>(a, plan, stream);
  if (!half) return launch_heads_t<T, false, true, false, Plan>(a, plan, stream);
  return a.rope.rot_dim % 8 == 0 ? launch_heads_t<T, true, true, false, Plan>(a, plan, stream)
                                 : launch_heads_t<T, true, true, true, Plan>(a, plan, stream);
}

template <class Plan>
cudaError_t launch_heads_p(const HeadsArgs& a, const Plan& plan, cudaStream_t stream) {
  if (a.dtype == PACKKV_DTYPE_FP16) return launch_heads_d<__half, Plan>(a, plan, stream);
  if (a.dtype == PACKKV_DTYPE_BF16) return launch_heads_d<__nv_bfloat16, Plan>(a, plan, stream);
  return launch_heads_d<float, Plan>(a, plan, stream);
}

}  // namespace

cudaError_t launch_prompt_heads(const HeadsArgs& args, cudaStream_t stream) {
  HeadsArgs a = args;
  // A token per half-warp shares its sines and weights between all its heads; fewer tokens
  // per CTA spread a short prompt over more SMs: eight from three CTAs per SM (148 of them)
  // on, four from one on (3 x 257 tokens of 18 heads: 4.4 us with four, 8.0 with one; 4 x 4096
  // of 48, at 64 registers: 75 us with eight, 88 with four).
  const long n = (long)a.batch * a.tokens;
  a.tile = n >= 8 * 444 ? 8 : (n >= 4 * 148 ? 4 : 1);
  return launch_heads_p(a, PromptPlan{}, stream);
}

cudaError_t launch_append_heads(const HeadsArgs& a, uint32_t tokens, const RaggedLengths* lengths,
                                cudaStream_t stream) {
  if (lengths != nullptr && a.batch > kSmallBatch) return launch_heads_p(a, *lengths, stream);
  if (lengths != nullptr) {
    RaggedLengthsT<kSmallBatch> small;
    for (int b = 0; b < a.batch; ++b) small.tokens[b] = lengths->tokens[b];
    return launch_heads_p(a, small, stream);
  }
  return launch_heads_p(a, UniformLength{tokens}, stream);
}

}  // namespace packkv
