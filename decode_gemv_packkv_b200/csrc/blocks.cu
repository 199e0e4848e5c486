// The cache's blocks: forking sequences, giving blocks up, and compacting the arenas.
//
// Records are immutable and found through index entries {offset16, length16}, so a fork
// copies entries (two entries may name one record) and a free marks them.  Only
// compaction moves records: out of place, every live record once, in (sequence, head,
// logical block) order of the first entry that names it.
//
// Compaction.  A record is at least 1040 bytes (65 units of 16), and records do not
// overlap, so at most one starts in any 65 units: owner[offset16 / 65] (atomicMax of the
// complemented entry number, so the order of arrival does not matter) names the first
// entry of each record.  One pass of a decoupled look-back over tiles of entries sums
// the lengths of owned records into new offsets; a second kernel copies the records and
// writes the new entries.  Bound: HBM, 2 bytes moved per live byte.  The 22 k live records of
// 16 x 32 rows of 64 blocks (394 MB moved) take 88 us: 4 marking, 10 summing offsets, 77
// copying at 5.1 TB/s (a plain copy runs at 6.56).  The copy is not shared out evenly: a
// warp's next batch lies 4736 entries on, a multiple of 64, so it stays at the same four block
// numbers of its rows, and as rows end at different lengths the fullest of the 1184 warps
// has 44 records, the mean 19 and 52 none (the fullest SM 172, the mean 149).  Warps that
// copied with 16-byte loads and stores, four in flight, took 151.
// Forks and frees are a few entries per block: bound by the launch.  Three CTAs per (pair,
// head), four loads in flight: 32 pairs x 8 heads of 64 blocks in 3.8 us (6.9 with one CTA).
#include <atomic>

#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "mover.cuh"

namespace packkv {

namespace {

constexpr uint32_t kFreed = 0xFFFFFFFFu;
constexpr unsigned long long kFreedEntry = 0xFFFFFFFFull;  // {offset 0xFFFFFFFF, length 0}
constexpr uint32_t kMinRecord16 = 1040 / 16;

// Index row (in entries) of logical block j of (sequence b, head h), -1 if the block
// table names no block of the index.
__device__ __forceinline__ long entry_at(const packkv_cache& c, int b, int h, int j) {
  long rb = b, jb = j;
  if (c.block_table != nullptr) {
    const int p = c.block_table[(size_t)b * c.max_blocks + j];
    if (p < 0 || (long)p >= (long)c.batch * c.max_blocks) return -1;
    rb = p / c.max_blocks;
    jb = p % c.max_blocks;
  }
  return (rb * c.kv_heads + h) * c.max_blocks + jb;
}

__device__ __forceinline__ unsigned long long* entry_ptr(uint32_t* index, long e) {
  return reinterpret_cast<unsigned long long*>(index) + e;
}

// Copies n uint4 with the whole CTA, four loads in flight per thread.
__device__ __forceinline__ void copy16(void* dst, const void* src, int n) {
  uint4* d = reinterpret_cast<uint4*>(dst);
  const uint4* s = reinterpret_cast<const uint4*>(src);
  for (int i0 = threadIdx.x; i0 < n; i0 += 4 * blockDim.x) {
    uint4 r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + k * (int)blockDim.x < n) r[k] = s[i0 + k * blockDim.x];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i0 + k * (int)blockDim.x < n) d[i0 + k * blockDim.x] = r[k];
  }
}

// Three CTAs per (pair, head): the K tail, the V tail, and the blocks' entries and
// permutations.
template <int N>
__global__ void __launch_bounds__(256) fork_kernel(const packkv_cache c, const __grid_constant__ PairPlanT<N> plan) {
  const int part = blockIdx.x % 3, ih = blockIdx.x / 3;
  const int i = ih / c.kv_heads, h = ih % c.kv_heads;
  const int src = plan.src[i], dst = plan.dst[i];
  if (part < 2) {
    const size_t ts = ((size_t)src * c.kv_heads + h) * 128 * 128, td = ((size_t)dst * c.kv_heads + h) * 128 * 128;
    uint16_t* tail = part == 0 ? c.k_tail : c.v_tail;
    copy16(tail + td, tail + ts, plan.tail[i] * 16);
    return;
  }
  const int nb = plan.blocks[i];
  for (int j = threadIdx.x; j < nb; j += blockDim.x) {
    const long from = entry_at(c, src, h, j), to = entry_at(c, dst, h, j);
    if (to < 0) continue;
    const unsigned long long ke = from < 0 ? kFreedEntry : *entry_ptr(c.k_index, from);
    const unsigned long long ve = from < 0 ? kFreedEntry : *entry_ptr(c.v_index, from);
    *entry_ptr(c.k_index, to) = ke;
    *entry_ptr(c.v_index, to) = ve;
  }
  if (c.perm == nullptr) return;
  if (c.block_table == nullptr) {  // the rows' permutations lie side by side
    copy16(c.perm + entry_at(c, dst, h, 0) * 128, c.perm + entry_at(c, src, h, 0) * 128, nb * 8);
    return;
  }
  for (int x = threadIdx.x; x < nb * 8; x += blockDim.x) {  // 128 bytes of a block: 8 uint4
    const int j = x >> 3, k = x & 7;
    const long from = entry_at(c, src, h, j), to = entry_at(c, dst, h, j);
    if (from < 0 || to < 0) continue;
    reinterpret_cast<uint4*>(c.perm + to * 128)[k] = reinterpret_cast<const uint4*>(c.perm + from * 128)[k];
  }
}

template <int N>
__global__ void __launch_bounds__(128) free_kernel(const packkv_cache c, const __grid_constant__ RangePlanT<N> plan) {
  const int b = blockIdx.x / c.kv_heads, h = blockIdx.x % c.kv_heads;
  const int first = plan.first[b], n = plan.count[b];
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    const long e = entry_at(c, b, h, first + j);
    if (e < 0) continue;
    *entry_ptr(c.k_index, e) = kFreedEntry;
    *entry_ptr(c.v_index, e) = kFreedEntry;
  }
}

// ---- compaction --------------------------------------------------------------------
// Workspace: [2][slots] owners, [2][tiles] look-back words, tickets[2], totals[2] (all
// cleared first), then [2][entries] new offsets.
constexpr int kTile = 1024;  // entries of a look-back tile, one per thread

struct CompactWs {
  uint32_t* owner[2];
  unsigned long long* tile[2];
  uint32_t* ticket;            // [2]
  unsigned long long* total;   // [2], written by the last tile
  uint32_t* moved[2];          // new offset of entry e (owners only)
  size_t clear_bytes, bytes;
};

CompactWs compact_ws(void* ws, int64_t entries, uint64_t arena16) {
  CompactWs w{};
  uint8_t* p = reinterpret_cast<uint8_t*>(ws);
  size_t at = 0;
  auto take = [&](size_t n) {
    uint8_t* r = p + at;
    at += (n + 15) / 16 * 16;
    return r;
  };
  const size_t slots = arena16 / kMinRecord16 + 1, tiles = (size_t)(entries + kTile - 1) / kTile;
  for (auto& o : w.owner) o = reinterpret_cast<uint32_t*>(take(slots * 4));
  for (auto& t : w.tile) t = reinterpret_cast<unsigned long long*>(take(tiles * 8));
  w.ticket = reinterpret_cast<uint32_t*>(take(8));
  w.total = reinterpret_cast<unsigned long long*>(take(16));
  w.clear_bytes = at;
  for (auto& m : w.moved) m = reinterpret_cast<uint32_t*>(take((size_t)entries * 4));
  w.bytes = at;
  return w;
}

// The entry list of a compaction: entry e is logical block e % most of row e / most.
struct CompactArgs {
  packkv_cache dst, src;
  CompactWs ws;
  int most;
  int64_t entries;
};

// Source entry e of a tensor: false past the sequence's blocks.  *rec = {offset, length},
// {0xFFFFFFFF, 0} for a freed or an invalid one (*bad).
template <class Plan>
__device__ __forceinline__ bool source_entry(const CompactArgs& a, const Plan& plan, int tensor, int64_t e,
                                             uint2* rec, long* at, bool* bad) {
  const int row = (int)(e / a.most), j = (int)(e - (int64_t)row * a.most);
  const int b = row / a.src.kv_heads, h = row - b * a.src.kv_heads;
  *rec = make_uint2(kFreed, 0u);
  *bad = false;
  if (j >= plan.blocks[b]) return false;
  *at = entry_at(a.src, b, h, j);
  if (*at < 0) {
    *bad = true;
    return true;
  }
  const uint2 r = *reinterpret_cast<const uint2*>((tensor ? a.src.v_index : a.src.k_index) + 2 * *at);
  if (r.x == kFreed) {
    *bad = r.y != 0u;
    return true;
  }
  const uint32_t most16 = (uint32_t)raw_record_bytes((int)a.src.fmt.bits) / 16u;
  if (r.y < kMinRecord16 || r.y > most16 || (uint64_t)r.x + r.y > a.src.arena_bytes / 16)
    *bad = true;
  else
    *rec = r;
  return true;
}

template <int N>
__global__ void __launch_bounds__(256) mark_kernel(const CompactArgs a, const __grid_constant__ LengthPlanT<N> plan) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t x = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (x >= 2 * a.entries) return;
  const int tensor = x >= a.entries;
  const int64_t e = x - (tensor ? a.entries : 0);
  uint2 r;
  long at;
  bool bad;
  if (!source_entry(a, plan, tensor, e, &r, &at, &bad) || r.x == kFreed) return;
  atomicMax(a.ws.owner[tensor] + r.x / kMinRecord16, ~(uint32_t)e);
}

// Whether entry e, record r, is the first that names its record; *first = that entry,
// -1 if the slot belongs to a record that overlaps r (a corrupt index).
template <class Plan>
__device__ __forceinline__ bool owns_record(const CompactArgs& a, const Plan& plan, int tensor, int64_t e,
                                            const uint2& r, int64_t* first) {
  *first = (int64_t)(uint32_t)~__ldcg(a.ws.owner[tensor] + r.x / kMinRecord16);
  if (*first == e) return true;
  uint2 o;
  long at;
  bool bad;
  source_entry(a, plan, tensor, *first, &o, &at, &bad);
  if (o.x != r.x || o.y != r.y) *first = -1;
  return false;
}

// Inclusive sums over the threads of a tile; warp_sums[last] = the whole.  All kTile threads.
__device__ __forceinline__ uint32_t tile_scan(uint32_t len, uint32_t* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31;
  uint32_t incl = len;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sums[tid >> 5] = incl;
  __syncthreads();
  if (tid < 32) {
    uint32_t s = warp_sums[tid];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[tid] = s;
  }
  __syncthreads();
  return incl + (tid >= 32 ? warp_sums[(tid >> 5) - 1] : 0u);
}

constexpr unsigned long long kAggregate = 1ull << 62, kPrefix = 2ull << 62, kValue = (1ull << 62) - 1;

// Exclusive sums of the owned records' lengths: tile `ticket` of tensor blockIdx.y.
template <int N>
__global__ void __launch_bounds__(kTile) offsets_kernel(const CompactArgs a, const __grid_constant__ LengthPlanT<N> plan) {
  __shared__ uint32_t warp_sums[kTile / 32];
  __shared__ uint32_t my_tile;
  __shared__ unsigned long long before;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tensor = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) my_tile = atomicAdd(a.ws.ticket + tensor, 1u);  // every earlier tile's CTA has started
  __syncthreads();
  const uint32_t tile = my_tile;
  const int64_t e = (int64_t)tile * kTile + tid;
  uint32_t len = 0u;
  if (e < a.entries) {
    uint2 r;
    long at;
    bool bad;
    int64_t first;
    if (source_entry(a, plan, tensor, e, &r, &at, &bad) && r.x != kFreed && owns_record(a, plan, tensor, e, r, &first))
      len = r.y;
  }
  const uint32_t incl = tile_scan(len, warp_sums);
  const uint32_t tile_sum = warp_sums[kTile / 32 - 1];
  if (tid < 32) {  // warp 0 looks back over 32 tiles at a time
    unsigned long long* words = a.ws.tile[tensor];
    if (tid == 0 && tile > 0) atomicExch(words + tile, kAggregate | tile_sum);
    unsigned long long sum = 0ull;
    const uint64_t start = global_ns();
    for (int64_t t = (int64_t)tile - 1; t >= 0;) {
      const int64_t mine = t - lane;  // lane 0 the nearest
      const unsigned long long w = mine >= 0 ? atomicAdd(words + mine, 0ull) : kPrefix;
      if (__any_sync(0xffffffffu, w == 0ull)) {  // not published yet: bounded wait (a CTA that is running)
        if (__any_sync(0xffffffffu, global_ns() - start > 1000000000ull)) {
          if (lane == 0) set_status(a.dst.ctrl, PACKKV_DEV_TIMEOUT);
          break;
        }
        continue;
      }
      const uint32_t done = __ballot_sync(0xffffffffu, (w & kPrefix) != 0ull);
      unsigned long long add = done == 0u || lane <= __ffs(done) - 1 ? w & kValue : 0ull;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
      sum += add;
      if (done) break;
      t -= 32;
    }
    if (tid == 0) {
      atomicExch(words + tile, kPrefix | (sum + tile_sum));
      before = sum;
      if ((int64_t)(tile + 1) * kTile >= a.entries) a.ws.total[tensor] = sum + tile_sum;
    }
  }
  __syncthreads();
  if (len != 0u)
    a.ws.moved[tensor][e] = (uint32_t)(before + incl - len);
}

// Small caches (one tile): a CTA per tensor clears the owner slots, marks and sums, one launch
// instead of a clearing and two kernels (10.3 against 12.2 us for the whole compaction of 384
// entries; looped over more tiles it drew level at 2048 entries).
constexpr uint64_t kOneCtaSlots = 16 * kTile;

template <int N>
__global__ void __launch_bounds__(kTile) small_offsets_kernel(const CompactArgs a, uint32_t slots,
                                                              const __grid_constant__ LengthPlanT<N> plan) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint32_t warp_sums[kTile / 32];
  const int tensor = blockIdx.x, tid = threadIdx.x;
  uint32_t* owner = a.ws.owner[tensor];
  for (uint32_t i = tid; i < slots; i += kTile) __stcg(owner + i, 0u);
  __syncthreads();
  uint2 r = make_uint2(kFreed, 0u);
  long at;
  bool bad;
  const bool there = tid < a.entries && source_entry(a, plan, tensor, tid, &r, &at, &bad) && r.x != kFreed;
  if (there) atomicMax(owner + r.x / kMinRecord16, ~(uint32_t)tid);
  __syncthreads();
  int64_t first;
  const uint32_t len = there && owns_record(a, plan, tensor, tid, r, &first) ? r.y : 0u;
  const uint32_t incl = tile_scan(len, warp_sums);
  if (len != 0u) a.ws.moved[tensor][tid] = incl - len;
  if (tid == 0) a.ws.total[tensor] = warp_sums[kTile / 32 - 1];
}

// ---- the copy ----
// A warp takes batches of four entries of both tensors: eight lanes look their entries
// up side by side and write the new ones, then lane 0 moves the owned records through
// three shared-memory stages with bulk copies (a load and a store in flight at a time).
constexpr int kMoveWarps = 4;
constexpr int kBatch = 4;

__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

struct BulkPort {  // a warp's stages and their barriers
  unsigned char* base;
  uint32_t stage_bytes;
  uint64_t* bar;
  uint64_t* ctrl;

  __device__ __forceinline__ void load(int s, const void* from, uint32_t bytes) {
    mbar_arrive_expect_tx(bar + s, bytes);
    bulk_g2s(base + s * stage_bytes, from, bytes, bar + s);
  }
  __device__ __forceinline__ bool landed(int s, uint32_t phase) { return mbar_wait_bounded(bar + s, phase, ctrl); }
  __device__ __forceinline__ void store(int s, void* to, uint32_t bytes) { bulk_s2g(to, base + s * stage_bytes, bytes); }
  __device__ __forceinline__ void await_reads() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
  __device__ __forceinline__ void await_stores() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
};

// Two CTAs per SM, as many as the grid has (registers to spare: at the compiler's own choice of
// 64 a few were spilled).
template <int N>
__global__ void __launch_bounds__(kMoveWarps * 32, 2) move_kernel(const CompactArgs a, uint32_t stage_bytes,
                                                              const __grid_constant__ LengthPlanT<N> plan) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint64_t bars[kMoveWarps][kMoveStages];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t warps = (int64_t)gridDim.x * kMoveWarps;
  const int64_t warp0 = (int64_t)warp * gridDim.x + blockIdx.x;  // neighbours in the list go to different SMs
  const unsigned long long total_k = a.ws.total[0], total_v = a.ws.total[1];
  const unsigned long long room = a.dst.arena_bytes / 16;
  const bool fits = total_k <= room && total_v <= room;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.dst.ctrl[kCtrlKEnd] = fits ? total_k : 0ull;
    a.dst.ctrl[kCtrlVEnd] = fits ? total_v : 0ull;
    a.dst.ctrl[kCtrlScratch] = 0ull;
    if (!fits) set_status(a.dst.ctrl, PACKKV_DEV_CAPACITY);
  }
  if (lane == 0) {
    for (int s = 0; s < kMoveStages; ++s) mbar_init(&bars[warp][s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  Mover<BulkPort> mv{{smem + warp * kMoveStages * stage_bytes, stage_bytes, bars[warp], a.dst.ctrl}, 0, nullptr, 0u, false};
  const int64_t batches = (a.entries + kBatch - 1) / kBatch;
  for (int64_t x = warp0; x < batches; x += warps) {
    const int tensor = (lane / kBatch) & 1;
    const int64_t e = x * kBatch + lane % kBatch;
    uint2 r = make_uint2(kFreed, 0u);
    long at = -1, to = -1;
    bool bad = false, own = false, live = false;
    uint32_t off = 0u;
    if (lane < 2 * kBatch && e < a.entries) live = source_entry(a, plan, tensor, e, &r, &at, &bad);
    if (live) {
      const int row = (int)(e / a.most), j = (int)(e - (int64_t)row * a.most);
      const int b = row / a.src.kv_heads;
      to = entry_at(a.dst, b, row - b * a.src.kv_heads, j);
      unsigned long long entry = kFreedEntry;
      if (r.x != kFreed && fits) {
        int64_t first;
        own = owns_record(a, plan, tensor, e, r, &first);
        if (first < 0) {
          bad = true;
        } else {
          off = a.ws.moved[tensor][first];
          entry = (unsigned long long)off | ((unsigned long long)r.y << 32);
          own = own && off + (uint64_t)r.y <= room;  // always, unless the look-back gave up (status set)
        }
      }
      if (bad) set_status(a.dst.ctrl, PACKKV_DEV_BAD_RECORD);
      if (to >= 0) *entry_ptr(tensor ? a.dst.v_index : a.dst.k_index, to) = entry;
    }
    uint32_t todo = __ballot_sync(0xffffffffu, own);
    while (todo) {
      const int k = __ffs(todo) - 1;
      todo &= todo - 1;
      const uint32_t so = __shfl_sync(0xffffffffu, r.x, k), n16 = __shfl_sync(0xffffffffu, r.y, k);
      const uint32_t dof = __shfl_sync(0xffffffffu, off, k);
      if (lane == 0)
        mv.move((k >= kBatch ? a.dst.v_arena : a.dst.k_arena) + (uint64_t)dof * 16,
                (k >= kBatch ? a.src.v_arena : a.src.k_arena) + (uint64_t)so * 16, n16 * 16u);
    }
    if (a.dst.perm != nullptr) {
      const int k = lane >> 3;  // four entries, eight lanes each
      const long from = __shfl_sync(0xffffffffu, at, k), dest = __shfl_sync(0xffffffffu, to, k);
      if (from >= 0 && dest >= 0)
        reinterpret_cast<uint4*>(a.dst.perm + dest * 128)[lane & 7] =
            reinterpret_cast<const uint4*>(a.src.perm + from * 128)[lane & 7];
    }
  }
  // tails: 32 tokens (512 uint4) of K or V per task
  const int64_t rows = (int64_t)a.src.batch * a.src.kv_heads;
  for (int64_t x = warp0; x < rows * 8; x += warps) {
    const int64_t row = x >> 3;
    const int part = (int)(x & 3);
    const int n = min(512, plan.tail[row / a.src.kv_heads] * 16 - part * 512);
    const uint4* s = reinterpret_cast<const uint4*>(((x & 4) ? a.src.v_tail : a.src.k_tail) + row * 128 * 128) + part * 512;
    uint4* d = reinterpret_cast<uint4*>(((x & 4) ? a.dst.v_tail : a.dst.k_tail) + row * 128 * 128) + part * 512;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int q = (half * 8 + i) * 32 + lane;
        if (q < n) v[i] = __ldcs(s + q);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int q = (half * 8 + i) * 32 + lane;
        if (q < n) __stcs(d + q, v[i]);
      }
    }
  }
  if (lane == 0) mv.finish();
}

// SMs of the current device; the first time there, raises the move kernels' shared memory limit.
cudaError_t move_configure(int* sms) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  const int smem = kMoveWarps * kMoveStages * raw_record_bytes(4);
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(&move_kernel<kSmallBatch>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(&move_kernel<kMaxRaggedBatch>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && dev < kMaxDevices) known[dev].store(*sms, std::memory_order_relaxed);
  return e;
}

}  // namespace

cudaError_t launch_fork(const packkv_cache& c, const PairPlan& plan, int n, cudaStream_t stream) {
  const unsigned grid = (unsigned)(3 * n * c.kv_heads);
  if (n > kSmallBatch) {
    fork_kernel<<<grid, 256, 0, stream>>>(c, plan);
  } else {
    PairPlanT<kSmallBatch> small;
    for (int i = 0; i < n; ++i) {
      small.src[i] = plan.src[i];
      small.dst[i] = plan.dst[i];
      small.blocks[i] = plan.blocks[i];
      small.tail[i] = plan.tail[i];
    }
    fork_kernel<<<grid, 256, 0, stream>>>(c, small);
  }
  return cudaGetLastError();
}

cudaError_t launch_free(const packkv_cache& c, const RangePlan& plan, int most, cudaStream_t stream) {
  const int threads = most >= 128 ? 128 : (most + 31) / 32 * 32;
  const unsigned grid = (unsigned)(c.batch * c.kv_heads);
  if (c.batch > kSmallBatch) {
    free_kernel<<<grid, threads, 0, stream>>>(c, plan);
  } else {
    RangePlanT<kSmallBatch> small;
    for (int b = 0; b < c.batch; ++b) {
      small.first[b] = plan.first[b];
      small.count[b] = plan.count[b];
    }
    free_kernel<<<grid, threads, 0, stream>>>(c, small);
  }
  return cudaGetLastError();
}

size_t compact_workspace_bytes(int64_t entries, uint64_t arena16) { return compact_ws(nullptr, entries, arena16).bytes; }

namespace {

template <int N>
cudaError_t compact_with(const packkv_cache& dst, const packkv_cache& src, const LengthPlanT<N>& plan, int most,
                         void* ws, cudaStream_t stream) {
  CompactArgs a{};
  a.dst = dst;
  a.src = src;
  a.most = most > 0 ? most : 1;
  a.entries = (int64_t)src.batch * src.kv_heads * a.most;
  a.ws = compact_ws(ws, a.entries, src.arena_bytes / 16);
  int sms = 0;
  cudaError_t e = move_configure(&sms);
  if (e != cudaSuccess) return e;
  // each launch may start while the one before drains (griddepcontrol.wait in the later ones)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const uint64_t slots = src.arena_bytes / 16 / kMinRecord16 + 1;
  if (a.entries <= kTile && slots <= kOneCtaSlots) {
    small_offsets_kernel<<<2, kTile, 0, stream>>>(a, (uint32_t)slots, plan);
    e = cudaGetLastError();
  } else {
    e = cudaMemsetAsync(ws, 0, a.ws.clear_bytes, stream);
    if (e != cudaSuccess) return e;
    mark_kernel<<<(unsigned)((2 * a.entries + 255) / 256), 256, 0, stream>>>(a, plan);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)((a.entries + kTile - 1) / kTile), 2);
    cfg.blockDim = dim3(kTile);
    e = cudaLaunchKernelEx(&cfg, &offsets_kernel<N>, a, plan);
  }
  if (e != cudaSuccess) return e;
  const uint32_t stage = (uint32_t)raw_record_bytes((int)src.fmt.bits);
  const size_t smem = (size_t)kMoveWarps * kMoveStages * stage;
  const int64_t tasks = (a.entries + kBatch - 1) / kBatch, want = (tasks + kMoveWarps - 1) / kMoveWarps;
  cfg.gridDim = dim3((unsigned)(want < 2L * sms ? want : 2L * sms));
  cfg.blockDim = dim3(kMoveWarps * 32);
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, &move_kernel<N>, a, stage, plan);
}

}  // namespace

cudaError_t launch_compact(const packkv_cache& dst, const packkv_cache& src, const LengthPlan& plan, int most, void* ws,
                           cudaStream_t stream) {
  if (src.batch > kSmallBatch) return compact_with(dst, src, plan, most, ws, stream);
  LengthPlanT<kSmallBatch> small;
  for (int b = 0; b < src.batch; ++b) {
    small.blocks[b] = plan.blocks[b];
    small.tail[b] = plan.tail[b];
  }
  return compact_with(dst, src, small, most, ws, stream);
}

}  // namespace packkv
