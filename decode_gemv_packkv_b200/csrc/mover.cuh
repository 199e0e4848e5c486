// The order in which one thread moves records through shared-memory stages: load n goes to
// stage n % kMoveStages, the store of load n - 1 is issued behind it, so a load and a store
// are in flight at a time.  The copies themselves are a Port's (blocks.cu: bulk copies), so
// that the order can be checked on the host:
//   load(stage, from, bytes)      starts a load
//   landed(stage, phase)          waits for the stage's load number 2k + phase, bounded
//   store(stage, to, bytes)       starts a store
//   await_reads()                 until all stores but the latest have read their stage
//   await_stores()                until all stores are done
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define PACKKV_DEVICE __device__ __forceinline__
#else
#define PACKKV_DEVICE inline
#endif

namespace packkv {

constexpr int kMoveStages = 3;

template <class Port>
struct Mover {
  Port port;
  long n;          // loads issued
  void* dst;       // of load n - 1, whose store is not issued yet
  uint32_t bytes;
  bool dead;       // a load gave up: nothing more is moved

  PACKKV_DEVICE static int stage_of(long i) { return (int)(i % kMoveStages); }
  PACKKV_DEVICE static uint32_t phase_of(long i) { return (uint32_t)((i / kMoveStages) & 1); }

  PACKKV_DEVICE void store_last() {
    if (n == 0 || dead) return;
    if (!port.landed(stage_of(n - 1), phase_of(n - 1))) {
      dead = true;
      return;
    }
    port.store(stage_of(n - 1), dst, bytes);
  }
  PACKKV_DEVICE void move(void* to, const void* from, uint32_t nbytes) {
    if (dead) return;
    port.await_reads();  // stores up to n - 2 are issued; the stage held record n - 3
    port.load(stage_of(n), from, nbytes);
    store_last();
    ++n;
    dst = to;
    bytes = nbytes;
  }
  PACKKV_DEVICE void finish() {
    // a load that gave up in move() has left one behind it in flight, which must land before
    // the block may leave; one that gives up here has none
    if (dead)
      port.landed(stage_of(n - 1), phase_of(n - 1));
    else
      store_last();
    port.await_stores();
  }
};

}  // namespace packkv
