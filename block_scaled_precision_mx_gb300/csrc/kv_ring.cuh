// kv_ring.cuh -- which phase of its barrier a ring slot's last fill completes.
//
// Item i of a ring goes to slot i % slots as that slot's fill i / slots, and a slot's barrier starts in phase 0.
// Host and device; nothing else is included, so that it can be tested by itself.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MXGB_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MXGB_HOST_DEVICE inline
#endif

namespace mxgb {

// After `issued` items (those that were really issued: a loader that gave up in front of one does not count it),
// the parity of the phase that the last fill of `slot` completes.  slot < issued.
MXGB_HOST_DEVICE uint32_t kv_ring_last_parity(uint32_t issued, uint32_t slot, uint32_t slots) {
  return ((issued - 1 - slot) / slots) & 1;
}

}  // namespace mxgb
