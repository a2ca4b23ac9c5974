// status.cuh -- device side of the status block: word 0 is what happened (0: nothing unread), word 1 where.
#pragma once
#include <cstdint>

#include "sage_internal.h"

namespace sage {

// An expired wait replaces a bad index that nobody has read yet (later calls have to skip their work, and the caller has
// to learn that the workspace needs zeroing); of several expired waits the first one stays.
__device__ __forceinline__ void record_timeout(int32_t* status, int32_t where) {
  if (atomicExch(status, kStatusTimeout) != kStatusTimeout) atomicExch(status + 1, where);
}

// The first bad index stays recorded until the host reads it; nothing stops for it.  (`where` only over 0: a timeout
// that comes between the two keeps its own.)
__device__ __forceinline__ void record_bad_index(int32_t* status, int32_t where) {
  if (atomicCAS(status, 0, kStatusBadIndex) == 0) atomicCAS(status + 1, 0, where);
}

}  // namespace sage
