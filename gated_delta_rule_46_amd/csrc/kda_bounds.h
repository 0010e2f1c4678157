// What a kernel makes of numbers that it reads back from a workspace: they are its own
// call's, unless the caller has given the workspace to two calls at once. Then the results
// are undefined, but no index formed from them may leave the call's arrays. (Nothing but
// arithmetic, so that a test on the host can go through it.)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// The number of the work that a workgroup takes, from a counter of which it found `counted`:
// all ones before the first. -1 where that is none of this launch's.
__host__ __device__ inline int drawn_work(uint32_t counted, uint32_t workgroups) {
    const uint32_t work = counted + 1u;
    return work < workgroups ? (int)work : -1;
}

// Whether workgroups `first` to `last` can have left the parts of an item that `wgs` share.
__host__ __device__ inline bool parts_exist(int first, int last, int wgs) { return first >= 0 && first <= last && last < wgs; }

}  // namespace kda
