// The check of an accepted path's nodes (pva_kvcache_accept), apart from the kernel
// so that a host compiler takes it too: what it lets pass bounds the kernel's
// look-ups, whatever the rest of the path holds.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PVA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PVA_HOST_DEVICE inline
#endif

namespace pva {

// Whether node i of a path may be looked up: rows past + path[i] and past + i then
// lie in [0, rows).  past >= 0.  A rising path from 0 on has path[i] >= i
// throughout, but each thread sees only its own node and the one before, so that is
// asked here too.
PVA_HOST_DEVICE bool path_node_ok(const int32_t* path, int i, int past, long long rows) {
  const int x = path[i];
  return x >= i && (i == 0 || path[i - 1] < x) && past + (long long)x < rows;
}

}  // namespace pva
