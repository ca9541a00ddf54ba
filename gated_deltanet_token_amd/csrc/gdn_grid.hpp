// gdn_grid.hpp -- launches of more workgroups than one dimension holds.
//
// A dispatch counts its threads per dimension in 32 bits: 2^24 workgroups of 256
// threads are too many for x alone. Such a launch gets rows of workgroups in y,
// as few and as equal as possible; the last workgroups of the last row may have
// nothing to do. Plain C++ for the host, so that a host-only test can walk it.
#pragma once
#include <stdint.h>

namespace gdn {

struct GridShape {
    uint32_t x, y;
};
// Rows for n workgroups (1 <= n < 2^31) of up to 1,024 threads.
static inline GridShape grid_shape(int64_t n, int threads) {
    const int64_t most = 0xFFFFFFFFll / threads, rows = (n + most - 1) / most;
    return GridShape{(uint32_t)((n + rows - 1) / rows), (uint32_t)rows};
}

#ifdef __HIPCC__
// The number of a workgroup of such a launch, which may be n or above.
__device__ __forceinline__ uint32_t workgroup() {
    return blockIdx.y == 0 ? blockIdx.x : blockIdx.y * gridDim.x + blockIdx.x;
}
static inline dim3 grid_of(int64_t n, int threads) {
    const GridShape g = grid_shape(n, threads);
    return dim3(g.x, g.y);
}
#endif

}  // namespace gdn
