// gdn_xcd.hpp -- which chain of tiles a workgroup of the scan kernels takes.
//
// Plain C++ for host and device, so that a host-only test can walk it.
#pragma once
#include <stdint.h>

#ifdef __HIPCC__
#define GDN_HOST_DEVICE __host__ __device__
#else
#define GDN_HOST_DEVICE
#endif

namespace gdn {

// Workgroups go to the 8 XCDs in turn, and each XCD has its own L2. Neighbouring
// column blocks share the lines that their pieces of a row end in (every piece,
// where the width is odd) and the DRAM pages, so an XCD takes runs of
// neighbouring chains, a sequence's column blocks at the most: runs in turn,
// then what is left in shorter ones. Measured against chains in turn: 4 x
// 4,097 x 2,048 bf16 forward and backward 168 against 176 us, 2 x 2,048 x 2,047
// 58 against 74; runs of several sequences lose, 64 x 512 x 2,048 115 against 102.
constexpr int kXcds = 8;
struct XcdRuns {
    int32_t chains, run, full, grid;  // run 0: chains in turn; full: chains in whole runs

    // ncb column blocks per sequence.
    static XcdRuns make(int64_t chains, int64_t ncb) {
        // not where whole chains would leave the XCDs unequal work
        if (chains % kXcds != 0 && chains < 8 * kXcds)
            return XcdRuns{(int32_t)chains, 0, 0, (int32_t)chains};
        const int64_t run = ncb < chains / kXcds ? ncb : chains / kXcds;
        const int64_t full = chains / (kXcds * run) * (kXcds * run);
        return XcdRuns{(int32_t)chains, (int32_t)run, (int32_t)full,
                       (int32_t)(full + (chains - full + kXcds - 1) / kXcds * kXcds)};
    }
    // The chain of workgroup i, or -1 (among the first `grid`, and for all behind them).
    GDN_HOST_DEVICE int chain(uint32_t i) const {
        if (i >= (uint32_t)grid) return -1;
        if (run == 0) return (int)i;
        const int x = i % kXcds, j = i / kXcds;
        if (i < (uint32_t)full) return (j / run * kXcds + x) * run + j % run;
        const int k = j - full / kXcds, each = (chains - full) / kXcds;
        const int more = (chains - full) % kXcds;
        if (k >= each + (x < more)) return -1;
        return full + x * each + (x < more ? x : more) + k;
    }
};

}  // namespace gdn
