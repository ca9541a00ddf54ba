// Launches of many workgroups (gdn_grid.hpp): threads per dimension stay below 2^32, rows
// below 2^16, every workgroup has a number, and fewer numbers than rows are left over. Chains
// (gdn_xcd.hpp): numbers past a round's end have none.
#include <stdio.h>

#include <initializer_list>

#include "../gated_deltanet_token_amd/csrc/gdn_grid.hpp"
#include "../gated_deltanet_token_amd/csrc/gdn_xcd.hpp"

int main() {
    long bad = 0;
    for (int threads : {64, 256, 512, 640, 1024})
        for (int shift = 0; shift < 31; ++shift)
            for (int64_t off = -3; off <= 3; ++off) {
                const int64_t n = ((int64_t)1 << shift) + off;
                if (n < 1) continue;
                const gdn::GridShape g = gdn::grid_shape(n, threads);
                const int64_t all = (int64_t)g.x * g.y;
                bad += (int64_t)g.x * threads > 0xFFFFFFFFll || g.y > 65535 || g.y < 1;
                bad += all < n || all - n >= g.y || all > 0xFFFFFFFFll;
                bad += n * threads <= 0xFFFFFFFFll && (g.y != 1 || g.x != n);
            }
    const gdn::GridShape most = gdn::grid_shape(0x7FFFFFFF, 1024);
    bad += (int64_t)most.x * 1024 > 0xFFFFFFFFll || most.y > 65535;
    for (int64_t chains : {1ll, 7ll, 9ll, 64ll, 65ll, 4194309ll, 2147483000ll})
        for (int64_t ncb : {1ll, 3ll, 64ll}) {
            if (chains % ncb) continue;
            const gdn::XcdRuns r = gdn::XcdRuns::make(chains, ncb);
            for (int64_t i = (int64_t)r.grid; i < (int64_t)r.grid + 70; ++i)
                bad += r.chain((uint32_t)i) != -1;
            bad += r.chain(0xFFFFFFFFu) != -1;
        }
    printf(bad ? "bad: %ld\n" : "grids ok\n", bad);
    return bad != 0;
}
