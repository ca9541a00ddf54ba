// Every chain is taken by exactly one workgroup of a round, whatever the number of
// sequences and column blocks, and a round holds at most 7 workgroups more than chains.
#include <stdio.h>

#include <vector>

#include "../gated_deltanet_token_amd/csrc/gdn_xcd.hpp"

int main() {
    long bad = 0;
    for (int ncb = 1; ncb < 100; ++ncb)
        for (int n = 1; n < 100; ++n) {
            const int chains = n * ncb;
            const gdn::XcdRuns r = gdn::XcdRuns::make(chains, ncb);
            std::vector<int> taken(chains, 0);
            for (int i = 0; i < r.grid; ++i) {
                const int k = r.chain(i);
                if (k < -1 || k >= chains)
                    ++bad;
                else if (k >= 0)
                    ++taken[k];
            }
            for (int t : taken) bad += t != 1;
            bad += r.grid < chains || r.grid > chains + 7;
        }
    printf(bad ? "bad: %ld\n" : "xcd runs ok\n", bad);
    return bad != 0;
}
