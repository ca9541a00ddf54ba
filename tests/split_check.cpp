// The scan kernels' bounds on the host (gdn_split.hpp): whatever the offsets of a packed batch and
// the counts from a counter hold, every slot that is written or looked at lies in the workspace;
// a wait that nothing ends gives up after its looks with NaN; one that ends gives the state that
// walking the tiles gives, however far it had to look.
#include <stdio.h>

#include <initializer_list>
#include <utility>
#include <vector>

#include "../gated_deltanet_token_amd/csrc/gdn_split.hpp"

using namespace gdn;
static long bad = 0;
static uint32_t seed = 1;
static uint32_t rnd() { return seed = seed * 1664525u + 1013904223u, seed >> 8; }

static void check_slots(const std::vector<int32_t> &cu, int64_t total, int tile) {
    const int N = (int)cu.size() - 1;
    const int64_t slots = total / tile + N;
    for (int count : {-2147483647 - 1, -1, 0, 1, (int)slots - 1, (int)slots, (int)slots + 1,
                      2147483647})
        for (bool back : {false, true}) {
            const int64_t k = counted_tile(count, slots, back);
            bad += (count >= 0 && count < slots) != (k >= 0) || k >= slots;
        }
    bad += counted_tile(0, slots, false) != 0 || counted_tile(0, slots, true) != slots - 1;
    for (int n = 0; n < N; ++n) {
        int64_t base, len;
        clamp_sequence(cu[n], cu[n + 1], total, base, len);
        bad += base < 0 || len < 0 || base + len > total;
        const int64_t first = first_slot(base, n, tile), last = len > 0 ? (len - 1) / tile : 0;
        bad += first < 0 || first + last >= slots;
        // a workgroup that takes slot k for sequence n looks only where the sequence has tiles
        for (int64_t k = 0; k < slots; ++k) {
            const int64_t mine = k - first;
            if (mine < 0 || mine * tile >= len) continue;  // publishes slot k and leaves
            bad += mine > last;
            if (mine > 0) bad += k - 1 < 0 || k - mine < 0;                // forward
            if (mine < last) bad += k + 1 >= slots || k + (last - mine) >= slots;  // backward
        }
    }
}

template <int DEPTH> static void check_wait() {
    const int tiles = 9;
    std::vector<float> A(tiles), H(tiles);
    for (int i = 0; i < tiles; ++i) A[i] = 0.5f + 0.01f * i, H[i] = 1.0f - 0.3f * i;
    std::vector<float> want(tiles + 1, 0.25f);  // behind i tiles
    for (int i = 0; i < tiles; ++i) want[i + 1] = fmaf(A[i], want[i], H[i]);
    const auto word = [](float x) { return __builtin_bit_cast(uint32_t, x); };
    for (int mine = 1; mine < tiles; ++mine)
        for (int known = 0; known <= mine; ++known)  // `known` tiles have their state published
            for (int maps = 0; maps < (1 << mine); ++maps) {
                int looks = 0, pauses = 0;
                const float got = await_state<DEPTH>(
                    mine, 5,
                    [&](int j, uint32_t &state, uint64_t &map) {
                        const int i = mine - 1 - j;
                        bad += j < 0 || i < 0;
                        ++looks;
                        state = i < known ? word(want[i + 1]) : kAbsent;
                        map = maps >> i & 1 ? (uint64_t)word(H[i]) << 32 | word(A[i])
                                            : ~(uint64_t)0;
                    },
                    [&] { ++pauses; });
                bool ends = false;  // a state among the nearest DEPTH and all maps behind it
                for (int i = mine - 1, all = 1; i >= 0 && i >= mine - DEPTH; --i) {
                    if (i < known) {
                        ends = all;
                        break;
                    }
                    all &= maps >> i & 1;
                }
                bad += ends ? word(got) != word(want[mine]) || pauses != 0 || looks != DEPTH
                            : got == got || pauses != 5 || looks != 5 * DEPTH;
            }
}

int main() {
    const int tile = 128;
    for (int round = 0; round < 3000; ++round) {
        const int N = 1 + rnd() % 12;
        const int64_t total = rnd() % 2000;
        std::vector<int32_t> cu(N + 1);
        for (int i = 0; i <= N; ++i) cu[i] = (int32_t)(rnd() % (total + 1));
        if (round % 3 == 0) {  // well formed
            for (int i = 0; i <= N; ++i)
                for (int j = 0; j < i; ++j)
                    if (cu[j] > cu[i]) std::swap(cu[i], cu[j]);
            cu[0] = 0;
            cu[N] = (int32_t)total;
            int64_t before = -1;  // first slots rise, and no sequence's tiles pass the next one's
            for (int n = 0; n < N; ++n) {
                const int64_t first = first_slot(cu[n], n, tile);
                bad += first <= before;
                const int64_t tiles = (cu[n + 1] - cu[n] + tile - 1) / tile;
                before = first + (tiles > 0 ? tiles : 1) - 1;
            }
            bad += before >= total / tile + N;
        } else if (round % 3 == 1) {  // anything
            for (int i = 0; i <= N; ++i)
                if (rnd() % 3 == 0) cu[i] = (int32_t)(rnd() * 2654435761u);
        }
        check_slots(cu, total, tile);
    }
    check_wait<1>();
    check_wait<2>();
    check_wait<4>();
    printf(bad ? "bad: %ld\n" : "bounds ok\n", bad);
    return bad != 0;
}
