// gdn_split.hpp -- what keeps the scan kernels that are cut along time inside their
// workspace and from waiting for ever: the bounds of a sequence, the tile of a
// count, and the wait for the state in front of a tile.
//
// Plain C++ for host and device, so that a host-only test can walk it.
#pragma once
#include <math.h>
#include <stdint.h>

#include "gdn_xcd.hpp"

namespace gdn {

constexpr uint32_t kAbsent = 0xFFFFFFFFu;  // a state or half a map that is not there yet

// First token and length of a packed sequence from its two offsets, clamped into the
// batch whatever they hold.
GDN_HOST_DEVICE inline void clamp_sequence(int64_t lo, int64_t hi, int64_t total, int64_t &base,
                                           int64_t &len) {
    base = lo < 0 ? 0 : (lo > total ? total : lo);
    len = (hi < base ? base : (hi > total ? total : hi)) - base;
}

// First slot of packed sequence n that starts at token base: it owns as many from
// there on as it has tiles, and at least one (a sequence without tokens has its
// state handed on there). floor(total / tile) + N slots hold them all.
GDN_HOST_DEVICE inline int64_t first_slot(int64_t base, int n, int tile) { return base / tile + n; }

// The tile of a chain that a count from its counter stands for, or -1: counts are
// 0 to per_chain - 1 unless something else writes to the workspace.
GDN_HOST_DEVICE inline int64_t counted_tile(int count, int64_t per_chain, bool back) {
    if (count < 0 || count >= per_chain) return -1;
    return back ? per_chain - 1 - count : count;
}

// The state in front of a tile with `ahead` (at least 1) tiles of its sequence in
// front of it. look(j, state, map) reads the words of the j-th of them (0 the
// nearest), pause() passes some time. NaN after `spins` looks without success.
template <int DEPTH, typename Look, typename Pause>
GDN_HOST_DEVICE inline float await_state(int32_t ahead, int spins, const Look &look,
                                         const Pause &pause) {
    for (int spin = 0; spin < spins; ++spin) {
        uint32_t state[DEPTH];
        uint64_t map[DEPTH];
#pragma unroll
        for (int j = 0; j < DEPTH; ++j) look(j < ahead ? j : ahead - 1, state[j], map[j]);
        float c = 0.f;
        bool found = false;
#pragma unroll
        for (int j = DEPTH - 1; j >= 0; --j) {
            if (j >= ahead) continue;
            if (state[j] != kAbsent) {
                c = __builtin_bit_cast(float, state[j]);
                found = true;
            } else {
                found &= map[j] != ~(uint64_t)0;
                c = fmaf(__builtin_bit_cast(float, (uint32_t)map[j]), c,
                         __builtin_bit_cast(float, (uint32_t)(map[j] >> 32)));
            }
        }
        if (found) return c;
        pause();
    }
    return __builtin_nanf("");
}

}  // namespace gdn
