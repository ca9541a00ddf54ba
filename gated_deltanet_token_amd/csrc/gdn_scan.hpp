// gdn_scan.hpp -- device-side pieces of the gated linear recurrence kernels:
// vector access, the gates, and the tile shape.
#pragma once
#include "gdn_device.hpp"
#include "gdn_ops_launch.hpp"
#include "gdn_split.hpp"

namespace gdn {

// VEC neighbouring elements in their storage type, as the words they are
// loaded in (a struct of bf16 members would take a register for each).
template <typename DT, int VEC> struct Raw {
    static constexpr int kWords = VEC * (int)sizeof(DT) < 4 ? 1 : VEC * (int)sizeof(DT) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (sizeof(DT) == 4) return __builtin_bit_cast(float, w[e]);
        return __builtin_bit_cast(float, e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    }
    // Elements e and e + 1 (VEC == 1: e alone).
    __device__ __forceinline__ void set(int e, float a, float b) {
        if constexpr (sizeof(DT) == 4) {
            w[e] = __builtin_bit_cast(uint32_t, a);
            if constexpr (VEC > 1) w[e + 1] = __builtin_bit_cast(uint32_t, b);
        } else {
            typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
            w[e / 2] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
        }
    }
};
template <int N> struct Words {
    typedef uint32_t type __attribute__((ext_vector_type(N)));
};
template <> struct Words<1> { typedef uint32_t type; };

// VEC elements `bytes` behind base: 32-bit byte offsets within a tile
// (kMaxScanWidth keeps them in range), so that the tile's start stays in scalar
// registers.
template <int VEC, typename DT>
__device__ __forceinline__ Raw<DT, VEC> load_raw(const DT *base, uint32_t bytes) {
    const char *p = reinterpret_cast<const char *>(base) + bytes;
    Raw<DT, VEC> r;
    if constexpr (VEC * sizeof(DT) == 2) {
        r.w[0] = *reinterpret_cast<const uint16_t *>(p);
    } else {
        typedef typename Words<Raw<DT, VEC>::kWords>::type V;
        const V v = __builtin_nontemporal_load(reinterpret_cast<const V *>(p));
        __builtin_memcpy(r.w, &v, sizeof(v));
    }
    return r;
}
template <typename DT, int VEC>
__device__ __forceinline__ void store_raw(DT *base, uint32_t bytes, const Raw<DT, VEC> &r) {
    char *p = reinterpret_cast<char *>(base) + bytes;
    if constexpr (VEC * sizeof(DT) == 2) {
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)r.w[0];
    } else {
        typedef typename Words<Raw<DT, VEC>::kWords>::type V;
        V v;
        __builtin_memcpy(&v, r.w, sizeof(v));
        __builtin_nontemporal_store(v, reinterpret_cast<V *>(p));
    }
}
// VEC values in type DT.
template <typename DT, int VEC>
__device__ __forceinline__ Raw<DT, VEC> pack(const float (&x)[VEC]) {
    Raw<DT, VEC> r;
#pragma unroll
    for (int e = 0; e < VEC; e += 2) r.set(e, x[e], x[VEC > 1 ? e + 1 : 0]);
    return r;
}
template <typename DT> __device__ __forceinline__ const DT *as(const void *p, int64_t at) {
    return static_cast<const DT *>(p) + at;
}
template <typename DT> __device__ __forceinline__ DT *as(void *p, int64_t at) {
    return static_cast<DT *>(p) + at;
}

// Makes the compiler forget what it derived from x: what is needed behind this
// is computed anew instead of being kept in registers across a barrier.
template <typename DT, int VEC, int R>
__device__ __forceinline__ void forget(Raw<DT, VEC> (&x)[R]) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < Raw<DT, VEC>::kWords; ++i) asm volatile("" : "+v"(x[r].w[i]));
}

// Gates of fp32 logits: e^z for z in [-110, 80] (held there outside), the
// product z log2(e) carried in two terms (Cody and Waite's reduction in base
// 2): a plain product would be off by |z| 2^-24, and the small gates 1 - alpha
// inherit that error whole.
__device__ __forceinline__ float exp_logit(float z, float) {
    constexpr float kLog2e = 0x1.715476p+0f, kLog2eLow = 0x1.4ae0bep-26f, kLn2 = 0x1.62e430p-1f;
    z = z > 80.f ? 80.f : z;  // keeps 1 + e^z finite; a NaN stays one
    z = z < -110.f ? -110.f : z;  // e^z is 0 there, and the product stays finite
    const float t = z * kLog2e;
    const float low = fmaf(z, kLog2eLow, fmaf(z, kLog2e, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, low * kLn2, e);
}
// Of bf16 logits: the plain product. Its error, |z| 2^-24 at the most, is far
// below that of the outputs' rounding to bf16 (2^-9), and the forward kernel is
// short of vector instructions.
__device__ __forceinline__ float exp_logit(float z, __bf16) {
    return __builtin_amdgcn_exp2f((z > 80.f ? 80.f : z) * 0x1.715476p+0f);
}

// s = 1 / (1 + e^z) and its complement e^z / (1 + e^z): the reciprocal takes
// one Newton step, because the errors of an alpha near 1 add up over its
// memory of 1 / (1 - alpha) tokens.
template <typename DT> __device__ __forceinline__ void sigmoid_pair(float z, float &s, float &c) {
    const float e = exp_logit(z, DT());
    const float d = 1.f + e;
    float r = __builtin_amdgcn_rcpf(d);
    r = fmaf(r, fmaf(-d, r, 1.f), r);
    s = r;
    c = e * r;
}

// beta = 1 / (1 + e^-b), whose errors do not add up: of a bf16 logit without
// the Newton step (the reciprocal is good to a unit of 2^-23).
__device__ __forceinline__ float write_strength(float b, float) {
    float s, c;
    sigmoid_pair<float>(-b, s, c);
    return s;
}
__device__ __forceinline__ float write_strength(float b, __bf16) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(b * -0x1.715476p+0f));
}

// The same with 1 - beta, for its gradient beta (1 - beta).
__device__ __forceinline__ void write_pair(float b, float &beta, float &rest, float) {
    sigmoid_pair<float>(-b, beta, rest);
}
// 1 - beta = e^-b beta of a bf16 logit.
__device__ __forceinline__ float write_rest(float b, float beta) {
    // e^-b may be infinite where beta is 0
    return fminf(__builtin_amdgcn_exp2f(b * -0x1.715476p+0f), 0x1p127f) * beta;
}
__device__ __forceinline__ void write_pair(float b, float &beta, float &rest, __bf16) {
    beta = write_strength(b, __bf16());
    rest = write_rest(b, beta);
}

// Gates of one element from what the caller passes: the decay, its complement
// and the write strength (tied: the complement).
template <typename DT, bool TIED, bool LOGITS>
__device__ __forceinline__ void gates(float a, float b, float &alpha, float &keep, float &beta) {
    if constexpr (LOGITS) {
        sigmoid_pair<DT>(a, alpha, keep);
        if constexpr (!TIED) beta = write_strength(b, DT());
    } else {
        alpha = a;
        keep = 1.f - a;
        beta = b;
    }
    if constexpr (TIED) beta = keep;
}

// A tile is kRows tokens by kCols channels on kThreads threads. kLanes
// neighbouring lanes hold one token's kCols channels, VEC each; the kGroups
// groups of them hold kPer consecutive tokens each. Rows that start off 8 or 16
// bytes are read in pairs of bf16 where the width is even: what such rows cost
// is their segments that straddle cache lines, and a pair's are 256 bytes long
// (5 x 2,143 x 7,764 186 us, 226 one by one in segments of 128 bytes, 229 in
// fours of the same length; a width of 7,808 128).
template <typename DT, int VEC> struct ScanShape {
    static constexpr int kThreads = VEC <= 2 ? 1024 : 512;
    static constexpr int kRows = GDN_SCAN_TILE;
    static constexpr int kLanes = VEC <= 2 ? 64 : 16;
    static constexpr int kCols = kLanes * VEC;
    static constexpr int kGroups = kThreads / kLanes;
    static constexpr int kPer = kRows / kGroups;
    static_assert(kGroups * kPer == kRows, "tile shape");
};

// First token and length of sequence n, clamped into the batch.
__device__ __forceinline__ void scan_bounds(const ScanParams &p, int n, int64_t &base,
                                            int64_t &len) {
    if (p.cu) {
        clamp_sequence(p.cu[n], p.cu[n + 1], p.total, base, len);
    } else {
        base = (int64_t)n * p.T;
        len = p.T;
    }
}

// Row of the prefix states of sequence n's block 0.
__device__ __forceinline__ int64_t scan_prefix_row(const ScanParams &p, int n, int64_t base) {
    return p.cu ? base / p.prefix_len + n : (int64_t)n * (p.T / p.prefix_len);
}

// Block that ends at token t, a multiple of 64 (the blocks are 64 m tokens):
// its index, or -1 when no block ends there.
__device__ __forceinline__ int64_t scan_block_ending(const ScanParams &p, int64_t t) {
    const uint32_t units = (uint32_t)(t >> 6), per = (uint32_t)(p.prefix_len >> 6);
    const uint32_t i = units / per;
    return i * per == units ? (int64_t)i - 1 : -1;
}

// Tiles of one sequence side by side (SPLIT kernels)
//
// A workgroup takes one tile: it loads it and sums it up (A and H of every
// channel), finds the state in front of it, publishes the state behind it,
// A * (state in front) + H, and only then walks its tokens. So a chain of tiles
// advances by one published word per channel and tile, while all else of the
// tiles overlaps.
//
// With SPLIT > 1 a tile also publishes its A and H as soon as it knows them, and
// looks at SPLIT tiles in front of it at once for the nearest published state,
// to carry it over the maps in between itself. Every state is formed the same
// way by whoever forms it, so the result does not depend on how far a
// workgroup had to look.
//
// A value and its presence travel in one word (all bits set: not there yet; the
// launch's first kernel sets them), written and read by relaxed atomics of
// device scope, so no fence orders them.
//
// Workgroups take the tiles of a chain in order from a counter. A tile waits
// only for tiles of its chain that were taken before it, by workgroups that run
// already and in turn wait only for earlier ones, and every taken tile
// publishes: every wait ends. A wait is bounded all the same (about 3 s, where
// a right one takes microseconds) and a count from the counter is checked: two
// calls that a caller lets overlap on one workspace neither hang nor leave the
// buffers. Their results are undefined: NaN, tiles left out, or finite values
// made from the other call's words.
struct ScanSplit {
    uint32_t *ticket;  // [chains]
    uint64_t *map;     // [slots][width], SPLIT > 1: A low, H high
    uint32_t *state;   // [slots][width]
    XcdRuns runs;      // chains: N * column blocks (dense) or column blocks (packed)
    int32_t slots;     // dense: tiles * N (tile-major), packed: floor(total / tile) + N
    int32_t width;     // columns, up to whole column blocks
    int32_t deep;      // the kernels' SPLIT
    int64_t per_chain; // workgroups that take a chain's tiles
};

constexpr int kScanSpins = 1 << 22;  // looks of about 0.7 us

// A value's bits; any NaN becomes the plain one, never kAbsent.
__device__ __forceinline__ uint32_t scan_word(float x) {
    return x == x ? __builtin_bit_cast(uint32_t, x) : 0x7FC00000u;
}
template <typename T> __device__ __forceinline__ void publish(T *p, T v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T> __device__ __forceinline__ T observe(const T *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish_state(const ScanSplit &sp, int64_t slot, int col, float x) {
    publish(sp.state + slot * sp.width + col, scan_word(x));
}
__device__ __forceinline__ void publish_map(const ScanSplit &sp, int64_t slot, int col, float A,
                                            float H) {
    publish(sp.map + slot * sp.width + col, (uint64_t)scan_word(H) << 32 | scan_word(A));
}

// The state in front of a tile: `ahead` (at least 1) tiles of its sequence lie
// in front, at slots `at`, at + step, ... (step is positive for the backward
// pass, whose tiles come from the end).
template <int SPLIT>
__device__ __forceinline__ float find_state(const ScanSplit &sp, int64_t at, int64_t step,
                                            int32_t ahead, int col) {
    return await_state<SPLIT>(
        ahead, kScanSpins,
        [&](int j, uint32_t &state, uint64_t &map) {
            const int64_t i = (at + j * step) * sp.width + col;
            state = observe(sp.state + i);
            map = ~(uint64_t)0;
            if constexpr (SPLIT > 1) map = observe(sp.map + i);
        },
        [] { __builtin_amdgcn_s_sleep(1); });
}

__device__ __forceinline__ int64_t scan_first_slot(const ScanParams &p, int n) {
    int64_t base, len;
    clamp_sequence(p.cu[n], p.total, p.total, base, len);
    return first_slot(base, n, GDN_SCAN_TILE);
}

// The sequence of a slot: the last one that starts at or before it, looked for
// by the whole workgroup, which probes as many sequences at once as it has
// threads (a binary search by one thread would be a chain of loads in front of
// every tile). s_found[0] starts at 0, and every thread reaches this call.
__device__ __forceinline__ int scan_slot_sequence(const ScanParams &p, int64_t slot,
                                                  int *s_found) {
    int lo = 0, size = p.N, turn = 0;
    while (size > 1) {
        const int step = (size + (int)blockDim.x - 1) / (int)blockDim.x;
        const int at = (int)threadIdx.x * step;
        if (threadIdx.x == 0) s_found[turn ^ 1] = 0;  // of the round after this one
        if (at > 0 && at < size && scan_first_slot(p, lo + at) <= slot)
            atomicMax(s_found + turn, at);
        __syncthreads();
        const int found = __builtin_amdgcn_readfirstlane(s_found[turn]);
        lo += found;
        size = min(step, size - found);
        turn ^= 1;
        __syncthreads();
    }
    return lo;
}

}  // namespace gdn
