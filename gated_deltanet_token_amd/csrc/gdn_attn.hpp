// gdn_attn.hpp -- device building blocks of the attention kernels (gfx950).
//
// Every product of attention and its gradients is formed the same way: a wave
// OWNS some rows (queries, or keys in the key and value gradients), 16 per
// column tile, and streams rows of the other side through LDS, 32 at a time:
//   scores^T [streamed x owned] = Y X^T   A: rows of the tile, natural order;
//                                         B: the owned rows, in registers
//   acc^T    [d x owned]       += Y^T P^T A: columns of the tile, chain order;
//                                         B: P^T as the accumulators hold it
// so a lane holds one owned row (column c = lane & 15 of every tile), the
// statistics of a row are per-lane scalars, and neither P nor the sums are ever
// moved between lanes (gdn_device.hpp has the fragment orders).
//
// Tiles lie in LDS row by row as copied (LDS-DMA), in chunks of 16 bytes whose
// place within the row is exchanged by the row number: 16 neighbouring rows'
// chunks c then lie in 16 different places, and both the natural reads (16 rows x
// 64 bytes) and the transposing ones (16 rows x 32 bytes) touch every bank
// equally often.
#pragma once
#include "gdn_device.hpp"
#include "gdn_attn_launch.hpp"

namespace gdn {

typedef __attribute__((address_space(3))) unsigned char lds_u8;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// s_waitcnt with only vmcnt(n) (n < 64), the other counters not waited for
template <int N> __device__ __forceinline__ void wait_copies() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
    asm volatile("" ::: "memory");
}

// The lane id through an empty asm: what is derived from it cannot be kept from one step to
// the next. LDS addresses are a few operations; kept, they would hold a dozen registers,
// which rows of more than 256 bytes do not have (up to there they are kept: the operations
// would be a fifth of the vector instructions).
template <bool YES = true> __device__ __forceinline__ int fresh(int lane) {
    if constexpr (YES) asm volatile("" : "+v"(lane));
    return lane;
}
template <typename DT, int D> constexpr bool kFresh = D * sizeof(DT) > 256;

// Allows a kernel its dynamic LDS on the current device.
template <typename K> hipError_t with_lds(K kernel, int bytes) {
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                               hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// A wave-uniform 64-bit value, in scalar registers (where the copies take their base).
__device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)x);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ const unsigned char *uniform(const unsigned char *p) {
    return reinterpret_cast<const unsigned char *>(uniform((int64_t)p));
}

// A tile of rows of D elements in LDS.
template <typename DT, int D> struct Rows {
    static constexpr int kChunk = 16 / (int)sizeof(DT);  // elements per 16 bytes
    static constexpr int kChunks = D / kChunk;           // chunks per row
    static constexpr int kPitch = D * (int)sizeof(DT);
    static constexpr int kCopies = 16 * kChunks / 64;    // wave copies per 16 rows

    static __device__ __forceinline__ int place(int row, int chunk) {
        return kChunks >= 16 ? chunk ^ (row & 15) : chunk ^ ((row >> 1) & 7);
    }
    static __device__ __forceinline__ int at(int row, int d) {  // byte offset of an element
        return row * kPitch + place(row, d / kChunk) * 16 + (d % kChunk) * (int)sizeof(DT);
    }

    // Copies 16 rows: row i from base + i * stride, rows from `rows` on as copies of the
    // last one (1 <= rows). Asynchronous: the caller waits for its copies.
    static __device__ __forceinline__ void copy16(const unsigned char *base, uint32_t stride,
                                                  int rows, unsigned char *lds, int lane) {
        const unsigned char *const from = uniform(base);
        lane = fresh<kFresh<DT, D>>(lane);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int p = i * 64 + lane, row = p / kChunks;
            const uint32_t off = (uint32_t)min(row, rows - 1) * stride +
                                 (uint32_t)place(row, p % kChunks) * 16;
            dma16_async(from, off, lds + i * 1024);
        }
    }

    // Natural fragment: row `row` (16 of them over the lanes' c), elements 32 kk + 8 g4 + e.
    static __device__ __forceinline__ Frag<DT> natural(const unsigned char *t, int row, int kk,
                                                       int g4) {
        Frag<DT> f;
        if constexpr (sizeof(DT) == 2) {
            f = *reinterpret_cast<const bf16x8 *>(t + row * kPitch +
                                                  place(row, 4 * kk + g4) * 16);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 x = *reinterpret_cast<const f32x4 *>(
                    t + row * kPitch + place(row, 8 * kk + 2 * g4 + h) * 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[4 * h + e] = x[e];
            }
        }
        return f;
    }
    // Chain fragment of column 16 dt + c: rows r0 + 4 g4 + e and r0 + 16 + 4 g4 + e. bf16:
    // two transposing reads, each of which hands lane i of 16 the four rows' element i.
    static __device__ __forceinline__ Frag<DT> chain(const unsigned char *t, int r0, int dt,
                                                     int c, int g4) {
        Frag<DT> f;
        if constexpr (sizeof(DT) == 2) {
            const int row = r0 + 4 * g4 + (c >> 2);
            const unsigned char *p =
                t + row * kPitch + place(row, 2 * dt + ((c >> 1) & 1)) * 16 + (c & 1) * 8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (lds_s16x4 *)(p + h * 16 * kPitch));
                const bf16x4 y = __builtin_bit_cast(bf16x4, x);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[4 * h + e] = y[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = r0 + 4 * g4 + (e & 3) + 16 * (e >> 2);
                f[e] = *reinterpret_cast<const float *>(t + at(row, 16 * dt + c));
            }
        }
        return f;
    }
    // Natural fragment of a row in global memory (elements 32 kk + 8 g4 + e).
    static __device__ __forceinline__ Frag<DT> load(const DT *row, int kk, int g4) {
        Frag<DT> f;
        ld_nat(row + 32 * kk + 8 * g4, f);
        return f;
    }
};

// Whether 16 bytes of elements hold an infinity or NaN, and the same with zeros for those.
__device__ __forceinline__ bool not_finite(const u32x4 &w, __bf16) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad |= (w[i] & 0x7F80u) == 0x7F80u || (w[i] & 0x7F800000u) == 0x7F800000u;
    return bad;
}
__device__ __forceinline__ bool not_finite(const u32x4 &w, float) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= (w[i] & 0x7F800000u) == 0x7F800000u;
    return bad;
}
__device__ __forceinline__ u32x4 only_finite(u32x4 w, __bf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u;
        if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0xFFFFu;
    }
    return w;
}
__device__ __forceinline__ u32x4 only_finite(u32x4 w, float) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] = 0;
    return w;
}
__device__ __forceinline__ bool is_finite(float x) {
    return (__builtin_bit_cast(uint32_t, x) & 0x7F800000u) != 0x7F800000u;
}

// Over the four lanes that hold one owned row (same c, every g4). A swap of a register's rows
// with those of its copy leaves each lane its own value and its partner's.
__device__ __forceinline__ float across_max(float x) {
    const uint32_t a = __builtin_bit_cast(uint32_t, x);
    const auto h = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const uint32_t h0 = h[0], h1 = h[1];
    x = fmaxf(__builtin_bit_cast(float, h0), __builtin_bit_cast(float, h1));
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    const auto w = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t w0 = w[0], w1 = w[1];
    return fmaxf(__builtin_bit_cast(float, w0), __builtin_bit_cast(float, w1));
}
__device__ __forceinline__ float across_sum(float x) {
    const uint32_t a = __builtin_bit_cast(uint32_t, x);
    const auto h = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const uint32_t h0 = h[0], h1 = h[1];
    x = __builtin_bit_cast(float, h0) + __builtin_bit_cast(float, h1);
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    const auto w = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t w0 = w[0], w1 = w[1];
    return __builtin_bit_cast(float, w0) + __builtin_bit_cast(float, w1);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Four neighbouring elements from fp32.
__device__ __forceinline__ void store4(__bf16 *p, const f32x4 &x) {
    bf16x4 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = (__bf16)x[e];
    *reinterpret_cast<bf16x4 *>(p) = y;
}
__device__ __forceinline__ void store4(float *p, const f32x4 &x) {
    *reinterpret_cast<f32x4 *>(p) = x;
}

// The softmax-weighted sums of a wave's queries, 16 CT of them, over the keys seen so far:
// with the reference mc (log2 units, any value near the row's maximum),
//   l = sum 2^(c s - mc),  acc = sum 2^(c s - mc) v,  c = scale log2(e).
// l is the lane's own part (its 8 of every 32 keys) until finish(). The reference moves
// only when a score passes it by more than 8, so that the sums are rescaled once or twice
// per row and not once per tile (2^8 of headroom costs fp32 nothing).
template <typename DT, int D, int CT, bool FRESH = kFresh<DT, D>> struct Attend {
    using R = Rows<DT, D>;
    f32x4 acc[D / 16][CT];
    float l[CT], mc[CT];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            l[ct] = 0.f;
            mc[ct] = -__builtin_inff();
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) acc[dt][ct] = zero4();
        }
    }

    // Fragments are read DEPTH steps ahead of the products that take them: an LDS read takes as
    // long as several products, and left alone the compiler reads just ahead of the use where
    // registers are short. Vector instructions may move across the fixed order.
    static __device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0x406); }

    // Scores of 16 NT keys (rows from r0 of the tile) against the queries q.
    template <int NT, int DEPTH = FRESH ? 1 : 0>
    static __device__ __forceinline__ void scores(const unsigned char *kt, int r0,
                                                  const Frag<DT> (&q)[D / 32][CT],
                                                  f32x4 (&s)[NT][CT], int lane) {
        lane = fresh<FRESH>(lane);
        const int c = lane & 15, g4 = lane >> 4;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) s[t][ct] = zero4();
        Frag<DT> a[DEPTH + 1][NT];
        auto read = [&](int kk) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
                a[kk % (DEPTH + 1)][t] = R::natural(kt, r0 + 16 * t + c, kk, g4);
        };
#pragma unroll
        for (int kk = 0; kk < DEPTH && kk < D / 32; ++kk) read(kk);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
            if (kk + DEPTH < D / 32) read(kk + DEPTH);
            if constexpr (DEPTH > 0) in_order();
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    s[t][ct] = mma(a[kk % (DEPTH + 1)][t], q[kk][ct], s[t][ct]);
            if constexpr (DEPTH > 0) in_order();
        }
    }

    // Keys from seen[ct] on (counted from the first) do not count for the lane's query.
    template <int NT>
    static __device__ __forceinline__ void mask(f32x4 (&s)[NT][CT], const int (&seen)[CT],
                                                int lane) {
        const int g4 = fresh<FRESH>(lane) >> 4;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (16 * t + 4 * g4 + r >= seen[ct]) s[t][ct][r] = -__builtin_inff();
    }

    // Moves the reference where a score passes it by more than 8.
    template <int NT> __device__ __forceinline__ void settle(const f32x4 (&s)[NT][CT], float c) {
        float top[CT];
        bool up = false;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            top[ct] = s[0][ct][0];
#pragma unroll
            for (int i = 1; i < 4 * NT; ++i) top[ct] = fmaxf(top[ct], s[i >> 2][ct][i & 3]);
            up |= fmaf(top[ct], c, -8.f) > mc[ct];
        }
        if (__any(up)) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                // a row by itself, whatever the others of the wave do: its bits are its own
                const float most = across_max(top[ct]);
                const bool moves = fmaf(most, c, -8.f) > mc[ct];
                const float m = moves ? most * c : mc[ct];
                const float f = moves ? exp2_fast(mc[ct] - m) : 1.f;  // 0 of nothing seen yet
                mc[ct] = m;
                l[ct] *= f;
#pragma unroll
                for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[dt][ct][r] *= f;
            }
        }
    }

    // Settled scores to weights; p as the B operands of the next product, rounded to the
    // tensors' type: off by half a step of each weight, which is sqrt(2) times the error of
    // rounding the result alone (bf16: 2.3e-3 of its norm and not 1.7e-3). The rest as a second
    // term (below) is not worth its products where these are what bounds: 8,192 tokens of 24/4
    // heads of 256 808 us, so 1,057; 2 x 8,192 of 16/4 heads of 128 525 and 710; 64 sequences
    // behind 32,768 shared tokens 113 and 126.
    template <int NT>
    __device__ __forceinline__ void weights(f32x4 (&s)[NT][CT], Frag<DT> (&p)[NT / 2][CT],
                                            float c) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const float m = mc[ct] == -__builtin_inff() ? 0.f : mc[ct];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    s[t][ct][r] = exp2_fast(fmaf(s[t][ct][r], c, -m));
                    l[ct] += s[t][ct][r];
                }
#pragma unroll
            for (int h = 0; h < NT / 2; ++h) c_to_frag(s[2 * h][ct], s[2 * h + 1][ct], p[h][ct]);
        }
    }

    // What the weights of 32 keys lose as operands in bf16, as operands too (together off by
    // 2^-17 at the most).
    static __device__ __forceinline__ void rest(const f32x4 (&s)[2][CT], const Frag<DT> (&p)[CT],
                                                Frag<DT> (&low)[CT]) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            f32x4 d[2];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i >> 2][i & 3] = s[i >> 2][ct][i & 3] - to_f32(p[ct][i]);
            c_to_frag(d[0], d[1], low[ct]);
        }
    }

    // acc += p v over the 32 keys.
    template <int DEPTH = FRESH ? 1 : 0>
    __device__ __forceinline__ void add(const unsigned char *vt, int r0, const Frag<DT> (&p)[CT],
                                        int lane) {
        add_to<DEPTH>(acc, vt, r0, p, lane);
    }
    template <int DEPTH = FRESH ? 1 : 0>
    static __device__ __forceinline__ void add_to(f32x4 (&acc)[D / 16][CT],
                                                  const unsigned char *vt, int r0,
                                                  const Frag<DT> (&p)[CT], int lane) {
        const Frag<DT> *const terms[1] = {p};
        add_terms<DEPTH>(acc, vt, r0, terms, lane);
    }
    // acc += (p_0 + .. + p_(N-1)) v.
    template <int DEPTH = FRESH ? 1 : 0, int N>
    static __device__ __forceinline__ void add_terms(f32x4 (&acc)[D / 16][CT],
                                                     const unsigned char *vt, int r0,
                                                     const Frag<DT> *const (&p)[N], int lane) {
        lane = fresh<FRESH>(lane);
        const int c = lane & 15, g4 = lane >> 4;
        constexpr int kStep = 2;  // columns of 16 per step
        Frag<DT> a[DEPTH + 1][kStep];
        auto read = [&](int i) {
#pragma unroll
            for (int j = 0; j < kStep; ++j)
                a[i % (DEPTH + 1)][j] = R::chain(vt, r0, kStep * i + j, c, g4);
        };
#pragma unroll
        for (int i = 0; i < DEPTH && i < D / 16 / kStep; ++i) read(i);
#pragma unroll
        for (int i = 0; i < D / 16 / kStep; ++i) {
            if (i + DEPTH < D / 16 / kStep) read(i + DEPTH);
            if constexpr (DEPTH > 0) in_order();
#pragma unroll
            for (int j = 0; j < kStep; ++j)
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        acc[kStep * i + j][ct] =
                            mma(a[i % (DEPTH + 1)][j], p[n][ct], acc[kStep * i + j][ct]);
            if constexpr (DEPTH > 0) in_order();
        }
    }

    // A weight of 0 times an infinity or NaN is NaN, so where a mask cuts a tile, values that are
    // not finite are taken out of the product (the caller clears them in the tile). Before
    // that, this makes NaN of the sums that they reach: seen as for mask(), for the 32 keys
    // from r0. How many of them a sum sees is a product of ones and zeros. Rare.
    __device__ __forceinline__ void mark_odd(const unsigned char *vt, int r0,
                                             const int (&seen)[CT], int lane) {
        lane = fresh<FRESH>(lane);
        const int c = lane & 15, g4 = lane >> 4;
        Frag<DT> sees[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sees[ct][e] =
                    from_f32<DT>(16 * (e >> 2) + 4 * g4 + (e & 3) < seen[ct] ? 1.f : 0.f);
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
            Frag<DT> a = R::chain(vt, r0, dt, c, g4);
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = from_f32<DT>(is_finite(to_f32(a[e])) ? 0.f : 1.f);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const f32x4 n = mma(a, sees[ct], zero4());
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (n[r] > 0.f) acc[dt][ct][r] = __builtin_nanf("");
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // The rows' whole sums of weights.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) l[ct] = across_sum(l[ct]);
    }
    __device__ __forceinline__ float lse(int ct) const {
        return l[ct] == 0.f ? -__builtin_inff() : mc[ct] * kLn2 + logf(l[ct]);
    }
};

// The keys [key0, key1) of one key head through a workgroup of NW waves, BK at a time, two
// tiles in LDS: the copies of one run behind the products on the other. `src(key, half)` names
// 16 rows: their first key's addresses, how many are there (at least 1: rows past them are
// copies of the last) and whether their page is bad (NaN scores). A lane's query sees the
// keys before lim[ct]; every query of the workgroup sees those before `common`, every query
// of the wave those before `lo`, none of the wave those from `hi` on.
struct KeyRows {
    const unsigned char *k, *v;
    int rows;
    bool bad;
};
template <typename DT, int D, int CT, int NW, int BK, bool FRESH = kFresh<DT, D>>
struct KeyTiles {
    using R = Rows<DT, D>;
    static constexpr int kTile = BK * R::kPitch;  // bytes of the keys or the values
    static constexpr int kLds = 4 * kTile;
    static constexpr int kGroups = BK / 16;
    static constexpr bool kAhead = D <= 128;  // registers for the scores of two tiles

    // Keys from `key` on into kb and values from `val` on into vb (either may be null), 16 rows
    // per wave and turn.
    template <typename Src>
    static __device__ __forceinline__ void issue(Src &src, int key, int val,
                                                 uint32_t stride, unsigned char *kb,
                                                 unsigned char *vb, int wave, int lane) {
#pragma unroll
        for (int g = 0; g < 2 * kGroups; g += NW) {
            const int i = __builtin_amdgcn_readfirstlane(g + wave);
            const bool keys = i < kGroups;
            if (i < 2 * kGroups && (keys ? kb : vb)) {
                const int half = i % kGroups;
                const KeyRows s = src((keys ? key : val) + 16 * half);
                R::copy16(keys ? s.k : s.v, stride, s.rows,
                          (keys ? kb : vb) + half * 16 * R::kPitch, lane);
            }
        }
    }
    template <typename Src>
    static __device__ __forceinline__ void issue(Src &src, int key, uint32_t stride,
                                                 unsigned char *buf, int wave, int lane) {
        issue(src, key, key, stride, buf, buf + kTile, wave, lane);
    }

    // Keys of a bad page have NaN scores.
    template <int NT, typename Src>
    static __device__ __forceinline__ void spoil(f32x4 (&s)[NT][CT], Src &src, int key) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (src(key + 16 * t).bad) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) s[t][ct] = zero4() + __builtin_nanf("");
            }
    }

    // The whole tiles that every query of the workgroup sees: n of them from key0. The scores
    // of a tile are formed beside the exponentials of the one before, so that a wave has
    // matrix and vector instructions to issue side by side: keys are one tile ahead of the
    // values.
    template <bool PAGED, typename Src>
    static __device__ __forceinline__ void run_whole(Attend<DT, D, CT, FRESH> &st,
                                                     const Frag<DT> (&q)[D / 32][CT],
                                                     Src &src, int key0, int n,
                                                     bool active, uint32_t stride, float scale2,
                                                     unsigned char *lds) {
        constexpr int NT = BK / 16;
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        unsigned char *const kb[2] = {lds, lds + kTile};
        unsigned char *const vb[2] = {lds + 2 * kTile, lds + 3 * kTile};
        issue(src, key0, key0, stride, kb[0], nullptr, wave, lane);
        wait_copies<0>();
        __syncthreads();
        issue(src, key0 + BK, key0, stride, n > 1 ? kb[1] : nullptr, vb[0], wave, lane);
        f32x4 s0[NT][CT], s1[NT][CT];
        st.template scores<NT, 0>(kb[0], 0, q, s0, lane);
        if constexpr (PAGED) spoil(s0, src, key0);
        st.settle(s0, scale2);
        // tile t: s of its scores, `next` for the following tile's
        auto step = [&](int t, f32x4 (&s)[NT][CT], f32x4 (&next)[NT][CT]) {
            wait_copies<0>();
            __syncthreads();
            const int key = key0 + t * BK;
            issue(src, key + 2 * BK, key + BK, stride, t + 2 < n ? kb[t & 1] : nullptr,
                  vb[(t + 1) & 1], wave, lane);
            if (!active) return;
            Frag<DT> p[NT / 2][CT];
            st.template scores<NT, 0>(kb[(t + 1) & 1], 0, q, next, lane);
            st.weights(s, p, scale2);
#pragma unroll
            for (int h = 0; h < NT / 2; ++h) st.template add<0>(vb[t & 1], 32 * h, p[h], lane);
            if constexpr (PAGED) spoil(next, src, key + BK);
            st.settle(next, scale2);
        };
        int t = 0;
        for (; t + 2 < n; t += 2) {
            step(t, s0, s1);
            step(t + 1, s1, s0);
        }
        if (t + 1 < n) {
            step(t, s0, s1);
            ++t;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) s0[i][ct] = s1[i][ct];
        }
        wait_copies<0>();
        __syncthreads();
        if (active) {
            Frag<DT> p[NT / 2][CT];
            st.weights(s0, p, scale2);
#pragma unroll
            for (int h = 0; h < NT / 2; ++h) st.template add<0>(vb[t & 1], 32 * h, p[h], lane);
        }
        __syncthreads();  // the tiles may be filled again
    }

    template <bool PAGED, typename Src>
    static __device__ __forceinline__ void run(Attend<DT, D, CT, FRESH> &st,
                                               const Frag<DT> (&q)[D / 32][CT], Src &src,
                                               int key0, int key1, const int (&lim)[CT],
                                               int common, int lo, int hi, uint32_t stride,
                                               float scale2, unsigned char *lds) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        if (key0 >= key1) return;
        if constexpr (kAhead) {
            const int n = (min(common, key1) - key0) / BK;
            if (n > 0) {
                run_whole<PAGED>(st, q, src, key0, n, hi > 0, stride, scale2, lds);
                key0 += n * BK;
                if (key0 >= key1) return;
            }
        }
        issue(src, key0, stride, lds, wave, lane);
        int parity = 0;
        for (int key = key0; key < key1; key += BK, parity ^= 1) {
            wait_copies<0>();
            __syncthreads();
            unsigned char *kt = lds + parity * 2 * kTile, *vt = kt + kTile;
            if (key + BK < key1)
                issue(src, key + BK, stride, lds + (parity ^ 1) * 2 * kTile, wave, lane);
            if (key + BK > common) {  // some query does not see all of the tile
                bool odd = false;
                for (int i = threadIdx.x; i < kTile / 16; i += 64 * NW)
                    odd |= not_finite(reinterpret_cast<const u32x4 *>(vt)[i], DT{});
                if (__syncthreads_or(odd)) {
#pragma unroll 1
                    for (int sub = 0; sub < BK && key + sub < hi; sub += 32) {
                        int seen[CT];
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) seen[ct] = lim[ct] - key - sub;
                        st.mark_odd(vt, sub, seen, lane);
                    }
                    __syncthreads();
                    for (int i = threadIdx.x; i < kTile / 16; i += 64 * NW) {
                        u32x4 &w = reinterpret_cast<u32x4 *>(vt)[i];
                        w = only_finite(w, DT{});
                    }
                    __syncthreads();
                }
            }
#pragma unroll 1
            for (int sub = 0; sub < BK; sub += 32) {
                const int k = key + sub;
                if (k < hi) {
                    f32x4 s[2][CT];
                    Frag<DT> p[1][CT];
                    st.scores(kt, sub, q, s, lane);
                    if constexpr (PAGED) spoil(s, src, k);
                    if (k + 32 > lo) {
                        int seen[CT];
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) seen[ct] = lim[ct] - k;
                        st.mask(s, seen, lane);
                    }
                    st.settle(s, scale2);
                    st.weights(s, p, scale2);
                    st.add(vt, sub, p[0], lane);
                }
            }
        }
    }
};

// The sequence of a packed batch whose tiles of M rows hold slot `slot`: sequence n's tiles
// start at slot floor(each * start / M) + n (`each` rows per token). 64 probes at a time.
// Offsets are clamped into [0, total], so malformed ones give meaningless results but address
// nothing outside the batch.
__device__ __forceinline__ int64_t clamped(const int32_t *cu, int n, int64_t total) {
    const int64_t a = cu[n];
    return a < 0 ? 0 : a > total ? total : a;
}
__device__ __forceinline__ int find_seq(const int32_t *cu, int N, int64_t total, int each,
                                        int M, int64_t slot, int lane) {
    int lo = 0, n = N;
    while (n > 1) {
        const int step = (n + 63) / 64, i = lo + lane * step;
        const bool in = lane * step < n && clamped(cu, i, total) * each / M + i <= slot;
        const int hits = __popcll(__ballot(in));
        const int skip = hits > 0 ? (hits - 1) * step : 0;
        lo += skip;
        n = min(step, n - skip);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Which (tile, head) a workgroup takes. Workgroups go to the 8 XCDs in turn, each with its
// own L2: an XCD takes whole heads, neighbouring ones, so that the query heads of a key head
// read its keys from one L2; the heads that are left over are dealt out tile by tile. Long
// tiles (the last queries, which see the most keys) come first.
struct HeadOrder {
    int tiles, each, rest, first;  // heads per XCD, left over; workgroups of those
    static HeadOrder make(int64_t units, int64_t tiles) {
        const int64_t each = units / 8, rest = units % 8;
        return HeadOrder{(int)tiles, (int)each, (int)rest,
                         (int)((rest * tiles + 7) / 8)};
    }
    int64_t grid() const { return 8 * ((int64_t)first + (int64_t)each * tiles); }
    __device__ __forceinline__ bool pick(uint32_t i, int &unit, int &tile) const {
        const int x = i & 7;
        int j = i >> 3;
        if (j < first) {
            const int64_t r = (int64_t)j * 8 + x;
            if (r >= (int64_t)rest * tiles) return false;
            tile = (int)(r / rest);
            unit = each * 8 + (int)(r % rest);
            return true;
        }
        j -= first;
        if (each == 0) return false;
        tile = j / each;
        unit = x * each + j % each;
        return tile < tiles;
    }
};

// The rows of one head of a sequence in memory order.
struct DenseKeys {
    const unsigned char *k, *v;  // the sequence's first row of this head
    int64_t stride;              // bytes
    int len;
    __device__ __forceinline__ KeyRows operator()(int key) const {
        const int first = min(key, len - 1);
        return KeyRows{k + first * stride, v + first * stride, min(16, len - first), false};
    }
};

// The tile of M rows that (unit, slot) of a HeadOrder names. Dense: units are sequences times
// heads, slots their tiles; packed: units are heads, slots those of find_seq.
struct SeqTile {
    int64_t tok0;
    int len, head, tile, tiles;  // tile >= tiles: none
};
template <int M>
__device__ __forceinline__ SeqTile seq_tile(const int32_t *cu, int N, int64_t T, int64_t total,
                                            int unit, int slot, int tiles, int heads, int lane) {
    SeqTile s;
    if (cu) {
        const int n = find_seq(cu, N, total, 1, M, slot, lane);
        s.tok0 = uniform(clamped(cu, n, total));
        const int64_t end = clamped(cu, n + 1, total);
        s.len = __builtin_amdgcn_readfirstlane(end > s.tok0 ? (int)(end - s.tok0) : 0);
        s.head = unit;
        s.tiles = (s.len + M - 1) / M;
        s.tile = __builtin_amdgcn_readfirstlane(slot - (int)(s.tok0 / M) - n);
        if (s.tile < 0) s.tile = s.tiles;  // malformed offsets
    } else {
        s.tok0 = unit / heads * T;
        s.len = (int)T;
        s.head = unit % heads;
        s.tiles = tiles;
        s.tile = slot;
    }
    return s;
}

}  // namespace gdn
