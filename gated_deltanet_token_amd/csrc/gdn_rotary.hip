// gdn_rotary.hip -- rotary positions, and appending keys and values to a paged
// cache with the rotation applied on the way (gfx950).
//
// Pair j of a head's first R columns, (x, y), turns by the angle
// pos[axis(j)] * freq[j]:  (x cos - y sin, y cos + x sin). Pairs are columns
// (j, j + R / 2), or neighbours (2j, 2j + 1). The inverse turns back, which is
// the gradient too, the rotation being orthogonal.
//
// A few operations per element: bound by HBM traffic, every element read and
// written once: 16,384 tokens of 16/16 heads of 128 44 us (6.1 TB/s), 16,385 into
// the cache, 24/4 heads of 256, 137 us (4.1 TB/s: rows of 512 bytes go to pages).
// A workgroup takes whole tokens: cos and sin of a token's pairs are formed
// once, for all of its heads, before the first row is asked for. Few tokens are
// bound by that and by the rows' round trips behind it: 64 tokens of 24/4 heads of
// 256 into the cache (912 items for 128 threads of each of 64 workgroups) 9.5 us.
// Angles are formed and reduced to a part of a turn in 64 bits (a position of a
// million times a frequency rounded in 32 bits would be off by 0.06 radians); cos
// and sin of the reduced angle in fp32 are off by at most 3 units of 2^-24.
#include "gdn_attn_launch.hpp"
#include "gdn_device.hpp"

namespace gdn {

namespace {

constexpr int kThreads = 128, kMaxTokens = 16;

template <typename DT, int VEC> struct Vec {
    typedef DT type __attribute__((ext_vector_type(VEC)));
};
template <typename DT> struct Vec<DT, 1> {
    typedef DT type;
};

template <typename DT, int VEC>
__device__ __forceinline__ void unpack(const typename Vec<DT, VEC>::type &v, float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        x[0] = to_f32(v);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] = to_f32(v[e]);
    }
}
template <typename DT, int VEC>
__device__ __forceinline__ typename Vec<DT, VEC>::type pack(const float (&x)[VEC]) {
    typename Vec<DT, VEC>::type v;
    if constexpr (VEC == 1) {
        v = from_f32<DT>(x[0]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = from_f32<DT>(x[e]);
    }
    return v;
}

// The last sequence that starts at or before token `tok` (the one it is in, if any).
__device__ __forceinline__ int seq_of(const int32_t *cu, int N, int64_t tok, int lane) {
    int lo = 0, n = N;
    while (n > 1) {
        const int step = (n + 63) / 64, i = lo + lane * step;
        const bool in = lane * step < n && cu[i] <= tok;
        const int hits = __popcll(__ballot(in));
        const int skip = hits > 0 ? (hits - 1) * step : 0;
        lo += skip;
        n = min(step, n - skip);
    }
    return lo;
}

// Each element is touched once (16,385 tokens into the cache, 24/4 heads of 256: 137 us with
// these hints, 145 without).
template <typename V> __device__ __forceinline__ V take(const void *p) {
    return __builtin_nontemporal_load(static_cast<const V *>(p));
}
template <typename V> __device__ __forceinline__ void give(void *p, const V &v) {
    __builtin_nontemporal_store(v, static_cast<V *>(p));
}

template <typename DT, int VEC, bool PAIRS>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryParams p, int per_wg) {
    using V = typename Vec<DT, VEC>::type;
    extern __shared__ float2 turn[];  // [per_wg][R / 2]: cos, sin
    __shared__ int64_t row_of[kMaxTokens];  // the token's row in the cache; -1: none
    __shared__ int64_t place[kMaxTokens];   // its place in its sequence
    __shared__ bool in_seq[kMaxTokens];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = p.R / 2;
    const int64_t tok0 = (int64_t)workgroup() * per_wg;
    if (tok0 >= p.tokens) return;
    const int here = (int)min((int64_t)per_wg, p.tokens - tok0);
    if (p.table) {
        for (int t = wave; t < here; t += kThreads / 64) {
            const int64_t tok = tok0 + t;
            int n;
            int64_t i;
            bool in = true;
            if (p.cu) {
                n = seq_of(p.cu, p.N, tok, lane);
                i = tok - p.cu[n];
                in = i >= 0 && tok < p.cu[n + 1];
            } else {
                n = (int)(tok / p.T);
                i = tok - n * p.T;
            }
            const int64_t at = p.lengths[n] + i, col = at >> p.page_shift;
            int64_t row = -1;
            if (in && at >= 0 && col < p.max_pages) {
                const int page = p.table[(int64_t)n * p.max_pages + col];
                if ((unsigned)page < (unsigned)p.num_pages)
                    row = ((int64_t)page << p.page_shift) + (at & ((1 << p.page_shift) - 1));
            }
            if (lane == 0) {
                row_of[t] = row;
                place[t] = at;
                in_seq[t] = in;
            }
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < here * half; i += kThreads) {
        const int t = i / half, j = i - t * half;
        const int axis = p.axis ? p.axis[j] : 0;
        float2 cs = make_float2(__builtin_nanf(""), __builtin_nanf(""));
        if ((unsigned)axis < (unsigned)p.axes) {
            const int64_t at = p.pos ? p.pos[axis * p.tokens + tok0 + t] : place[t];
            const double turns = (double)at * (double)p.freq[j] * 0.15915494309189533577;
            const float part = (float)(turns - rint(turns));
            sincospif(2.f * part, &cs.y, &cs.x);
            if (p.inverse) cs.y = -cs.y;
        }
        turn[i] = cs;
    }
    __syncthreads();

    // items: a pair of VEC columns (or VEC columns that hold their pairs) that turns, or VEC
    // columns that do not
    const int turning = PAIRS ? p.R / VEC : half / VEC, per_row = turning + (p.D - p.R) / VEC;
    const int copies = p.D / VEC;
    const int nq = p.q ? p.Hq * per_row : 0, nk = p.k ? p.Hk * per_row : 0;
    const int nv = p.v ? p.Hk * copies : 0, items = nq + nk + nv;
    const DT *const qs = static_cast<const DT *>(p.q), *const ks = static_cast<const DT *>(p.k),
                   *const vs = static_cast<const DT *>(p.v);
    for (int i = threadIdx.x; i < here * items; i += kThreads) {
        const int t = i / items;
        int it = i - t * items;
        const int64_t tok = tok0 + t, cached = p.table ? row_of[t] : -1;
        if (p.table && !in_seq[t]) continue;
        const DT *from;
        DT *to, *to2 = nullptr;
        if (it < nq + nk) {
            const bool key = it >= nq;
            if (key) it -= nq;
            const int head = it / per_row, heads = key ? p.Hk : p.Hq;
            it -= head * per_row;
            const int64_t at = (tok * heads + head) * p.D;
            from = (key ? ks : qs) + at;
            to = static_cast<DT *>(key ? p.k_out : p.q_out);
            if (to) to += at;
            if (key && cached >= 0) to2 = static_cast<DT *>(p.kc) + (cached * p.Hk + head) * p.D;
        } else {
            it -= nq + nk;
            const int head = it / copies;
            it -= head * copies;
            if (cached < 0) continue;
            from = vs + (tok * p.Hk + head) * p.D;
            to = static_cast<DT *>(p.vc) + (cached * p.Hk + head) * p.D;
            const int d = it * VEC;
            give<V>(to + d, take<V>(from + d));
            continue;
        }
        if (it >= turning) {
            const int d = p.R + (it - turning) * VEC;
            const V x = take<V>(from + d);
            if (to && to != from) give<V>(to + d, x);
            if (to2) give<V>(to2 + d, x);
            continue;
        }
        const float2 *cs = turn + t * half;
        if constexpr (PAIRS) {
            const int d = it * VEC;
            float x[VEC];
            unpack<DT, VEC>(take<V>(from + d), x);
#pragma unroll
            for (int e = 0; e + 1 < VEC; e += 2) {
                const float2 w = cs[(d + e) / 2];
                const float a = x[e], b = x[e + 1];
                x[e] = fmaf(a, w.x, -(b * w.y));
                x[e + 1] = fmaf(b, w.x, a * w.y);
            }
            const V y = pack<DT, VEC>(x);
            if (to) give<V>(to + d, y);
            if (to2) give<V>(to2 + d, y);
        } else {
            const int d = it * VEC;
            float a[VEC], b[VEC];
            unpack<DT, VEC>(take<V>(from + d), a);
            unpack<DT, VEC>(take<V>(from + half + d), b);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float2 w = cs[d + e];
                const float x = a[e], y = b[e];
                a[e] = fmaf(x, w.x, -(y * w.y));
                b[e] = fmaf(y, w.x, x * w.y);
            }
            const V x = pack<DT, VEC>(a), y = pack<DT, VEC>(b);
            if (to) {
                give<V>(to + d, x);
                give<V>(to + half + d, y);
            }
            if (to2) {
                give<V>(to2 + d, x);
                give<V>(to2 + half + d, y);
            }
        }
    }
}

template <typename DT, int VEC, bool PAIRS>
hipError_t launch(const RotaryParams &p, hipStream_t stream) {
    // whole tokens, about 512 items per workgroup
    const int rows = (p.q ? p.Hq : 0) + (p.k ? p.Hk : 0) + (p.v ? p.Hk : 0);
    const int64_t items = (int64_t)rows * p.D / VEC;
    int64_t per = 512 / (items < 1 ? 1 : items);
    per = per < 1 ? 1 : per > kMaxTokens ? kMaxTokens : per;
    const int64_t wgs = (p.tokens + per - 1) / per;
    rotary_kernel<DT, VEC, PAIRS>
        <<<grid_of(wgs, kThreads), kThreads, (size_t)per * (p.R / 2) * sizeof(float2), stream>>>(
            p, (int)per);
    return hipGetLastError();
}

template <typename DT> hipError_t by_width(const RotaryParams &p, hipStream_t stream) {
    constexpr int kMost = 16 / (int)sizeof(DT);
    if (p.pairs) {  // a chunk holds whole pairs
        if (p.R % kMost == 0) return launch<DT, kMost, true>(p, stream);
        return launch<DT, 2, true>(p, stream);
    }
    const int half = p.R / 2;  // both columns of a pair in chunks at the same place
    if (half % kMost == 0) return launch<DT, kMost, false>(p, stream);
    if constexpr (kMost > 4)
        if (half % 4 == 0) return launch<DT, 4, false>(p, stream);
    return launch<DT, 1, false>(p, stream);
}

}  // namespace

hipError_t launch_rotary(const RotaryParams &p, int dtype, hipStream_t stream) {
    return dtype == 1 ? by_width<__bf16>(p, stream) : by_width<float>(p, stream);
}

}  // namespace gdn
