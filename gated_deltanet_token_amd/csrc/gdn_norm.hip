// gdn_norm.hip -- root-mean-square norm with the residual's addition and an
// output in 8 bits with scales (gfx950), and its gradients.
//
//   r = x + residual,  s = 1 / sqrt(mean(r^2) + eps),  y = r s w
//   out8 = e4m3(y / scale),  scale = max |y| / 448 per row or 128 columns
//   dr = s (w dy - u mean(w dy u)) + dresidual,  dw = sum over rows of dy u,  u = r s
//
// A handful of operations per element: bound by HBM traffic, each row read
// once and held in registers between the sum of squares and the outputs.
//
// Mapping: a thread holds chunks of 8 neighbouring columns (16 bytes of bf16).
// 16 threads share a row of up to 128 columns, a wave one of up to 512 (1,024 in
// the backward pass), and a workgroup a wider one, so that a 128-column group is
// always 16 neighbouring lanes and its maximum one DPP row reduction.
#include "gdn_device.hpp"
#include "gdn_ops_launch.hpp"

namespace gdn {

namespace {

constexpr float kScaleFloor = 0x1p-100f;  // groups of zeros keep a finite scale and its inverse

// 1 / sqrt(x) to about a unit in its last place: the instruction's value and one
// Newton step (x > 0: a mean of squares and eps).
__device__ __forceinline__ float inv_sqrt(float x) {
    const float s = __builtin_amdgcn_rsqf(x);
    return s * fmaf(-0.5f * x * s, s, 1.5f);
}

__device__ __forceinline__ float row16_max(float x) {
    x = fmaxf(x, GDN_DPP(x, 0xB1));
    x = fmaxf(x, GDN_DPP(x, 0x4E));
    x = fmaxf(x, GDN_DPP(x, 0x141));
    x = fmaxf(x, GDN_DPP(x, 0x140));
    return x;
}

// The scale of a group whose largest magnitude is `most`: most / 448, rounded once
// (the product with the inverse in two terms, both positive for an infinity).
__device__ __forceinline__ float e4m3_scale(float most) {
    constexpr float high = (float)(1.0 / 448.0 - 0x1p-33), low = (float)(1.0 / 448.0 - (double)high);
    static_assert(low >= 0.f, "inf - inf");
    return fmaxf(fmaf(most, high, most * low), kScaleFloor);
}

// The row's s as a power of two times `rest`, in [4, 8) (NaN of a NaN).
struct RowScale {
    float pow2, rest;
    __device__ __forceinline__ explicit RowScale(float s) {  // 2^-64 < s <= 2^63
        const uint32_t top = __builtin_bit_cast(uint32_t, s) & 0x7F800000u;
        pow2 = __builtin_bit_cast(float, top - (2u << 23));
        rest = s * __builtin_bit_cast(float, (256u << 23) - top);
    }
};

// y / scale of a group without y's roundings. With t = y / rest, the product of r,
// a power of two and w, s cancels out and the quotient is 448 t / max |t|.
// Products of bf16 are exact in t, their quotients are often halfway between two
// e4m3 values (one in 10,000), and such a tie has to come out exactly to go to the
// even one: the factor is kept in two terms, off by less than 2^-44 beside the one
// rounding. (From the rounded y either side of a tie came out: 1,818 of 25 million
// values of 196,608 x 128 bf16.) 448 / max |t| is a normal number in groups above
// the smallest scale, t being at most a quarter of fp32's range where y is in it.
struct E4m3Group {
    float scale, high, low, rest;
    __device__ __forceinline__ E4m3Group(float most, float s_rest) : rest(s_rest) {
        scale = e4m3_scale(most * rest);
        const float r = __builtin_amdgcn_rcpf(most);
        high = 448.f * r;
        low = fmaf(-most, high, 448.f) * r;
        if (!(scale > kScaleFloor)) {  // the smallest scale: y over it
            high = rest * (1.f / kScaleFloor);
            low = 0.f;
        }
    }
    __device__ __forceinline__ void quotients(float (&t)[8]) const {
        if (scale < __builtin_inff()) {
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = fmaf(t[e], high, t[e] * low);
        } else {  // 0, and NaN of an infinite y
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = t[e] * rest * 0.f;
        }
    }
};

struct SumOp {
    static __device__ __forceinline__ float row16(float x) { return row16_sum(x); }
    static __device__ __forceinline__ float two(float a, float b) { return a + b; }
};
struct MaxOp {
    static __device__ __forceinline__ float row16(float x) { return row16_max(x); }
    static __device__ __forceinline__ float two(float a, float b) { return fmaxf(a, b); }
};

// Reduction over the threads that share a row: 16 lanes, a wave, or the
// workgroup (TPR 0; `red` holds one value per wave and is free for the next
// reduction only after another barrier).
template <int TPR, typename Op> __device__ __forceinline__ float row_reduce(float x, float *red) {
    x = Op::row16(x);
    if constexpr (TPR != 16) {
        x = Op::two(x, __shfl_xor(x, 16));
        x = Op::two(x, __shfl_xor(x, 32));
    }
    if constexpr (TPR == 0) {
        const int waves = blockDim.x >> 6;
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
        __syncthreads();
        x = red[0];
        for (int w = 1; w < waves; ++w) x = Op::two(x, red[w]);
    }
    return x;
}

// 8 elements at p: one or two 16-byte accesses, or element by element where only
// `left` of them are the row's. ONCE: non-temporal, for
// rows that are touched once. Wide rows gain from it (16,384 x 5,120: 112
// against 118 us), narrow ones lose (196,608 x 128: 15.9 against 14.7 us).
// Rows that do not start on 16 bytes (VEC false) are read and written by the
// same accesses without that alignment and hint.
typedef __bf16 bf16x8_any __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

template <bool ONCE, typename V> __device__ __forceinline__ V take(const V *p) {
    if constexpr (ONCE) return __builtin_nontemporal_load(p);
    return *p;
}
template <bool ONCE, typename V> __device__ __forceinline__ void give(V v, V *p) {
    if constexpr (ONCE)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}
template <bool ONCE, typename V8>
__device__ __forceinline__ void load_wide(const __bf16 *p, float (&x)[8]) {
    const V8 v = take<ONCE>(reinterpret_cast<const V8 *>(p));
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)v[e];
}
template <bool ONCE, typename V4>
__device__ __forceinline__ void load_wide(const float *p, float (&x)[8]) {
    const V4 a = take<ONCE>(reinterpret_cast<const V4 *>(p));
    const V4 b = take<ONCE>(reinterpret_cast<const V4 *>(p) + 1);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[e] = a[e];
        x[e + 4] = b[e];
    }
}
template <bool ONCE, typename V8>
__device__ __forceinline__ void store_wide(__bf16 *p, const float (&x)[8]) {
    V8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (__bf16)x[e];
    give<ONCE>(v, reinterpret_cast<V8 *>(p));
}
template <bool ONCE, typename V4>
__device__ __forceinline__ void store_wide(float *p, const float (&x)[8]) {
    give<ONCE>(V4{x[0], x[1], x[2], x[3]}, reinterpret_cast<V4 *>(p));
    give<ONCE>(V4{x[4], x[5], x[6], x[7]}, reinterpret_cast<V4 *>(p) + 1);
}
template <typename DT> struct Wide;
template <> struct Wide<__bf16> { using on16 = bf16x8; using any = bf16x8_any; };
template <> struct Wide<float> { using on16 = f32x4; using any = f32x4_any; };

template <typename DT, bool VEC, bool ONCE>
__device__ __forceinline__ void load8(const DT *p, int left, float (&x)[8]) {
    if constexpr (VEC) {
        load_wide<ONCE, typename Wide<DT>::on16>(p, x);
    } else if (left >= 8) {
        load_wide<false, typename Wide<DT>::any>(p, x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = e < left ? to_f32(p[e]) : 0.f;
    }
}
template <typename DT, bool VEC, bool ONCE>
__device__ __forceinline__ void store8(DT *p, int left, const float (&x)[8]) {
    if constexpr (VEC) {
        store_wide<ONCE, typename Wide<DT>::on16>(p, x);
    } else if (left >= 8) {
        store_wide<false, typename Wide<DT>::any>(p, x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) p[e] = from_f32<DT>(x[e]);
    }
}

// 8 values in OCP e4m3, rounded to nearest even.
template <bool VEC, bool ONCE>
__device__ __forceinline__ void store8_e4m3(uint8_t *p, int left, const float (&x)[8]) {
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
    if constexpr (VEC) {
        give<ONCE>(u32x2{(uint32_t)lo, (uint32_t)hi}, reinterpret_cast<u32x2 *>(p));
    } else if (left >= 8) {
        *reinterpret_cast<u32x2_any *>(p) = u32x2_any{(uint32_t)lo, (uint32_t)hi};
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) p[e] = (uint8_t)((uint32_t)(e < 4 ? lo : hi) >> (8 * (e & 3)));
    }
}

// Threads that share a row and the row of this thread.
template <int TPR> __device__ __forceinline__ int row_threads() {
    return TPR == 0 ? (int)blockDim.x : TPR;
}

// One row of a thread: x and the residual as fp32, from memory.
template <typename DT, bool VEC, int TPR, int CH> struct NormRow {
    float r[CH][8];

    __device__ __forceinline__ void load(const NormParams &p, int64_t row, bool live, int tpr,
                                         int j) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int c = (k * tpr + j) * 8, left = live ? p.D - c : 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) r[k][e] = 0.f;
            if (left <= 0) continue;
            load8<DT, VEC, TPR == 0>(reinterpret_cast<const DT *>(p.x) + row * p.D + c, left, r[k]);
            if (p.res) {
                float q[8];
                load8<DT, VEC, TPR == 0>(reinterpret_cast<const DT *>(p.res) + row * p.D + c, left, q);
#pragma unroll
                for (int e = 0; e < 8; ++e) r[k][e] += q[e];
            }
        }
    }
};

// Everything behind a row's loads. A row past the last one takes part with
// zeros, for the lanes of a wave reduce together.
// The weights of a thread's columns: `held` where it has them for several rows.
template <typename DT, bool VEC, int TPR, int CH, bool HELD>
__device__ __forceinline__ void norm_row(const NormParams &p, int64_t row, int tpr, int j,
                                         float (&r)[CH][8], const float (&held)[HELD ? CH : 1][8],
                                         float (*s_red)[16]) {
    const int D = p.D;
    const bool live = row < p.rows;
    const int64_t at = row * D;
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        const int c = (k * tpr + j) * 8, left = live ? D - c : 0;
        if (left > 0 && p.res_out)
            store8<DT, VEC, TPR == 0>(reinterpret_cast<DT *>(p.res_out) + at + c, left, r[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(r[k][e], r[k][e], ss);
    }
    ss = row_reduce<TPR, SumOp>(ss, s_red[0]);
    const float s = inv_sqrt(fmaf(ss, p.inv_d, p.eps));
    const RowScale rs(s);
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        const int c = (k * tpr + j) * 8, left = live ? D - c : 0;
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 0.f;
        if (left > 0) {
            if constexpr (HELD) {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = held[k][e];
            } else {
                load8<DT, VEC, false>(reinterpret_cast<const DT *>(p.w) + c, left, w);
            }
            if (p.out) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = r[k][e] * s * w[e];
                store8<DT, VEC, TPR == 0>(reinterpret_cast<DT *>(p.out) + at + c, left, y);
            }
        }
        if (!p.out8) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) r[k][e] = r[k][e] * rs.pow2 * w[e];
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(r[k][e]));
        if (p.group == 0) {
            most = fmaxf(most, m);
        } else {  // 128 columns: the 16 lanes of a DPP row
            const E4m3Group g(row16_max(m), rs.rest);
            g.quotients(r[k]);
            if (left > 0) {
                store8_e4m3<VEC, TPR == 0>(p.out8 + at + c, left, r[k]);
                if ((j & 15) == 0) p.scales[row * ((D + 127) / 128) + c / 128] = g.scale;
            }
        }
    }
    if (p.out8 && p.group == 0) {
        const E4m3Group g(row_reduce<TPR, MaxOp>(most, s_red[1]), rs.rest);
        if (live && j == 0) p.scales[row] = g.scale;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int c = (k * tpr + j) * 8, left = live ? D - c : 0;
            g.quotients(r[k]);
            if (left > 0) store8_e4m3<VEC, TPR == 0>(p.out8 + at + c, left, r[k]);
        }
    }
}

// NROWS rows per thread, their loads issued together. Bound by HBM for wide rows:
// 16,384 x 5,120 bf16 with residual, to e4m3 and the new residual, 115 us (5.1
// TB/s, a copy's rate); by vector instructions for rows of 128: 196,608 rows 15
// us, of which the 327 instructions of each of 24,576 waves fill 13 (4 rows per
// thread took 20 us where 2 took 14 and 1 17); 8 rows of 5,120 3.4 us.
template <typename DT, bool VEC, int TPR, int CH, int NROWS>
__global__ __launch_bounds__(1024) void norm_kernel(NormParams p) {
    __shared__ float s_red[2][16];
    const int tpr = row_threads<TPR>();
    const int j = TPR == 0 ? threadIdx.x : threadIdx.x % tpr;
    const int per = TPR == 0 ? 1 : blockDim.x / tpr;
    const int64_t row0 = (int64_t)workgroup() * per * NROWS + (TPR == 0 ? 0 : threadIdx.x / tpr);
    NormRow<DT, VEC, TPR, CH> rows[NROWS];
#pragma unroll
    for (int i = 0; i < NROWS; ++i)
        rows[i].load(p, row0 + i * per, row0 + i * per < p.rows, tpr, j);
    constexpr bool HELD = NROWS > 1;
    float w[HELD ? CH : 1][8];
    if constexpr (HELD)
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int c = (k * tpr + j) * 8;
            if (c < p.D) load8<DT, VEC, false>(reinterpret_cast<const DT *>(p.w) + c, p.D - c, w[k]);
        }
#pragma unroll
    for (int i = 0; i < NROWS; ++i)
        norm_row<DT, VEC, TPR, CH, HELD>(p, row0 + i * per, tpr, j, rows[i].r, w, s_red);
}

// dx per row, and each workgroup's share of dw: a thread keeps the sums of its
// columns over the workgroup's rows, the workgroup joins the threads that hold
// the same columns, and norm_dweight_kernel joins the workgroups in order. As
// many workgroups as give every CU 1,024 threads, but not under 512 unless the
// rows are fewer, and 4 turns for each above that (16,384 x 2,048 bf16, both
// directions, 98 us, 112 with 512, 103 with 2,048 threads). 8,191 x 4,096 bf16
// 47 us (5.7 TB/s).
template <typename DT, bool VEC, int TPR, int CH>
__global__ __launch_bounds__(1024) void norm_backward_kernel(NormBackwardParams p) {
    __shared__ float s_red[2][16];
    __shared__ float s_dw[TPR == 0 ? 1 : 256 * 8 * CH];
    const int tpr = row_threads<TPR>();
    const int j = TPR == 0 ? threadIdx.x : threadIdx.x % tpr;
    const int per = TPR == 0 ? 1 : blockDim.x / tpr;  // rows side by side
    const int D = p.D;
    float w[CH][8], dw[CH][8];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        const int c = (k * tpr + j) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[k][e] = 0.f;
            dw[k][e] = 0.f;
        }
        if (c < D) load8<DT, VEC, false>(reinterpret_cast<const DT *>(p.w) + c, D - c, w[k]);
    }
    int turn = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * per; row0 < p.rows;
         row0 += (int64_t)gridDim.x * per, turn ^= 1) {
        const int64_t row = row0 + (TPR == 0 ? 0 : threadIdx.x / tpr);
        const bool live = row < p.rows;
        const int64_t at = row * D;
        float r[CH][8], dy[CH][8];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int c = (k * tpr + j) * 8, left = live ? D - c : 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                r[k][e] = 0.f;
                dy[k][e] = 0.f;
            }
            if (left > 0) {
                load8<DT, VEC, TPR == 0>(reinterpret_cast<const DT *>(p.r) + at + c, left, r[k]);
                load8<DT, VEC, TPR == 0>(reinterpret_cast<const DT *>(p.dout) + at + c, left, dy[k]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(r[k][e], r[k][e], ss);
                dot = fmaf(w[k][e] * dy[k][e], r[k][e], dot);
            }
        }
        if constexpr (TPR == 0) {  // both sums in one exchange
            __shared__ float s_two[2][2][16];
            const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
            ss = row_reduce<64, SumOp>(ss, nullptr);
            dot = row_reduce<64, SumOp>(dot, nullptr);
            if ((threadIdx.x & 63) == 0) {
                s_two[turn][0][wave] = ss;
                s_two[turn][1][wave] = dot;
            }
            __syncthreads();  // the other turn's values were read before this barrier
            ss = s_two[turn][0][0];
            dot = s_two[turn][1][0];
            for (int i = 1; i < waves; ++i) {
                ss += s_two[turn][0][i];
                dot += s_two[turn][1][i];
            }
        } else {
            ss = row_reduce<TPR, SumOp>(ss, s_red[0]);
            dot = row_reduce<TPR, SumOp>(dot, s_red[1]);
        }
        const float s = inv_sqrt(fmaf(ss, p.inv_d, p.eps));
        // mean(w dy u): no power of s by itself, which would leave fp32's range for
        // rows near 0 under a small eps, or vanish for large ones
        const float m = dot * p.inv_d * s;
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int c = (k * tpr + j) * 8, left = live ? D - c : 0;
            if (left <= 0) continue;
            float dx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) dx[e] = 0.f;
            if (p.dres) load8<DT, VEC, TPR == 0>(reinterpret_cast<const DT *>(p.dres) + at + c, left, dx);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float u = r[k][e] * s;
                dx[e] = fmaf(s, fmaf(-u, m, w[k][e] * dy[k][e]), dx[e]);
                dw[k][e] = fmaf(dy[k][e], u, dw[k][e]);
            }
            store8<DT, VEC, TPR == 0>(reinterpret_cast<DT *>(p.dx) + at + c, left, dx);
        }
    }
    if (!p.dw) return;
    float *part = p.partial + (int64_t)blockIdx.x * norm_partial_width(D);
    if constexpr (TPR == 0) {
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const int c = (k * tpr + j) * 8;
            if (c < D) store8<float, true, false>(part + c, 8, dw[k]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) s_dw[(threadIdx.x * CH + k) * 8 + e] = dw[k][e];
        __syncthreads();
        if ((int)threadIdx.x < tpr) {
            for (int i = 1; i < per; ++i)
#pragma unroll
                for (int k = 0; k < CH; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dw[k][e] += s_dw[((threadIdx.x + i * tpr) * CH + k) * 8 + e];
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                const int c = (k * tpr + j) * 8;
                if (c < D) store8<float, true, false>(part + c, 8, dw[k]);
            }
        }
    }
}

// dw[c] = sum over the partials in a fixed order: 32 columns per workgroup, 4
// per lane (partial rows are padded to 8 columns), 128 threads beside each other
// down the partials. 512 x 4,096 in 4.0 us (one lane per column and 16
// threads down took 9.5: too few loads at once).
__global__ __launch_bounds__(1024) void norm_dweight_kernel(const float *partial, int count,
                                                            float *dw, int D) {
    constexpr int VEC = 4, kLanes = 32 / VEC, kParts = 1024 / kLanes;
    const int width = norm_partial_width(D);
    __shared__ float s_sum[16][32];
    const int l = threadIdx.x % kLanes, part = threadIdx.x / kLanes;
    const int c = blockIdx.x * 32 + l * VEC;
    float sum[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum[e] = 0.f;
    if (c < D)
#pragma unroll 4
        for (int i = part; i < count; i += kParts) {
            const f32x4 x = *reinterpret_cast<const f32x4 *>(partial + (int64_t)i * width + c);
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum[e] += x[e];
        }
    // the parts of a wave, then the 16 waves
#pragma unroll
    for (int e = 0; e < VEC; ++e)
#pragma unroll
        for (int o = kLanes; o < 64; o <<= 1) sum[e] += __shfl_xor(sum[e], o);
    if ((threadIdx.x & 63) < kLanes)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s_sum[threadIdx.x >> 6][l * VEC + e] = sum[e];
    __syncthreads();
    const int o = blockIdx.x * 32 + threadIdx.x;
    if (threadIdx.x < 32 && o < D) {
        float all = s_sum[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < 16; ++i) all += s_sum[i][threadIdx.x];
        dw[o] = all;
    }
}

// How a row is shared out: threads per row (16, 64 or a workgroup), chunks of
// 8 columns per thread, threads per workgroup and rows per workgroup.
struct NormPlan {
    int tpr, ch, threads, per;
};

// The backward pass stays with one wave up to 1,024 columns, without a barrier
// (16,384 x 1,024 bf16, both directions, 52 against 59 us); the forward one does
// not, whose workgroups read rows once past the caches (32,768 x 1,024 41
// against 44 us).
NormPlan plan_norm(int32_t D, bool back) {
    const int chunks = (D + 7) / 8;
    if (chunks <= 16) return {16, 1, 256, 16};
    if (chunks <= 64) return {64, 1, 256, 4};
    if (back && chunks <= 128) return {64, 2, 256, 4};
    const int ch = chunks > 1024 ? 2 : 1;
    const int threads = ((chunks + ch - 1) / ch + 63) / 64 * 64;
    return {0, ch, threads, 1};
}

template <typename F> hipError_t with_norm_types(int dtype, int32_t D, const NormPlan &n, const F &f) {
    const bool vec = D % 8 == 0;
#define GDN_NORM_CASE(DT, VEC)                                                   \
    do {                                                                         \
        if (n.tpr == 16) return f.template run<DT, VEC, 16, 1>(n);               \
        if (n.tpr == 64 && n.ch == 1) return f.template run<DT, VEC, 64, 1>(n);  \
        if constexpr (F::kBack)                                                  \
            if (n.tpr == 64) return f.template run<DT, VEC, 64, 2>(n);           \
        if (n.ch == 1) return f.template run<DT, VEC, 0, 1>(n);                  \
        return f.template run<DT, VEC, 0, 2>(n);                                 \
    } while (0)
    if (dtype == 1) {
        if (vec) GDN_NORM_CASE(__bf16, true);
        GDN_NORM_CASE(__bf16, false);
    }
    if (vec) GDN_NORM_CASE(float, true);
    GDN_NORM_CASE(float, false);
#undef GDN_NORM_CASE
}

struct RunNorm {
    static constexpr bool kBack = false;
    const NormParams &p;
    hipStream_t stream;
    template <typename DT, bool VEC, int TPR, int CH> hipError_t run(const NormPlan &n) const {
        if constexpr (TPR != 0) {
            if (p.rows >= (int64_t)n.per * 2 * 4096) {
                hipLaunchKernelGGL((norm_kernel<DT, VEC, TPR, CH, 2>),
                                   grid_of((p.rows + 2 * n.per - 1) / (2 * n.per), n.threads),
                                   dim3(n.threads), 0, stream, p);
                return hipGetLastError();
            }
        }
        hipLaunchKernelGGL((norm_kernel<DT, VEC, TPR, CH, 1>),
                           grid_of((p.rows + n.per - 1) / n.per, n.threads), dim3(n.threads),
                           0, stream, p);
        return hipGetLastError();
    }
};

struct RunNormBackward {
    static constexpr bool kBack = true;
    const NormBackwardParams &p;
    hipStream_t stream;
    template <typename DT, bool VEC, int TPR, int CH> hipError_t run(const NormPlan &n) const {
        hipLaunchKernelGGL((norm_backward_kernel<DT, VEC, TPR, CH>),
                           dim3((unsigned)norm_partials(p.rows, p.D)), dim3(n.threads), 0,
                           stream, p);
        return hipGetLastError();
    }
};

}  // namespace

hipError_t launch_norm(const NormParams &p, int dtype, hipStream_t stream) {
    return with_norm_types(dtype, p.D, plan_norm(p.D, false), RunNorm{p, stream});
}

// Workgroups of the backward pass (see its kernel), each with a row of partial sums.
int norm_partials(int64_t rows, int32_t D) {
    const NormPlan n = plan_norm(D, true);
    const int64_t wgs = (rows + n.per - 1) / n.per, fill = (1 << 18) / n.threads;
    const int64_t most = std::max<int64_t>(512, std::min(fill, wgs / 4));
    return (int)std::min(wgs, most);
}

hipError_t launch_norm_backward(const NormBackwardParams &p, int dtype, hipStream_t stream) {
    const int count = norm_partials(p.rows, p.D);
    if (count > 0) {
        const hipError_t e =
            with_norm_types(dtype, p.D, plan_norm(p.D, true), RunNormBackward{p, stream});
        if (e != hipSuccess) return e;
    }
    if (p.dw) {
        const dim3 grid((unsigned)((p.D + 31) / 32)), block(1024);
        hipLaunchKernelGGL(norm_dweight_kernel, grid, block, 0, stream, p.partial, count, p.dw,
                           p.D);
    }
    return hipGetLastError();
}

}  // namespace gdn
