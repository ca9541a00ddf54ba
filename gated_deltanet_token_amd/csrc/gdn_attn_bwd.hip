// gdn_attn_bwd.hip -- gradients of causal softmax attention with grouped heads
// (gfx950), dense and packed.
//
// With p_tj = exp(scale q_t . k_j - lse_t), formed again from the stored lse:
//   delta_t = dout_t . out_t,   ds_tj = p_tj (dout_t . v_j - delta_t)
//   dq_t = scale sum_j ds_tj k_j
//   dv_j = sum_t p_tj dout_t,   dk_j = scale sum_t ds_tj q_t
// dk and dv sum over the query heads of the key head as well.
//
// lse is held in fp32, so a weight formed from it is off by up to 3 2^-24 |lse| (seen: 9 % at
// scores of 2^20, whose differences fp32 still holds, and a factor of 2 at 2^23). A row's weights
// share that factor. The dq kernel, which forms all of a row's weights, sums them, divides
// its row by the sum and leaves 1 / sum for the weights in dk and dv (4 x 2,048 tokens of 16/4
// heads of 64, forward and backward: 261 us, 258 without; 128 and 256 wide as fast). A sum further
// from 1 than the rounding of lse explains is that of a row whose lse and out are over more keys
// than these (a prefix in front, say): its weights stay as lse makes them.
//
// Three kernels: the rows' statistics; dq by query tiles (three products per pair
// of tiles); dk and dv by key tiles (four). Scores and dout . v are formed in both:
// 7 products where 5 would do, but every sum has one owner, so that no atomics and
// no order of workgroups enter the results. p and ds are rounded to the tensors'
// type as operands of the products (bf16: off by 2^-9 to 2^-8 relative, like
// the stored inputs), sums are fp32.
//
// Bound by the matrix instructions, busy 39 to 49 % of the time. 2 x 4,097 tokens of
// 16/4 heads of 128: dq 212 us, dk and dv 337, statistics 14, join 22; with the
// forward pass 719 to 728 us, 661 to 670 TFLOP/s counting 7 products in all.
#include <type_traits>

#include "gdn_attn.hpp"

namespace gdn {

namespace {

// log2-scaled lse and delta of every (head, token), the first two of p.stats. 16 lanes per row
// of D.
template <typename DT, int D>
__global__ __launch_bounds__(256) void attn_stats_kernel(AttnBackwardParams p) {
    const int64_t rows = p.total * p.Hq;
    const int64_t row = (int64_t)workgroup() * 16 + (threadIdx.x >> 4);
    if (row >= rows) return;
    const int c = threadIdx.x & 15;
    const DT *a = static_cast<const DT *>(p.dout) + row * D, *b =
        static_cast<const DT *>(p.out) + row * D;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = 64 * i + 4 * c + e;
            sum = fmaf(to_f32(a[d]), to_f32(b[d]), sum);
        }
    sum = row16_sum(sum);
    if (c == 0) {
        const int64_t tok = row / p.Hq, at = (row - tok * p.Hq) * p.total + tok;
        const float lse = p.lse[row];
        // a row of -inf scores has no weights
        p.stats[at] = lse == -__builtin_inff() ? __builtin_inff() : lse * kLog2e;
        p.stats[rows + at] = sum;
    }
}

// Where a mask cuts a tile: whether any of its rows holds an infinity or NaN.
template <typename DT> __device__ __forceinline__ bool odd_part(const unsigned char *t, int bytes) {
    bool odd = false;
    for (int i = threadIdx.x; i < bytes / 16; i += blockDim.x)
        odd |= not_finite(reinterpret_cast<const u32x4 *>(t)[i], DT{});
    return odd;
}
// Then: flags[r] says so of row r, for `tiles` tiles of `rows` rows, one after the other.
template <typename DT, int D>
__device__ __forceinline__ void odd_rows(const unsigned char *t, int rows, int tiles, int *flags) {
    if (threadIdx.x < rows) flags[threadIdx.x] = 0;
    __syncthreads();
    constexpr int kChunks = Rows<DT, D>::kChunks;
    for (int i = threadIdx.x; i < rows * tiles * kChunks; i += blockDim.x)
        if (not_finite(reinterpret_cast<const u32x4 *>(t)[i], DT{})) flags[i / kChunks % rows] = 1;
    __syncthreads();
}
// And the tile with zeros in their place: a weight of 0 times such a value would be NaN.
template <typename DT> __device__ __forceinline__ void clear_odd(unsigned char *t, int bytes) {
    for (int i = threadIdx.x; i < bytes / 16; i += blockDim.x) {
        u32x4 &w = reinterpret_cast<u32x4 *>(t)[i];
        w = only_finite(w, DT{});
    }
}

// Whether a row's weights sum up to 1 but for the rounding of its lse (log2-scaled; three roundings
// of 2^-24 each, and a fourth to spare) and of the sum.
__device__ __forceinline__ bool whole_row(float all, float lse2) {
    return all > 0.f && fabsf(log2f(all)) <= fmaf(fabsf(lse2), 0x1p-22f, 0x1p-16f);
}

template <typename DT, int D, int CT, int NW, int BK, int PER_SIMD>
__global__ __launch_bounds__(64 * NW, PER_SIMD) void attn_dq_kernel(AttnBackwardParams p,
                                                                    HeadOrder order) {
    using Tiles = KeyTiles<DT, D, CT, NW, BK>;
    using A = Attend<DT, D, CT>;
    using R = Rows<DT, D>;
    constexpr int BM = NW * CT * 16, kTile = Tiles::kTile;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    __shared__ int odd[BK];
    const int lane = threadIdx.x & 63, c = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int unit, slot;
    if (!order.pick(workgroup(), unit, slot)) return;
    const SeqTile s = seq_tile<BM>(p.cu, p.N, p.T, p.total, unit, slot, order.tiles, p.Hq, lane);
    const int tile = s.tiles - 1 - s.tile, len = s.len, head = s.head;
    const int64_t tok0 = s.tok0;
    if (s.tile >= s.tiles) return;
    const int q0 = tile * BM, w0 = q0 + wave * CT * 16, kh = head / (p.Hq / p.Hk);

    Frag<DT> qf[D / 32][CT], df[D / 32][CT];
    float lse[CT], delta[CT], sum[CT];  // sum: of the weights, the lane's own part of them
    // keys that the lane's query sees
    auto sees = [&](int ct) { return min(w0 + 16 * ct + (fresh(lane) & 15), len - 1) + 1; };
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int row = min(w0 + 16 * ct + c, len - 1);
        const int64_t at = ((tok0 + row) * p.Hq + head) * D;
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
            qf[kk][ct] = R::load(static_cast<const DT *>(p.q) + at, kk, g4);
            df[kk][ct] = R::load(static_cast<const DT *>(p.dout) + at, kk, g4);
        }
        sum[ct] = 0.f;
        lse[ct] = p.stats[(int64_t)head * p.total + tok0 + row];
        delta[ct] = p.stats[((int64_t)p.Hq + head) * p.total + tok0 + row];
    }
    const int64_t stride = (int64_t)p.Hk * D * sizeof(DT);
    DenseKeys src{static_cast<const unsigned char *>(p.k) + tok0 * stride + kh * R::kPitch,
                        static_cast<const unsigned char *>(p.v) + tok0 * stride + kh * R::kPitch,
                        stride, len};
    f32x4 acc[D / 16][CT];
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) acc[dt][ct] = zero4();
    const int end = min(q0 + BM, len), hi = w0 < len ? min(w0 + CT * 16, len) : 0;
    const float scale2 = p.scale * kLog2e;

    Tiles::issue(src, 0, (uint32_t)stride, lds, wave, lane);
    int parity = 0;
    for (int key = 0; key < end; key += BK, parity ^= 1) {
        wait_copies<0>();
        __syncthreads();
        unsigned char *kt = lds + parity * 2 * kTile, *vt = kt + kTile;
        if (key + BK < end)
            Tiles::issue(src, key + BK, (uint32_t)stride, lds + (parity ^ 1) * 2 * kTile, wave,
                         lane);
        if (key + BK > q0 + 1 && __syncthreads_or(odd_part<DT>(kt, kTile))) {
            // keys that are not finite make NaN of the queries that see them and are taken out
            // of the product with ds
            odd_rows<DT, D>(kt, BK, 1, odd);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                bool nan = false;
                for (int row = 0; row < BK; ++row) nan |= odd[row] && key + row < sees(ct);
                if (nan) lse[ct] = __builtin_nanf("");
            }
            __syncthreads();
            clear_odd<DT>(kt, kTile);
            __syncthreads();
        }
        if (sizeof(DT) == 2 && key == 0 && w0 < 32) {
            // The first 32 queries see few keys, and dout . v_j - delta is a small difference
            // of large terms where one key has most of the weight: from out as stored (off by
            // up to 2^-8) the gradients of two-token sequences came out up to 2e-2 off, relative
            // to their norm. delta is also sum_j p_tj (dout_t . v_j), here over one tile.
            f32x4 sc[2][CT], dp[2][CT];
            A::scores(kt, 0, qf, sc, lane);
            A::scores(vt, 0, df, dp, lane);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int lim = sees(ct);
                float all = 0.f, of = 0.f;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float w = exp2_fast(fmaf(sc[t][ct][r], scale2, -lse[ct]));
                        if (16 * t + 4 * g4 + r < lim) {
                            all += w;
                            of = fmaf(w, dp[t][ct][r], of);
                        }
                    }
                all = across_sum(all);
                of = across_sum(of);
                if (!whole_row(all, lse[ct])) continue;
                delta[ct] = of / all;
                const int row = w0 + 16 * ct + c;
                if (g4 == 0 && row < len)  // for dk and dv
                    p.stats[((int64_t)p.Hq + head) * p.total + tok0 + row] = delta[ct];
            }
        }
#pragma unroll 1
        for (int sub = 0; sub < BK; sub += 32) {
            const int k = key + sub;
            if (k >= hi) break;
            f32x4 sc[2][CT], dp[2][CT];
            A::scores(kt, sub, qf, sc, lane);
            A::scores(vt, sub, df, dp, lane);
            Frag<DT> f[CT];
            const bool cut = k + 32 > w0 + 1;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                if (cut) {
                    const int lim = sees(ct);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (k + 16 * (i >> 2) + 4 * g4 + (i & 3) >= lim) {
                            sc[i >> 2][ct][i & 3] = -__builtin_inff();
                            dp[i >> 2][ct][i & 3] = 0.f;
                        }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float w = exp2_fast(fmaf(sc[t][ct][r], scale2, -lse[ct]));
                        sum[ct] += w;
                        dp[t][ct][r] = w * (dp[t][ct][r] - delta[ct]);
                    }
                c_to_frag(dp[0][ct], dp[1][ct], f[ct]);
            }
            A::add_to(acc, kt, sub, f, lane);
        }
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int row = w0 + 16 * ct + c;
        const float all = across_sum(sum[ct]);
        if (row >= len) continue;
        const float f = whole_row(all, lse[ct]) ? 1.f / all : 1.f;
        DT *o = static_cast<DT *>(p.dq) + ((tok0 + row) * p.Hq + head) * D + 4 * g4;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) store4(o + 16 * dt, acc[dt][ct] * (p.scale * f));
        if (g4 == 0) p.stats[((int64_t)2 * p.Hq + head) * p.total + tok0 + row] = f;
    }
}

// Copies 64 words (4 bytes per lane) into LDS; as dma16_async.
__device__ __forceinline__ void dma4_async(const unsigned char *base, uint32_t off,
                                           unsigned char *lds) {
    const uint32_t m0 = (uint32_t)(uintptr_t)(lds_u8 *)lds;
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
                 :
                 : "v"(off), "s"(base), "s"(m0)
                 : "memory", "m0");
}

template <typename DT, int D, int CT, int NW, int BQ, int PER_SIMD>
__global__ __launch_bounds__(64 * NW, PER_SIMD) void attn_dkv_kernel(AttnBackwardParams p,
                                                                     HeadOrder order) {
    using Tiles = KeyTiles<DT, D, CT, NW, BQ>;
    using A = Attend<DT, D, CT>;
    using R = Rows<DT, D>;
    constexpr int BN = NW * CT * 16, kTile = Tiles::kTile;
    constexpr int kBuf = 2 * kTile + 768;  // queries, dout, 64 lse, 64 delta, 64 factors
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    __shared__ int odd[BQ];
    const int lane = threadIdx.x & 63, c = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int unit, slot;
    if (!order.pick(workgroup(), unit, slot)) return;
    const SeqTile s =
        seq_tile<BN>(p.cu, p.N, p.T, p.total, unit, slot, order.tiles, p.Hk * p.split, lane);
    if (s.tile >= s.tiles) return;
    const int len = s.len, kh = s.head / p.split, part = s.head % p.split;
    const int64_t tok0 = s.tok0;
    const int g = p.Hq / p.Hk;
    const int j0 = kh * g + part * g / p.split, j1 = kh * g + (part + 1) * g / p.split;
    const int k0 = s.tile * BN, w0 = k0 + wave * CT * 16;

    Frag<DT> kf[D / 32][CT], vf[D / 32][CT];
    int own[CT];      // first query that sees the lane's key
    bool lost[CT]{};  // NaN
    const int64_t kvstride = (int64_t)p.Hk * D;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int row = w0 + 16 * ct + c;
        own[ct] = row < len ? row : 0x7FFFFFFF;
        const int64_t at = (tok0 + min(row, len - 1)) * kvstride + kh * D;
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
            kf[kk][ct] = R::load(static_cast<const DT *>(p.k) + at, kk, g4);
            vf[kk][ct] = R::load(static_cast<const DT *>(p.v) + at, kk, g4);
        }
    }
    f32x4 dk[D / 16][CT], dv[D / 16][CT];
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) dk[dt][ct] = dv[dt][ct] = zero4();
    const int64_t stride = (int64_t)p.Hq * D * sizeof(DT);
    const float scale2 = p.scale * kLog2e;
    const int first = k0 / BQ * BQ;  // the first query tile that sees any of these keys

    auto issue = [&](int j, int q, unsigned char *buf) {
        DenseKeys src{
            static_cast<const unsigned char *>(p.q) + tok0 * stride + j * R::kPitch,
            static_cast<const unsigned char *>(p.dout) + tok0 * stride + j * R::kPitch, stride,
            len};
        Tiles::issue(src, q, (uint32_t)stride, buf, wave, lane);
        if (wave < 3) {
            const float *st = p.stats + ((int64_t)wave * p.Hq + j) * p.total + tok0 + q;
            dma4_async(uniform(reinterpret_cast<const unsigned char *>(st)),
                       (uint32_t)min(lane, len - 1 - q) * 4, buf + 2 * kTile + wave * 256);
        }
    };
    issue(j0, first, lds);
    int parity = 0;
    for (int j = j0; j < j1; ++j) {
        for (int q = first; q < len; q += BQ, parity ^= 1) {
            wait_copies<0>();
            __syncthreads();
            unsigned char *buf = lds + parity * kBuf, *qt = buf, *dt_ = buf + kTile;
            const float *lse = reinterpret_cast<const float *>(buf + 2 * kTile);
            const float *delta = lse + 64, *factor = lse + 128;
            const bool wrap = q + BQ >= len;
            if (!wrap || j + 1 < j1)
                issue(wrap ? j + 1 : j, wrap ? first : q + BQ, lds + (parity ^ 1) * kBuf);
            const bool cut_wg = q < k0 + BN || q + BQ > len;
            if (cut_wg && __syncthreads_or(odd_part<DT>(buf, 2 * kTile))) {
                // queries and gradients that are not finite make NaN of the keys that they
                // reach and are taken out of the products
                odd_rows<DT, D>(buf, BQ, 2, odd);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    bool nan = false;
                    for (int row = 0; row < BQ; ++row)
                        nan |= odd[row] && q + row >= own[ct] && q + row < len;
                    lost[ct] |= nan;
                }
                __syncthreads();
                clear_odd<DT>(buf, 2 * kTile);
                __syncthreads();
            }
#pragma unroll 1
            for (int sub = 0; sub < BQ; sub += 32) {
                const int qs = q + sub;
                if (qs >= len) break;
                if (qs + 31 < w0 || w0 >= len) continue;  // before all of the wave's keys
                f32x4 sc[2][CT], dp[2][CT];
                A::scores(qt, sub, kf, sc, lane);
                const bool cut = qs < w0 + CT * 16 || qs + 32 > len;
                Frag<DT> f[CT];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const f32x4 ls = *reinterpret_cast<const f32x4 *>(lse + sub + 16 * t + 4 * g4);
                    const f32x4 fa =
                        *reinterpret_cast<const f32x4 *>(factor + sub + 16 * t + 4 * g4);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int row = qs + 16 * t + 4 * g4 + r;
                            float w = exp2_fast(fmaf(sc[t][ct][r], scale2, -ls[r])) * fa[r];
                            if (cut && (row < own[ct] || row >= len)) w = 0.f;
                            sc[t][ct][r] = w;
                        }
                }
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) c_to_frag(sc[0][ct], sc[1][ct], f[ct]);
                A::add_to(dv, dt_, sub, f, lane);
                __builtin_amdgcn_sched_barrier(0);  // one product's registers at a time
                A::scores(dt_, sub, vf, dp, lane);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const f32x4 de =
                        *reinterpret_cast<const f32x4 *>(delta + sub + 16 * t + 4 * g4);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int row = qs + 16 * t + 4 * g4 + r;
                            float w = sc[t][ct][r] * (dp[t][ct][r] - de[r]);
                            if (cut && (row < own[ct] || row >= len)) w = 0.f;
                            dp[t][ct][r] = w;
                        }
                }
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) c_to_frag(dp[0][ct], dp[1][ct], f[ct]);
                A::add_to(dk, qt, sub, f, lane);
            }
        }
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int row = w0 + 16 * ct + c;
        if (row >= len) continue;
        const int64_t at = (tok0 + row) * kvstride + kh * D + 4 * g4;
        const int64_t all = p.total * kvstride;
        const float nan = lost[ct] ? __builtin_nanf("") : 0.f;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
            dk[dt][ct] += nan;
            dv[dt][ct] += nan;
            if (p.split == 1) {
                store4(static_cast<DT *>(p.dk) + at + 16 * dt, dk[dt][ct] * p.scale);
                store4(static_cast<DT *>(p.dv) + at + 16 * dt, dv[dt][ct]);
            } else {
                float *o = p.parts + 2 * part * all + at + 16 * dt;
                store4(o, dk[dt][ct] * p.scale);
                store4(o + all, dv[dt][ct]);
            }
        }
    }
}

// The same for bf16, with wave pairs that own 16 CT keys: the first of a pair forms p of tile
// t (and dv), the second ds of tile t - 1 from the p that the first left in LDS (and dk).
// One wave holds one set of owned rows and one of sums instead of two, so that two waves fit
// a SIMD, one of each kind, whose exponentials and products overlap. Three tiles in LDS:
// t - 1, t and the one under way.
//
// p lies in LDS in 16 bits (LDS holds no more at D = 128): of the fp32 value, whose sign is 0 and
// whose highest exponent bit is 0 for anything below 2, the other 7 bits of the exponent and 9 of
// the mantissa. Half a step is 2^-10 of p at any size that fp32 holds (rounded to bf16 there, and
// once more as ds, dk came out 2.9e-3 off, relative to its norm, and not 2.4e-3; fp16 times 2^13
// was as good for p above 2^-27 but nothing below 2^-38: keys that all queries nearly ignore lost
// their dk; 2 x 4,097 tokens of 16/4 heads of 128, forward and backward: 728 us, so 720). p is at
// most 1, its row's sum being 1 at the most; should it not be, it counts as just below 2.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t code_of(float p) {  // in the upper half
    return (min(__builtin_bit_cast(uint32_t, p), 0x3FFFC000u) << 2) + 0x8000u;
}
__device__ __forceinline__ uint32_t code_pair(float p0, float p1) {
    return __builtin_amdgcn_perm(code_of(p1), code_of(p0), 0x07060302u);
}
template <int I> __device__ __forceinline__ float code_value(uint32_t w) {
    return __builtin_bit_cast(float, (uint32_t)__builtin_bit_cast(u16x2, w)[I] << 14);
}
template <typename DT, int D, int CT, int BQ> struct KeyPairs {
    using Tiles = KeyTiles<DT, D, CT, 8, BQ>;
    using A = Attend<DT, D, CT>;
    using R = Rows<DT, D>;
    static constexpr int kRows = 4 * CT * 16, kTile = Tiles::kTile;
    static constexpr int kBuf = 2 * kTile + 768;  // queries, dout, 64 lse, 64 delta, 64 factors
    static constexpr int kP = BQ / 32 * CT * 1024;  // p of a pair and tile
    static constexpr int kLds = 3 * kBuf + 8 * kP;

    // Both kinds of wave pass the same barriers. vote: two words, zero; odd: BQ words.
    template <bool SECOND>
    static __device__ __forceinline__ void run(const AttnBackwardParams &p, const SeqTile &s,
                                               int wave, unsigned char *lds, int *vote, int *odd) {
        const int lane = threadIdx.x & 63, c = lane & 15, g4 = lane >> 4, pair = wave & 3;
        const int len = s.len, kh = s.head / p.split, part = s.head % p.split;
        const int64_t tok0 = s.tok0;
        const int g = p.Hq / p.Hk;
        const int j0 = kh * g + part * g / p.split, j1 = kh * g + (part + 1) * g / p.split;
        const int k0 = s.tile * kRows, w0 = k0 + pair * CT * 16;

        Frag<DT> of[D / 32][CT];  // the keys, or the values
        const int64_t kvstride = (int64_t)p.Hk * D;
        const DT *rows = static_cast<const DT *>(SECOND ? p.v : p.k);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const int64_t at = (tok0 + min(w0 + 16 * ct + c, len - 1)) * kvstride + kh * D;
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) of[kk][ct] = R::load(rows + at, kk, g4);
        }
        f32x4 acc[D / 16][CT];
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) acc[dt][ct] = zero4();
        const int64_t stride = (int64_t)p.Hq * D * sizeof(DT);
        const float scale2 = p.scale * kLog2e;
        const int first = k0 / BQ * BQ;  // the first query tile that sees any of these keys

        auto issue = [&](int j, int q, unsigned char *buf) {
            DenseKeys src{
                static_cast<const unsigned char *>(p.q) + tok0 * stride + j * R::kPitch,
                static_cast<const unsigned char *>(p.dout) + tok0 * stride + j * R::kPitch,
                stride, len};
            Tiles::issue(src, q, (uint32_t)stride, buf, wave, lane);
            if (wave < 3) {
                const float *st = p.stats + ((int64_t)wave * p.Hq + j) * p.total + tok0 + q;
                dma4_async(uniform(reinterpret_cast<const unsigned char *>(st)),
                           (uint32_t)min(lane, len - 1 - q) * 4, buf + 2 * kTile + wave * 256);
            }
        };
        const int steps = (len - first + BQ - 1) / BQ * (j1 - j0);
        issue(j0, first, lds);
        int j = j0, q = first, qlast = first;  // tile `step`; tile `step - 1`
        int now = 0;                           // its buffer
        for (int step = 0; step <= steps; ++step) {
            wait_copies<0>();
            __syncthreads();
            const int next = now == 2 ? 0 : now + 1, before = now == 0 ? 2 : now - 1;
            const bool wrap = q + BQ >= len;
            if (step + 1 < steps)
                issue(wrap ? j + 1 : j, wrap ? first : q + BQ, lds + next * kBuf);
            unsigned char *buf = lds + now * kBuf;
            if (step < steps && (q < k0 + kRows || q + BQ > len)) {
                int *const flag = vote + (step & 1);
                if (__any(odd_part<DT>(buf, 2 * kTile))) *flag = 1;
                __syncthreads();
                if (__builtin_amdgcn_readfirstlane(*flag)) {
                    // queries and gradients that are not finite make NaN of the keys that
                    // they reach and are taken out of the products
                    odd_rows<DT, D>(buf, BQ, 2, odd);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        bool nan = false;
                        for (int row = 0; row < BQ; ++row)
                            nan |= odd[row] && q + row >= w0 + 16 * ct + c && q + row < len;
                        if (nan) {
#pragma unroll
                            for (int dt = 0; dt < D / 16; ++dt)
                                acc[dt][ct] = zero4() + __builtin_nanf("");
                        }
                    }
                    if (threadIdx.x == 0) *flag = 0;
                    __syncthreads();
                    clear_odd<DT>(buf, 2 * kTile);
                    __syncthreads();
                }
            }
            const int mine = SECOND ? step - 1 : step, qm = SECOND ? qlast : q;
            if (mine >= 0 && mine < steps) {
                const unsigned char *tile = SECOND ? lds + before * kBuf : buf;
                unsigned char *ps = lds + 3 * kBuf + ((mine & 1) * 4 + pair) * kP;
                const float *stat =
                    reinterpret_cast<const float *>(tile + 2 * kTile) + (SECOND ? 64 : 0);
                const unsigned char *yt = SECOND ? tile + kTile : tile;  // the scores' rows
                const unsigned char *xt = SECOND ? tile : tile + kTile;  // the sums'
#pragma unroll 1
                for (int sub = 0; sub < BQ; sub += 32) {
                    const int qs = qm + sub;
                    if (qs >= len) break;
                    if (qs + 31 < w0 || w0 >= len) continue;  // before all of the pair's keys
                    f32x4 sc[2][CT];
                    A::scores(yt, sub, of, sc, lane);
                    // keys from len on see no query of these either
                    const bool cut = qs < w0 + CT * 16 || qs + 32 > len;
                    const int before_me = w0 + (lane & 15) - qs - 4 * g4;
                    const int left = len - qs - 4 * g4;
                    u32x4 *const pp =
                        reinterpret_cast<u32x4 *>(ps + sub / 32 * CT * 1024) + lane;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const float *of = stat + sub + 16 * t + 4 * g4;
                        const f32x4 st = *reinterpret_cast<const f32x4 *>(of);
                        f32x4 fa;
                        if constexpr (!SECOND) fa = *reinterpret_cast<const f32x4 *>(of + 128);
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const float w = sc[t][ct][r];
                                if constexpr (SECOND)
                                    sc[t][ct][r] = w - st[r];
                                else
                                    sc[t][ct][r] = exp2_fast(fmaf(w, scale2, -st[r])) * fa[r];
                            }
                    }
                    Frag<DT> f[CT];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        u32x4 h;
                        if constexpr (SECOND) h = pp[ct * 64];
                        if constexpr (SECOND) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                sc[i >> 2][ct][i & 3] *=
                                    i & 1 ? code_value<1>(h[i / 2]) : code_value<0>(h[i / 2]);
                        }
                        if (cut) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int row = 16 * (i >> 2) + (i & 3);
                                if (row < before_me + 16 * ct || row >= left)
                                    sc[i >> 2][ct][i & 3] = 0.f;
                            }
                        }
                        c_to_frag(sc[0][ct], sc[1][ct], f[ct]);
                        if constexpr (!SECOND) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                h[i] = code_pair(sc[i >> 1][ct][2 * (i & 1)],
                                                 sc[i >> 1][ct][2 * (i & 1) + 1]);
                            pp[ct * 64] = h;
                        }
                    }
                    A::add_to(acc, xt, sub, f, lane);
                }
            }
            qlast = q;
            q = wrap ? first : q + BQ;
            j += wrap;
            now = next;
        }
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const int row = w0 + 16 * ct + c;
            if (row >= len) continue;
            const int64_t at = (tok0 + row) * kvstride + kh * D + 4 * g4;
            const int64_t all = p.total * kvstride;
            const float scale = SECOND ? p.scale : 1.f;
            DT *to = static_cast<DT *>(SECOND ? p.dk : p.dv) + at;
            float *parts = p.parts + (2 * part + (SECOND ? 0 : 1)) * all + at;
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) {
                const f32x4 x = acc[dt][ct] * scale;
                if (p.split == 1)
                    store4(to + 16 * dt, x);
                else
                    store4(parts + 16 * dt, x);
            }
        }
    }
};

template <typename DT, int D, int CT, int BQ>
__global__ __launch_bounds__(512, 2) void attn_dkv_pair_kernel(AttnBackwardParams p,
                                                               HeadOrder order) {
    using Pairs = KeyPairs<DT, D, CT, BQ>;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    __shared__ int odd[BQ], vote[2];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int unit, slot;
    if (!order.pick(workgroup(), unit, slot)) return;
    const SeqTile s = seq_tile<Pairs::kRows>(p.cu, p.N, p.T, p.total, unit, slot, order.tiles,
                                             p.Hk * p.split, threadIdx.x & 63);
    if (s.tile >= s.tiles) return;
    if (threadIdx.x < 2) vote[threadIdx.x] = 0;
    if (wave < 4)
        Pairs::template run<false>(p, s, wave, lds, vote, odd);
    else
        Pairs::template run<true>(p, s, wave, lds, vote, odd);
}

// dk and dv from the parts over the query heads, in order; four elements per thread.
template <typename DT>
__global__ __launch_bounds__(256) void attn_dkv_join_kernel(AttnBackwardParams p, int64_t all) {
    const int64_t i = ((int64_t)workgroup() * 256 + threadIdx.x) * 4;
    const int64_t per = all / p.total, end = p.cu ? clamped(p.cu, p.N, p.total) : p.total;
    if (i >= 2 * all || (i < all ? i : i - all) >= end * per) return;  // behind the sequences
    f32x4 x = *reinterpret_cast<const f32x4 *>(p.parts + i);
    for (int s = 1; s < p.split; ++s)
        x += *reinterpret_cast<const f32x4 *>(p.parts + 2 * s * all + i);
    store4(i < all ? static_cast<DT *>(p.dk) + i : static_cast<DT *>(p.dv) + (i - all), x);
}

template <typename DT, int D> struct Shape {
    static constexpr bool kWide = sizeof(DT) == 4;
    // queries and dout in registers beside the sums (bf16: 32 rows per wave, the first 32 in one)
    static constexpr int kQCT = kWide ? 1 : 2;
    static constexpr int kQNW = kWide ? (D == 256 ? 4 : 8) : 4;
    static constexpr int kQBK = kWide && D == 256 ? 32 : 64;
    static constexpr int kQPer = D == 256 ? 1 : 2;
    // keys and values; bf16: wave pairs
    static constexpr int kKCT = kWide ? 1 : D == 64 ? 4 : D == 128 ? 3 : 2;
    static constexpr int kKBQ = D == 64 || (!kWide && D == 128) ? 64 : 32;
    static constexpr int kKPer = D == 256 ? 1 : 2;
    static constexpr int kBN = 4 * kKCT * 16;
};

template <typename DT, int D>
hipError_t launch(const AttnBackwardParams &p, int cus, hipStream_t stream) {
    using S = Shape<DT, D>;
    attn_stats_kernel<DT, D><<<grid_of((p.total * p.Hq + 15) / 16, 256), 256, 0, stream>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    auto order = [&](int64_t heads, int rows) {
        return p.cu ? HeadOrder::make(heads, p.total / rows + p.N)
                    : HeadOrder::make(p.N * heads, (p.T + rows - 1) / rows);
    };
    auto dq = [&](auto waves) {  // as the forward pass chooses: fewer waves where CUs are left
        constexpr int NW = decltype(waves)::value;
        constexpr int kLds = KeyTiles<DT, D, S::kQCT, NW, S::kQBK>::kLds;
        const auto kernel = attn_dq_kernel<DT, D, S::kQCT, NW, S::kQBK, S::kQPer>;
        const hipError_t e = with_lds(kernel, kLds);
        if (e != hipSuccess) return e;
        const HeadOrder o = order(p.Hq, NW * S::kQCT * 16);
        kernel<<<grid_of(o.grid(), 64 * NW), 64 * NW, kLds, stream>>>(p, o);
        return hipGetLastError();
    };
    constexpr int kRows = S::kQNW * S::kQCT * 16;
    const int64_t tiles = p.cu ? p.total / kRows + 1 : p.N * ((p.T + kRows - 1) / kRows);
    constexpr int kSmall = S::kWide || D == 256 ? 2 : S::kQNW;
    e = tiles * p.Hq >= cus ? dq(std::integral_constant<int, S::kQNW>{})
                            : dq(std::integral_constant<int, kSmall>{});
    if (e != hipSuccess) return e;
    const HeadOrder o = order((int64_t)p.Hk * p.split, S::kBN);
    if constexpr (S::kWide) {
        constexpr int kLds = KeyTiles<DT, D, S::kKCT, 4, S::kKBQ>::kLds + 2 * 768;
        const auto kernel = attn_dkv_kernel<DT, D, S::kKCT, 4, S::kKBQ, S::kKPer>;
        if ((e = with_lds(kernel, kLds)) != hipSuccess) return e;
        kernel<<<grid_of(o.grid(), 256), 256, kLds, stream>>>(p, o);
    } else {
        constexpr int kLds = KeyPairs<DT, D, S::kKCT, S::kKBQ>::kLds;
        const auto kernel = attn_dkv_pair_kernel<DT, D, S::kKCT, S::kKBQ>;
        if ((e = with_lds(kernel, kLds)) != hipSuccess) return e;
        kernel<<<grid_of(o.grid(), 512), 512, kLds, stream>>>(p, o);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (p.split > 1) {
        const int64_t all = p.total * p.Hk * D;
        attn_dkv_join_kernel<DT>
            <<<grid_of((2 * all / 4 + 255) / 256, 256), 256, 0, stream>>>(p, all);
        e = hipGetLastError();
    }
    return e;
}

template <typename DT, int D> int key_rows() { return Shape<DT, D>::kBN; }

}  // namespace

// Workgroups that share a key tile's query heads: as few as give the device two workgroups
// per CU (each part is written and read once more, in fp32). 2 x 4,097 tokens of 16/4 heads
// of 128, forward and backward: 714 us so, 751 with one per CU as the target.
int32_t attn_backward_split(int64_t N, int64_t T, int64_t total, int32_t Hq, int32_t Hk, int D,
                            int dtype, bool packed, int cus) {
    const int rows = dtype == 1 ? (D == 64    ? key_rows<__bf16, 64>()
                                   : D == 128 ? key_rows<__bf16, 128>()
                                              : key_rows<__bf16, 256>())
                                : (D == 64    ? key_rows<float, 64>()
                                   : D == 128 ? key_rows<float, 128>()
                                              : key_rows<float, 256>());
    const int64_t tiles = packed ? total / rows + N : N * ((T + rows - 1) / rows);
    int32_t split = 1;
    const int32_t g = Hq / Hk;
    while (split < g && tiles * Hk * split < 2 * (int64_t)cus) {
        ++split;
        while (g % split) ++split;
    }
    return split;
}

hipError_t launch_attn_backward(const AttnBackwardParams &p, int dtype, int D, int cus,
                                hipStream_t stream) {
    if (dtype == 1)
        return D == 64    ? launch<__bf16, 64>(p, cus, stream)
               : D == 128 ? launch<__bf16, 128>(p, cus, stream)
                          : launch<__bf16, 256>(p, cus, stream);
    return D == 64    ? launch<float, 64>(p, cus, stream)
           : D == 128 ? launch<float, 128>(p, cus, stream)
                      : launch<float, 256>(p, cus, stream);
}

}  // namespace gdn
