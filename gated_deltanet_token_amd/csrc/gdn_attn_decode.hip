// gdn_attn_decode.hip -- softmax attention of new tokens against a paged cache
// (gfx950), with prefixes that groups of sequences share.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(c q . k_j - m)
// over the keys of the shared prefix and of the sequence's own pages. Sums over
// any parts of the keys join by their references:
//   m = max m_i,  l = sum l_i 2^(m_i - m),  acc = sum acc_i 2^(m_i - m).
//
// attn_few_kernel: at most 32 query rows per key head and sequence (tokens times
// the query heads of a key head). Bound by HBM: each cached key and value is
// read once. All sequences' tiles of 32 keys, one after the other, are dealt out
// to the workgroups in equal runs, whatever the lengths; the waves of a workgroup
// stream tiles of their own through LDS of their own, no barrier between them, so
// that every wave always has a tile of keys or of values under way. 64 sequences of up
// to 16,384 tokens, 24/4 heads of 256, with the join: 102 us, 5.1 TB/s. The matrix instructions
// have time to spare: bf16 weights are two terms, rounded and rest, so that nothing but the result
// is rounded (102 us either way; with 4 new tokens each, 24 rows, 128 us, in one term 125).
//
// attn_rows_kernel: many query rows against one run of keys: the rows of all
// sequences of a group against their prefix (read once for all of them), or
// the rows of a long run of new tokens. The tiles are those of the prompts' kernel
// (gdn_attn_fwd.hip), dealt out in the same way. Bound by the matrix instructions: 64
// sequences behind 32,768 shared tokens 83 us for 51 GFLOP, of whose row tiles a quarter is
// empty (384 rows in tiles of 256); the whole call 113 us. A piece of 512 tokens of each of 4
// prompts behind 7,680 cached ones, 24/4 heads of 256: 425 us, 940 TFLOP/s; with nothing cached
// 83 us, 156 TFLOP/s, since every row tile is dealt out as if it saw all keys.
//
// attn_join_kernel: the parts of every row, in a fixed order. Bound by latency: 32
// parts of 1,536 rows 13 us (50 MB, 3.9 TB/s).
#include "gdn_attn.hpp"

namespace gdn {

namespace {

// Rows per (sequence, key head) that attn_few_kernel takes. With 24 rows of 64 sequences of up
// to 16,384 tokens (24/4 heads of 256, 4 new tokens) it takes 128 us, attn_rows_kernel 142; with
// 32 fp32 rows of 32 sequences (16/4 heads of 128) 51 against 66. More rows do not fit its
// registers.
constexpr int kFewRows = 32;
constexpr int kFewKeys = 32;   // keys per wave and step there
constexpr int kFewTiles = 4;   // tiles of a workgroup at the least
// What starting and ending a unit costs, in tiles: with 3, 6 and 12, 64 sequences of up to 16,384
// tokens of 24/4 heads of 256 take 111, 101 and 102 us, of 16/4 heads of 64 36, 32 and 32; 64 of
// up to 4,096 fp32 tokens of 16/4 heads of 128 49, 43 and 49.
constexpr int kFewStart = 6;

// The keys of a sequence, or of a prefix, in a paged cache, 16 at a time (pages hold whole
// ones). operator() reads page numbers 64 at a time into a register and takes them from there
// lane by lane: scalar loads, one per 16 keys, are waited for together with every LDS read (64
// sequences behind 32,768 shared tokens, 24/4 heads of 256: 123 us, so 115). attn_few_kernel is
// as fast with scalar loads (102 us either way for 64 sequences of up to 16,384 tokens).
struct PagedKeys {
    const unsigned char *k, *v;  // the pools, at this head
    const int32_t *table;
    int64_t stride;  // bytes per cached token
    int len, shift, num_pages;
    bool outside;  // longer than its table: every score is NaN
    int at = -1, pages = 0;  // the page of 16 keys number at + lane

    __device__ __forceinline__ KeyRows rows(int page, int first) const {
        const bool bad = (unsigned)page >= (unsigned)num_pages;
        const int64_t row = ((int64_t)(bad ? 0 : page) << shift) + (first & ((1 << shift) - 1));
        return KeyRows{k + row * stride, v + row * stride, min(16, len - first), bad};
    }
    __device__ __forceinline__ int page_of(int key) const {  // any lane, any key
        return outside ? -1 : table[min(key, len - 1) >> shift];
    }
    __device__ __forceinline__ KeyRows operator()(int key) {
        const int first = min(key, len - 1), n = first >> 4;
        if (at < 0 || (unsigned)(n - at) >= 64u) {
            at = n;
            pages = page_of(n * 16 + (int)(threadIdx.x & 63) * 16);
        }
        return rows(__builtin_amdgcn_readlane(pages, n - at), first);
    }
};
// Keys that a table of `most` can hold: longer ones stand for one key with a NaN score.
__device__ __forceinline__ int table_len(int length, int64_t most) {
    return length < 0 ? 0 : length > most ? 1 : length;
}
__device__ __forceinline__ int tiles_of(int len) { return max(1, (len + kFewKeys - 1) / kFewKeys); }

// What the workgroups of one kind leave for the join: sums of a unit's rows over a part of its
// keys, in slots; a unit's parts are in neighbouring ones.
struct Parts {
    int32_t wgs;     // workgroups that share the work (few: 0: one per unit)
    float *acc;      // [slots][rows of a unit][D]
    float *ml;       // [slots][rows of a unit][2]: reference and sum of weights
    int32_t *units;  // [units][2]: a unit's first slot and how many parts it has
};

struct DecodePlan {
    AttnDecodeParams p;
    int32_t rows;  // K * Hq / Hk per (sequence, key head)
    bool few;      // own keys by attn_few_kernel
    Parts pre, own;
};

__device__ __forceinline__ int64_t row_index(const DecodePlan &d, int b, int r, int h) {
    const int g = d.p.Hq / d.p.Hk, t = r / g;
    return ((int64_t)b * d.p.K + t) * d.p.Hq + h * g + (r - t * g);
}

__device__ __forceinline__ int own_len(const AttnDecodeParams &p, int b) {
    return table_len(p.lengths[b], (int64_t)p.max_pages << p.page_shift);
}

// Sums over a workgroup of NT threads; red: NT / 64 + 1 words.
template <int NT> __device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *red,
                                                                int64_t &all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 63) red[wave] = x;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        if (w < wave) x += red[w];
        all += red[w];
    }
    return x;
}

// How the work is dealt out. Every entry (a sequence, or a group) has Hk times places(entry)
// places in a row, entries in order; workgroup w takes `per` of them. A unit of work takes a
// few places for its start (queries, first pages and keys, its end), then some for each tile
// of keys; a tile is the workgroup's that has its first place.
struct Deal {
    int64_t per, at, end;  // places per workgroup; this workgroup's, none: at >= end
    int64_t front;         // places in front of the entry, over Hk
    int entry;             // the one that place `at` belongs to

    template <int NT, typename F>
    __device__ __forceinline__ void make(int entries, int Hk, int wgs, int64_t least, int64_t wg,
                                         int64_t *red, F &&places) {
        int64_t mine = 0, sum = 0, all;
        for (int i = threadIdx.x; i < entries; i += NT) sum += mine = places(i);
        int64_t upto = block_scan<NT>(sum, red, all);
        per = (all * Hk + wgs - 1) / wgs;
        per = per < least ? least : per;
        at = wg * per;
        end = min(at + per, all * Hk);
        front = 0;
        entry = 0;
        if (at >= end) return;
        // the scan above has the answer where every thread holds one entry
        for (int e0 = 0; e0 < entries; e0 += NT) {
            if (entries > NT) {
                mine = e0 + (int)threadIdx.x < entries ? places(e0 + threadIdx.x) : 0;
                upto = front + block_scan<NT>(mine, red, all);
            }
            __syncthreads();
            if ((int)threadIdx.x < entries - e0 && (upto - mine) * Hk <= at && at < upto * Hk) {
                red[0] = e0 + threadIdx.x;
                red[1] = upto - mine;
            }
            __syncthreads();
            front += all;
            if (at < front * Hk) break;
        }
        entry = __builtin_amdgcn_readfirstlane((int)red[0]);
        front = uniform(red[1]);
        per = uniform(per);
        at = uniform(at);
        end = uniform(end);
    }
};

template <typename DT, int D, int CT, int NW>
__global__ __launch_bounds__(64 * NW, 1) void attn_few_kernel(DecodePlan d) {
    using R = Rows<DT, D>;
    constexpr int kRing = 2 * kFewKeys * R::kPitch;  // a wave's keys and values
    constexpr int kHalf = kFewKeys * R::kPitch;
    constexpr int kCopies = 2 * R::kCopies;          // copies of one half
    static_assert(CT * 16 * D * 4 <= kRing, "a wave's sums fit its ring");
    static_assert(kCopies < 64, "vmcnt");
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    __shared__ float ml[NW][2][16 * CT];
    __shared__ int64_t red[NW + 2];
    const AttnDecodeParams &p = d.p;
    const int lane = threadIdx.x & 63, c = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    unsigned char *kt = lds + wave * kRing, *vt = kt + kHalf;
    const float scale2 = p.scale * kLog2e;
    const uint32_t stride = (uint32_t)p.Hk * D * sizeof(DT);

    const int wg = workgroup();
    int64_t at = 0, end = 0;  // places of this workgroup
    int64_t unit = 0;         // first place of the unit
    Deal deal;
    int b;
    if (d.own.wgs) {
        deal.make<64 * NW>(p.B, p.Hk, d.own.wgs, kFewTiles + kFewStart, wg, red,
                           [&](int i) { return tiles_of(own_len(p, i)) + kFewStart; });
        at = deal.at;
        end = deal.end;
        if (at >= end) return;
        b = deal.entry;
    } else {
        b = wg / p.Hk;
        if (b >= p.B) return;
    }
    b = __builtin_amdgcn_readfirstlane(b);
    int h;  // key head
    int len = __builtin_amdgcn_readfirstlane(own_len(p, b)), tiles = tiles_of(len);
    if (d.own.wgs) {
        const int64_t first = deal.front * p.Hk;
        h = __builtin_amdgcn_readfirstlane((int)((at - first) / (tiles + kFewStart)));
        unit = first + (int64_t)h * (tiles + kFewStart);
    } else {
        h = wg - b * p.Hk;
        at = kFewStart;
        end = at + tiles;
    }
    while (true) {
        // the tiles of this unit at places at .. end - 1
        const int64_t from = unit + kFewStart;
        const int t0 = __builtin_amdgcn_readfirstlane((int)max((int64_t)0, at - from));
        const int t1 =
            __builtin_amdgcn_readfirstlane((int)max((int64_t)0, min((int64_t)tiles, end - from)));
        if (t0 >= t1) return;  // the places end before the unit's first tile
        PagedKeys src{};
        src.at = -1;
        src.k = static_cast<const unsigned char *>(p.kc) + h * R::kPitch;
        src.v = static_cast<const unsigned char *>(p.vc) + h * R::kPitch;
        src.table = p.table + (int64_t)b * p.max_pages;
        src.stride = stride;
        src.len = len;
        src.shift = p.page_shift;
        src.num_pages = p.num_pages;
        src.outside = p.lengths[b] > (int64_t)p.max_pages << p.page_shift;

        Frag<DT> qf[D / 32][CT];
        int lim[CT];
        const DT *q = static_cast<const DT *>(p.q);
        const int g = p.Hq / p.Hk;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const int r = min(16 * ct + c, d.rows - 1);
            lim[ct] = src.outside ? 1 : max(0, len - p.K + 1 + r / g);
            const DT *row = q + row_index(d, b, r, h) * D;
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) qf[kk][ct] = R::load(row, kk, g4);
        }
        const int lo = src.outside ? 0 : max(0, len - p.K + 1);  // keys that every row sees

        Attend<DT, D, CT> st;
        st.clear();
        int t = t0 + wave;
        const bool some = t < t1 && len > 0;
        auto half_of = [&](int tile, int half) {
            const int first = min(tile * kFewKeys + 16 * half, len - 1);
            return src.rows(__builtin_amdgcn_readfirstlane(src.page_of(first)), first);
        };
        KeyRows now[2], next[2];
        if (some) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                now[half] = half_of(t, half);
                R::copy16(now[half].k, stride, now[half].rows, kt + half * 16 * R::kPitch, lane);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half)
                R::copy16(now[half].v, stride, now[half].rows, vt + half * 16 * R::kPitch, lane);
        }
        if (some)
            for (; t < t1; t += NW) {
                const int key = t * kFewKeys;
                const bool more = t + NW < t1;
                if (more) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) next[half] = half_of(t + NW, half);
                }
                f32x4 s[2][CT];
                Frag<DT> w[1][CT], low[CT];
                wait_copies<kCopies>();  // the keys; the values are still under way
                st.scores(kt, 0, qf, s, lane);
                if (more) {
                    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the keys have been read
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        R::copy16(next[half].k, stride, next[half].rows,
                                  kt + half * 16 * R::kPitch, lane);
                }
                const bool cut = key + kFewKeys > lo;
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    if (now[half].bad) {
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct)
                            s[half][ct] = zero4() + __builtin_nanf("");
                    }
                int seen[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) seen[ct] = lim[ct] - key;
                if (cut) st.mask(s, seen, lane);
                st.settle(s, scale2);
                st.weights(s, w, scale2);
                if constexpr (sizeof(DT) == 2) st.rest(s, w[0], low);
                if (more)
                    wait_copies<kCopies>();
                else
                    wait_copies<0>();
                if (cut) {  // some row does not see all of the tile
                    bool odd = false;
                    for (int i = lane; i < kHalf / 16; i += 64)
                        odd |= not_finite(reinterpret_cast<const u32x4 *>(vt)[i], DT{});
                    if (__any(odd)) {
                        st.mark_odd(vt, 0, seen, lane);
                        for (int i = lane; i < kHalf / 16; i += 64) {
                            u32x4 &x = reinterpret_cast<u32x4 *>(vt)[i];
                            x = only_finite(x, DT{});
                        }
                    }
                }
                if constexpr (sizeof(DT) == 2) {
                    const Frag<DT> *const terms[2] = {w[0], low};
                    st.add_terms(st.acc, vt, 0, terms, lane);
                } else {
                    st.add(vt, 0, w[0], lane);
                }
                if (more) {
                    __builtin_amdgcn_s_waitcnt(0xC07F);  // the values have been read
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        R::copy16(next[half].v, stride, next[half].rows,
                                  vt + half * 16 * R::kPitch, lane);
#pragma unroll
                    for (int half = 0; half < 2; ++half) now[half] = next[half];
                }
            }
        st.finish();

        // the waves' sums, joined in order
        float *sums = reinterpret_cast<float *>(kt);
        auto place = [](int row, int dd) { return Rows<float, D>::at(row, dd) / 4; };
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt)
                *reinterpret_cast<f32x4 *>(sums + place(16 * ct + c, 16 * dt + 4 * g4)) =
                    st.acc[dt][ct];
            if (g4 == 0) {
                ml[wave][0][16 * ct + c] = st.mc[ct];
                ml[wave][1][16 * ct + c] = st.l[ct];
            }
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == tiles && !p.ptable;
        const int64_t slot = (d.own.wgs ? wg : 0) + (int64_t)b * p.Hk + h;
        if (d.own.units && t0 == 0 && threadIdx.x == 0) {
            const int parts = d.own.wgs ? (int)((from + tiles - 1) / deal.per) - wg + 1 : 1;
            *reinterpret_cast<int2 *>(d.own.units + ((int64_t)b * p.Hk + h) * 2) =
                make_int2((int)slot, parts);
        }
        for (int i = threadIdx.x; i < d.rows * (D / 4); i += 64 * NW) {
            const int row = i / (D / 4), dd = i % (D / 4) * 4;
            float m = ml[0][0][row];
#pragma unroll
            for (int x = 1; x < NW; ++x) m = fmaxf(m, ml[x][0][row]);
            float l = 0.f;
            f32x4 a = zero4();
#pragma unroll
            for (int x = 0; x < NW; ++x) {
                const float mx = ml[x][0][row];
                // no key seen, or scores of -inf alone: sums of 0, or NaN
                const float f = mx == -__builtin_inff() ? 1.f : exp2_fast(mx - m);
                l += ml[x][1][row] * f;
                const float *from = reinterpret_cast<const float *>(lds + x * kRing);
                a += *reinterpret_cast<const f32x4 *>(from + place(row, dd)) * f;
            }
            if (whole) {
                const int64_t o = row_index(d, b, row, h);
                store4(static_cast<DT *>(p.out) + o * D + dd, a * (l == 0.f ? 0.f : 1.f / l));
                if (p.lse && dd == 0)
                    p.lse[o] = l == 0.f ? -__builtin_inff() : m * kLn2 + logf(l);
            } else {
                *reinterpret_cast<f32x4 *>(d.own.acc + (slot * d.rows + row) * D + dd) = a;
                if (dd == 0) {
                    d.own.ml[(slot * d.rows + row) * 2] = m;
                    d.own.ml[(slot * d.rows + row) * 2 + 1] = l;
                }
            }
        }
        unit += tiles + kFewStart;
        at = unit;
        if (!d.own.wgs || at >= end) return;
        __syncthreads();
        if (++h == p.Hk) {
            h = 0;
            ++b;
            len = __builtin_amdgcn_readfirstlane(own_len(p, b));
            tiles = tiles_of(len);
        }
    }
}

// Query rows against one run of keys: a group's against its prefix (PREFIX), or a sequence's
// against its own.
// Places of a unit's start, and of a tile of keys where all or more than half of the rows are
// there, or less. Taken from bf16 heads of 256 (64 sequences behind 32,768 shared tokens: start 10,
// 20, 40: 114.6, 112.4, 114.0 us; half 5, 7, 10: 125, 112.4, 115.4) and used for all. Others would
// gain up to 9 % from values of their own: 17 x 4 fp32 tokens of 128 78 us, with half 10 72; fp32
// heads of 64 48 us, with start 40 44.5; bf16 heads of 128 49.3 us, with half 10 47.2.
constexpr int kRowsStart = 20;
constexpr int kRowsFull = 10, kRowsHalf = 7;
constexpr int kRowsTiles = 4;             // tiles of a workgroup at the least
struct RowRun {
    int first, rows, len;  // first sequence
    bool outside;
};
template <bool PREFIX> __device__ __forceinline__ RowRun row_run(const DecodePlan &d, int i) {
    const AttnDecodeParams &p = d.p;
    if constexpr (PREFIX) {
        const int first = (int)clamped(p.pgroups, i, p.B);
        const int last = (int)clamped(p.pgroups, i + 1, p.B);
        const int64_t most = (int64_t)p.max_ppages << p.page_shift;
        return RowRun{first, max(0, last - first) * d.rows, table_len(p.plengths[i], most),
                      p.plengths[i] > most};
    } else {
        return RowRun{i, d.rows, own_len(p, i),
                      p.lengths[i] > (int64_t)p.max_pages << p.page_shift};
    }
}
// Row tiles of a run: full ones, and whether the last is half full at the most.
template <int BM> struct RowTiles {
    int full, tiles, full_places, half_places;
    template <int BK> static __device__ __forceinline__ RowTiles of(const RowRun &r) {
        RowTiles t;
        const int over = r.rows % BM;
        t.full = r.rows / BM + (over > BM / 2);
        t.tiles = t.full + (over > 0 && over <= BM / 2);
        const int keys = max(1, (r.len + BK - 1) / BK);
        t.full_places = kRowsStart + kRowsFull * keys;
        t.half_places = kRowsStart + kRowsHalf * keys;
        return t;
    }
    __device__ __forceinline__ int64_t places() const {
        return (int64_t)full * full_places + (tiles > full ? half_places : 0);
    }
};
// Units of the runs in front of entry i, at the most.
template <bool PREFIX, int BM>
__device__ __forceinline__ int64_t units_before(const DecodePlan &d, int i, int first) {
    return PREFIX ? (int64_t)first * d.rows / BM + i : (int64_t)i * ((d.rows + BM - 1) / BM);
}

template <typename DT, int D, int CT, int NW, int BK, int PER_SIMD, bool PREFIX>
__global__ __launch_bounds__(64 * NW, PER_SIMD) void attn_rows_kernel(DecodePlan d) {
    // the loop over units leaves fewer registers than the prompts' kernel has
    constexpr bool FRESH = sizeof(DT) == 4 || D > 64;
    using Tiles = KeyTiles<DT, D, CT, NW, BK, FRESH>;
    using R = Rows<DT, D>;
    constexpr int BM = NW * CT * 16;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    __shared__ int64_t red[NW + 2];
    const AttnDecodeParams &p = d.p;
    const Parts &parts = PREFIX ? d.pre : d.own;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wg = workgroup();
    const int entries = PREFIX ? p.G : p.B;
    Deal deal;
    deal.make<64 * NW>(entries, p.Hk, parts.wgs, kRowsStart + kRowsTiles * kRowsFull, wg, red,
                       [&](int i) {
                           return RowTiles<BM>::template of<BK>(row_run<PREFIX>(d, i)).places();
                       });
    int64_t at = deal.at;
    const int64_t end = deal.end;
    if (at >= end) return;
    int i = deal.entry;
    RowRun run = row_run<PREFIX>(d, i);
    RowTiles<BM> rt = RowTiles<BM>::template of<BK>(run);
    const int64_t in = at - deal.front * p.Hk;
    int h = __builtin_amdgcn_readfirstlane((int)(in / rt.places()));
    const int64_t rest = in - h * rt.places();
    int tile = __builtin_amdgcn_readfirstlane((int)min(rest / rt.full_places, (int64_t)rt.full));
    int64_t unit = uniform(deal.front * p.Hk + h * rt.places() + (int64_t)tile * rt.full_places);
    while (true) {
        const int cost = tile < rt.full ? kRowsFull : kRowsHalf;
        const int places = tile < rt.full ? rt.full_places : rt.half_places;
        const int keys = (places - kRowsStart) / cost;  // tiles of keys
        const int64_t from = unit + kRowsStart;
        const int t0 = __builtin_amdgcn_readfirstlane(
            at <= from ? 0 : (int)min((int64_t)keys, (at - from + cost - 1) / cost));
        const int t1 = __builtin_amdgcn_readfirstlane(
            end <= from ? 0 : (int)min((int64_t)keys, (end - from + cost - 1) / cost));
        if (t0 < t1) {
            const int r0 = tile * BM, rows = run.rows, first = run.first;
            const int len = __builtin_amdgcn_readfirstlane(run.len);
            const int64_t stride = (int64_t)p.Hk * D * sizeof(DT);
            PagedKeys src{};
            src.at = -1;
            src.k = static_cast<const unsigned char *>(p.kc) + h * R::kPitch;
            src.v = static_cast<const unsigned char *>(p.vc) + h * R::kPitch;
            src.table = PREFIX ? p.ptable + (int64_t)i * p.max_ppages
                               : p.table + (int64_t)i * p.max_pages;
            src.stride = stride;
            src.len = len;
            src.shift = p.page_shift;
            src.num_pages = p.num_pages;
            src.outside = run.outside;

            const int g = p.Hq / p.Hk, w0 = r0 + wave * CT * 16;
            // keys that row r of this run sees
            auto sees = [&](int r) {
                return PREFIX || run.outside ? len : max(0, len - p.K + 1 + r / g);
            };
            auto place = [&](int r) {  // in q and out
                const int s = PREFIX ? r / d.rows : 0;
                return row_index(d, first + s, r - s * d.rows, h);
            };
            Frag<DT> qf[D / 32][CT];
            int lim[CT];
            const DT *q = static_cast<const DT *>(p.q);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int lane = threadIdx.x & 63, g4 = lane >> 4;
                const int r = min(w0 + 16 * ct + (lane & 15), rows - 1);
                lim[ct] = sees(r);
                const DT *row = q + place(r) * D;
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk) qf[kk][ct] = R::load(row, kk, g4);
            }
            const int last = sees(min(r0 + BM, rows) - 1);  // keys that any row sees
            const int key0 = t0 * BK, key1 = min(t1 * BK, last);
            Attend<DT, D, CT, FRESH> st;
            st.clear();
            const int hi = w0 < rows ? sees(min(w0 + CT * 16, rows) - 1) : 0;
            Tiles::template run<true>(st, qf, src, key0, key1, lim, sees(r0),
                                      sees(min(w0, rows - 1)), hi, (uint32_t)stride,
                                      p.scale * kLog2e, lds);
            st.finish();
            const bool whole = !PREFIX && t0 == 0 && t1 == keys && !p.ptable;
            const int64_t u = units_before<PREFIX, BM>(d, i, first) * p.Hk + h * rt.tiles + tile;
            if (parts.units && t0 == 0 && threadIdx.x == 0) {
                const int64_t w1 = (from + (int64_t)(keys - 1) * cost) / deal.per;
                *reinterpret_cast<int2 *>(parts.units + u * 2) =
                    make_int2((int)(wg + u), (int)(w1 - wg) + 1);
            }
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int lane = fresh(threadIdx.x & 63), g4 = lane >> 4;
                const int r = w0 + 16 * ct + (lane & 15);
                if (r >= rows) continue;
                if (whole) {
                    const int64_t o = place(r);
                    const float inv = st.l[ct] == 0.f ? 0.f : 1.f / st.l[ct];
                    DT *to = static_cast<DT *>(p.out) + o * D + 4 * g4;
#pragma unroll
                    for (int dt = 0; dt < D / 16; ++dt)
                        store4(to + 16 * dt, st.acc[dt][ct] * inv);
                    if (p.lse && g4 == 0) p.lse[o] = st.lse(ct);
                } else {
                    const int64_t o = (wg + u) * BM + r - r0;
#pragma unroll
                    for (int dt = 0; dt < D / 16; ++dt)
                        store4(parts.acc + o * D + 16 * dt + 4 * g4, st.acc[dt][ct]);
                    if (g4 == 0) {
                        parts.ml[o * 2] = st.mc[ct];
                        parts.ml[o * 2 + 1] = st.l[ct];
                    }
                }
            }
            __syncthreads();  // the tiles may be filled again
        }
        unit += places;
        at = unit;
        if (at >= end) return;
        if (++tile == rt.tiles) {
            tile = 0;
            if (++h == p.Hk) {
                h = 0;
                do {  // groups of nobody have no places
                    run = row_run<PREFIX>(d, ++i);
                } while (PREFIX && run.rows == 0);
                rt = RowTiles<BM>::template of<BK>(run);
            }
        }
    }
}

// Four neighbouring elements of a row per thread: the parts of the row, in order. BM: rows of
// the units of attn_rows_kernel.
template <typename DT, int D, int BM>
__global__ __launch_bounds__(256) void attn_join_kernel(DecodePlan d) {
    const AttnDecodeParams &p = d.p;
    const int64_t x = (int64_t)workgroup() * 256 + threadIdx.x;
    const int64_t o = x / (D / 4);  // sequence, token and query head
    if (o >= (int64_t)p.B * p.K * p.Hq) return;
    const int dd = (int)(x % (D / 4)) * 4;
    const int b = (int)(o / ((int64_t)p.K * p.Hq)), row = (int)(o - (int64_t)b * p.K * p.Hq);
    const int g = p.Hq / p.Hk, tok = row / p.Hq, hq = row - tok * p.Hq, h = hq / g;
    const int r = tok * g + hq - h * g;
    // the parts: n of them, `step` rows apart, from row `at`
    auto parts_of = [](const Parts &q, int64_t unit, int rows, int in, int64_t &at, int &n) {
        const int2 u = *reinterpret_cast<const int2 *>(q.units + unit * 2);
        at = (int64_t)u.x * rows + in;
        n = u.y;
    };
    int64_t own, pre = 0;
    int no, np = 0;
    if (d.few)
        parts_of(d.own, (int64_t)b * p.Hk + h, d.rows, r, own, no);
    else
        parts_of(d.own,
                 units_before<false, BM>(d, b, b) * p.Hk + h * ((d.rows + BM - 1) / BM) + r / BM,
                 BM, r % BM, own, no);
    if (no == 1 && !p.ptable) return;  // written by its workgroup
    if (p.ptable) {
        int lo = 0, hi = p.G;  // the last group that starts at or before b
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            (clamped(p.pgroups, mid, p.B) <= b ? lo : hi) = mid;
        }
        const int first = (int)clamped(p.pgroups, lo, p.B);
        const int last = (int)clamped(p.pgroups, lo + 1, p.B);
        if (b >= first && b < last) {  // malformed groups may leave a sequence out
            const int all = (last - first) * d.rows, in = (b - first) * d.rows + r;
            parts_of(d.pre,
                     units_before<true, BM>(d, lo, first) * p.Hk + h * ((all + BM - 1) / BM) +
                         in / BM,
                     BM, in % BM, pre, np);
        }
    }
    const int so = d.few ? d.rows : BM;
    // each of the row's lanes looks at one part's reference and sum, and hands them round (64
    // sequences behind 32,768 shared tokens: 13.2 us, 16 where every lane reads all of them)
    constexpr int L = D / 4;
    const int me = threadIdx.x & (L - 1);
    float m = -__builtin_inff();
    for (int s = me; s < np; s += L) m = fmaxf(m, d.pre.ml[(pre + (int64_t)s * BM) * 2]);
    for (int s = me; s < no; s += L) m = fmaxf(m, d.own.ml[(own + (int64_t)s * so) * 2]);
#pragma unroll
    for (int x = 1; x < L; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
    float l = 0.f;
    f32x4 a = zero4();
    auto add = [&](const Parts &q, int64_t at, int n, int step) {
        for (int s0 = 0; s0 < n; s0 += L) {
            float f = 0.f, lf = 0.f;
            if (s0 + me < n) {
                const float2 w =
                    *reinterpret_cast<const float2 *>(q.ml + (at + (int64_t)(s0 + me) * step) * 2);
                // a part that saw no key has sums of 0, or NaN
                f = w.x == -__builtin_inff() ? 1.f : exp2_fast(w.x - m);
                lf = w.y * f;
            }
            const int here = min(L, n - s0);
            const float *from = q.acc + (at + (int64_t)s0 * step) * D + dd;
            for (int s = 0; s < here; s += 8) {
                f32x4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = *reinterpret_cast<const f32x4 *>(
                        from + (int64_t)min(s + i, here - 1) * step * D);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (s + i < here) {
                        l += __shfl(lf, s + i, L);
                        a += v[i] * __shfl(f, s + i, L);
                    }
            }
        }
    };
    add(d.pre, pre, np, BM);
    add(d.own, own, no, so);
    store4(static_cast<DT *>(p.out) + o * D + dd, a * (l == 0.f ? 0.f : 1.f / l));
    if (p.lse && dd == 0) p.lse[o] = l == 0.f ? -__builtin_inff() : m * kLn2 + logf(l);
}

// Shapes of the kernels, as the launches and the workspace's size both need them.
template <typename DT, int D> struct Shape {
    static constexpr bool kWide = sizeof(DT) == 4;
    static constexpr int kCT = kWide ? 1 : 2;
    // fp32: products take so long that small tiles and two workgroups per CU pay (17 x 4 tokens
    // behind two prefixes, 16/8 heads of 128: 80 us, with 8 waves and 64 keys 98)
    static constexpr int kNW = !kWide && D == 256 ? 8 : 4;
    static constexpr int kBK = kWide ? 32 : 64;
    static constexpr int kBM = kNW * kCT * 16;
    static constexpr int kPerCu = KeyTiles<DT, D, kCT, kNW, kBK>::kLds > 80 * 1024 ? 1 : 2;
    static constexpr int kFewNW = kWide && D == 256 ? 2 : 4;
    static constexpr int kFewLds = kFewNW * 2 * kFewKeys * Rows<DT, D>::kPitch;
};

struct Layout {
    DecodePlan d;
    size_t acc[2], ml[2], units[2], bytes;  // of d.pre, d.own
};
constexpr size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <typename DT, int D> Layout layout(const AttnDecodeParams &p, int cus) {
    using S = Shape<DT, D>;
    Layout o{};
    DecodePlan &d = o.d;
    d.p = p;
    d.rows = p.K * (p.Hq / p.Hk);
    d.few = d.rows <= kFewRows;
    auto room = [&](int which, int64_t units, int32_t wgs, int64_t rows) {
        const int64_t slots = units + wgs;
        o.acc[which] = (size_t)slots * rows * D * 4;
        o.ml[which] = (size_t)slots * rows * 8;
        o.units[which] = (size_t)units * 8;
    };
    // workgroups for `units` units of at most `tiles` tiles: no more than the device holds
    auto wgs = [&](int64_t units, int64_t tiles, int least, int64_t most) {
        const int64_t n = (units * tiles + least - 1) / least;
        return (int32_t)(n < most ? n : most);
    };
    const int64_t keys = (int64_t)p.max_pages << p.page_shift;
    if (p.ptable) {
        const int64_t pkeys = (int64_t)p.max_ppages << p.page_shift;
        const int64_t units = ((int64_t)p.B * d.rows / S::kBM + p.G) * p.Hk;
        d.pre.wgs = wgs(units, pkeys / S::kBK + 1, kRowsTiles, (int64_t)S::kPerCu * cus);
        room(0, units, d.pre.wgs, S::kBM);
    }
    if (d.few) {
        const int64_t units = (int64_t)p.B * p.Hk, tiles = keys / kFewKeys + 1;
        if (tiles > kFewTiles)
            d.own.wgs = wgs(units, tiles, kFewTiles, (int64_t)cus * (160 * 1024 / (S::kFewLds + 1024)));
        if (d.own.wgs || p.ptable) room(1, units, d.own.wgs, d.rows);
    } else {
        const int64_t units = (int64_t)p.B * ((d.rows + S::kBM - 1) / S::kBM) * p.Hk;
        d.own.wgs = wgs(units, keys / S::kBK + 1, kRowsTiles, (int64_t)S::kPerCu * cus);
        room(1, units, d.own.wgs, S::kBM);
    }
    for (int i = 0; i < 2; ++i) o.bytes += up256(o.acc[i]) + up256(o.ml[i]) + up256(o.units[i]);
    return o;
}

template <typename DT, int D, bool PREFIX>
hipError_t launch_rows(const DecodePlan &d, hipStream_t stream) {
    using S = Shape<DT, D>;
    constexpr int kLds = KeyTiles<DT, D, S::kCT, S::kNW, S::kBK>::kLds;
    const auto kernel = attn_rows_kernel<DT, D, S::kCT, S::kNW, S::kBK, 2, PREFIX>;
    const hipError_t e = with_lds(kernel, kLds);
    if (e != hipSuccess) return e;
    const int64_t n = PREFIX ? d.pre.wgs : d.own.wgs;
    kernel<<<grid_of(n, 64 * S::kNW), 64 * S::kNW, kLds, stream>>>(d);
    return hipGetLastError();
}

template <typename DT, int D, int CT>
hipError_t launch_few(const DecodePlan &d, hipStream_t stream) {
    using S = Shape<DT, D>;
    const auto kernel = attn_few_kernel<DT, D, CT, S::kFewNW>;
    const hipError_t e = with_lds(kernel, S::kFewLds);
    if (e != hipSuccess) return e;
    const int64_t n = d.own.wgs ? d.own.wgs : (int64_t)d.p.B * d.p.Hk;
    kernel<<<grid_of(n, 64 * S::kFewNW), 64 * S::kFewNW, S::kFewLds, stream>>>(d);
    return hipGetLastError();
}

template <typename DT, int D>
hipError_t launch(const AttnDecodeParams &p, int cus, void *ws, hipStream_t stream) {
    Layout o = layout<DT, D>(p, cus);
    DecodePlan &d = o.d;
    unsigned char *at = static_cast<unsigned char *>(ws);
    for (int i = 0; i < 2; ++i) {
        Parts &q = i == 0 ? d.pre : d.own;
        if (!o.units[i]) continue;
        q.acc = reinterpret_cast<float *>(at);
        q.ml = reinterpret_cast<float *>(at += up256(o.acc[i]));
        q.units = reinterpret_cast<int32_t *>(at += up256(o.ml[i]));
        at += up256(o.units[i]);
    }
    hipError_t e = hipSuccess;
    if (p.ptable) e = launch_rows<DT, D, true>(d, stream);
    if (e != hipSuccess) return e;
    if (!d.few)
        e = launch_rows<DT, D, false>(d, stream);
    else
        e = d.rows <= 16 ? launch_few<DT, D, 1>(d, stream) : launch_few<DT, D, 2>(d, stream);
    if (e != hipSuccess || o.bytes == 0) return e;
    const int64_t wgs = ((int64_t)p.B * p.K * p.Hq * (D / 4) + 255) / 256;
    attn_join_kernel<DT, D, Shape<DT, D>::kBM><<<grid_of(wgs, 256), 256, 0, stream>>>(d);
    return hipGetLastError();
}

}  // namespace

#define GDN_ATTN_CASES(call)                                                   \
    if (dtype == 1)                                                            \
        return D == 64    ? call<__bf16, 64> GDN_ATTN_ARGS                     \
               : D == 128 ? call<__bf16, 128> GDN_ATTN_ARGS                    \
                          : call<__bf16, 256> GDN_ATTN_ARGS;                   \
    return D == 64    ? call<float, 64> GDN_ATTN_ARGS                          \
           : D == 128 ? call<float, 128> GDN_ATTN_ARGS                         \
                      : call<float, 256> GDN_ATTN_ARGS

size_t attn_decode_workspace_bytes(const AttnDecodeParams &p, int dtype, int D, int cus) {
#define GDN_ATTN_ARGS (p, cus).bytes
    GDN_ATTN_CASES(layout);
#undef GDN_ATTN_ARGS
}

hipError_t launch_attn_decode(const AttnDecodeParams &p, int dtype, int D, int cus, void *ws,
                              hipStream_t stream) {
#define GDN_ATTN_ARGS (p, cus, ws, stream)
    GDN_ATTN_CASES(launch);
#undef GDN_ATTN_ARGS
}

}  // namespace gdn
