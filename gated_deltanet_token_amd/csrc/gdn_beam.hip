// gdn_beam.hip -- beam search's selection over beams and vocabulary, and the
// reordering of states by it (gfx950).
//
// Candidate (w, v) of a batch item scores s_w + l_wv - lse_w, lse_w the
// logsumexp of beam w's logits; the W best over all w, v are wanted, best
// first, ties to the lowest w V + v. Within a beam the order of candidates is
// that of its logits, so one pass over the logits gives, per piece of a row,
// the logsumexp's parts and the W best logits (exactly, as values and places),
// and a second, small kernel joins the pieces and orders the few candidates
// left by their score in fp64. The logits are read once: bound by HBM for
// large batches, by latency for one sequence.
//
// The best W of a piece: every lane keeps its best value; the W-th best of a
// wave's 64 (found bit by bit with ballots), and the largest of those over the
// waves, is a bound that at least W elements reach and few others do. They are
// collected and ranked against each other by value and place, so that neither
// ties nor the order of the collection change the result. Where too many reach
// the bound (rows of equal values, or of hardly anything but -inf), and in the
// join where the candidates are more than its threads hold, W rounds that each
// find the next best take its place.
#include "gdn_device.hpp"
#include "gdn_ops_launch.hpp"

namespace gdn {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kMaxW = 32;
constexpr int kList = 512;  // collected elements, at the most
constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kFusedMax = 0x1p20f;  // largest |maximum| of a piece that is summed in one pass

// A value's bits in an order of unsigned integers, -0 as +0.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __builtin_bit_cast(float, o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
// Larger value first, then lower place. Real keys are above 2^32: those
// values that order as 0 do not occur (they are NaN).
__device__ __forceinline__ uint64_t key_of(float x, uint32_t place) {
    return ((uint64_t)ordered(x) << 32) | (uint32_t)~place;
}

// Over the wave, by DPP within rows of 16 lanes and scalar reads of the rows.
__device__ __forceinline__ float lane_value(float x, int lane) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}
__device__ __forceinline__ float wave_max(float x) {
    x = fmaxf(x, GDN_DPP(x, 0xB1));
    x = fmaxf(x, GDN_DPP(x, 0x4E));
    x = fmaxf(x, GDN_DPP(x, 0x141));
    x = fmaxf(x, GDN_DPP(x, 0x140));
    return fmaxf(fmaxf(lane_value(x, 0), lane_value(x, 16)),
                 fmaxf(lane_value(x, 32), lane_value(x, 48)));
}
__device__ __forceinline__ float wave_sum(float x) {
    x = row16_sum(x);
    return (lane_value(x, 0) + lane_value(x, 16)) + (lane_value(x, 32) + lane_value(x, 48));
}

struct PieceSum {
    float m, sum;  // sum of e^(l - m) over the piece; m NaN: a NaN or +inf was there
};

// 8 logits from any element on: rows of an odd V start off 16 bytes, and a
// thread's share is counted from its row's start all the same, so that equal
// rows give equal sums bit by bit and their candidates tie.
template <typename DT> struct __attribute__((packed, aligned(sizeof(DT)))) Eight {
    uint32_t w[2 * sizeof(DT)];
    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (sizeof(DT) == 4) return __builtin_bit_cast(float, w[e]);
        return __builtin_bit_cast(float, e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    }
};

// The largest o such that at least `want` of the wave's lanes hold x >= o (0 if
// there is none), looked for from bit 31 down to bit `low`: bits below stay 0.
__device__ __forceinline__ uint32_t wave_bound(uint32_t x, int want, int low) {
    uint32_t o = 0;
    for (int bit = 31; bit >= low; --bit) {
        const uint32_t c = o | (1u << bit);
        if (__popcll(__ballot(x >= c)) >= want) o = c;
    }
    return o;
}

// Logits per workgroup: VECS times 8 per thread. Bound by vector instructions:
// 32 x 8 x 131,072 bf16 18 us, where its 67 MB would take 8 to 13. A wave of 32
// logits per lane has 389, 12 per logit, and its exponentials go at a quarter of
// the rate: together they fill 13 us of the SIMDs. Eight waves per SIMD cover the
// loads and the steps of a wave; the rounds read the logits again so that they do
// not cost the registers for that.
template <typename DT, int VECS>
__global__ __launch_bounds__(kThreads, 8) void beam_piece_kernel(const DT *logits, int64_t V, int W,
                                                                 int npieces, uint32_t total,
                                                                 PieceSum *sums, uint64_t *best) {
    constexpr int kPiece = VECS * 8 * kThreads;
    __shared__ uint64_t s_list[kList];
    __shared__ float s_top[kWaves], s_sum[kWaves];
    __shared__ uint32_t s_bound[kWaves];
    __shared__ int s_count;

    const uint32_t wg = workgroup();
    if (wg >= total) return;
    const int64_t row = wg / npieces;
    const int piece = wg - (int)(row * npieces);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const DT *from = logits + row * V + (int64_t)piece * kPiece;
    const uint32_t first = (uint32_t)piece * kPiece;  // the piece's first token
    const int here = (int)(V - first < kPiece ? V - first : kPiece);
    if (tid == 0) s_count = 0;

    // element e of vector j: the piece's (j * 256 + tid) * 8 + e
    float v[VECS][8], vtop[VECS];
    float top = -__builtin_inff();
    if (here == kPiece) {  // all loads before the first use
        Eight<DT> q[VECS];
#pragma unroll
        for (int j = 0; j < VECS; ++j)
            q[j] = *reinterpret_cast<const Eight<DT> *>(from + (j * kThreads + tid) * 8);
#pragma unroll
        for (int j = 0; j < VECS; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = q[j][e];
    } else {
#pragma unroll
        for (int j = 0; j < VECS; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = (j * kThreads + tid) * 8 + e;
                const float x = to_f32(from[at < here ? at : here - 1]);
                v[j][e] = at < here ? x : -__builtin_inff();
            }
    }
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
        vtop[j] = -__builtin_inff();  // a NaN is passed over here and found in the sum
#pragma unroll
        for (int e = 0; e < 8; ++e) vtop[j] = fmaxf(vtop[j], v[j][e]);
        top = fmaxf(top, vtop[j]);
    }
    // bf16 values differ in their upper 16 bits only
    const uint32_t wb = wave_bound(ordered(top), W, sizeof(DT) == 2 ? 16 : 0);
    const float wt = wave_max(top);
    if (lane == 0) {
        s_top[wave] = wt;
        s_bound[wave] = wb;
    }
    __syncthreads();
    float m = s_top[0];
    uint32_t ob = s_bound[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) {
        m = fmaxf(m, s_top[i]);
        ob = max(ob, s_bound[i]);
    }
    uint64_t *out = best + (int64_t)wg * W;
    const bool some = m > -__builtin_inff();
    // The sum of e^(l - m) as 2^(l log2e - c), c the rounded m log2e: one fused
    // multiply-add per exponent. The largest exponent is then what c is off, common
    // to all terms and taken out at the end; below kFusedMax that is at most 2^-4.
    // (It grows with m, and past 2^31 the sum would leave fp32's range.) Terms far
    // below the largest are 0. A NaN makes the sum NaN. Rows of a larger maximum, a
    // mask's fill over a whole piece above all, or of nothing but -inf, are summed
    // from memory by l - m, which is exact where it counts and overflows only to
    // -inf; a NaN or +inf there makes the sum NaN.
    float sum = 0.f;
    if (fabsf(m) <= kFusedMax) {
        const float c = m * kLog2e;
#pragma unroll
        for (int j = 0; j < VECS; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum += __builtin_amdgcn_exp2f(fmaf(v[j][e], kLog2e, -c));
        sum *= __builtin_amdgcn_exp2f(-fmaf(m, kLog2e, -c));
    } else {
        for (int i = tid; i < here; i += kThreads) {
            const float l = to_f32(from[i]);
            sum += some ? __builtin_amdgcn_exp2f((l - m) * kLog2e) : (l != l ? l : 0.f);
        }
    }
    sum = wave_sum(sum);
    if (lane == 0) s_sum[wave] = sum;

    // A bf16 bound has the lower half of its bits clear, which is the lowest
    // of the (negative) or the only (positive) pattern with that upper half.
    const float bound = unordered(ob);
    const bool picky = some && ob > ordered(-__builtin_inff());
    const bool few = here <= kList;  // all of them fit the list
    if (picky && top >= bound) {
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            if (!(vtop[j] >= bound)) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (v[j][e] >= bound) {  // places past the end are -inf
                    const int i = atomicAdd(&s_count, 1);
                    if (i < kList)
                        s_list[i] = key_of(v[j][e], first + (j * kThreads + tid) * 8 + e);
                }
        }
    }
    if (!picky && few)
        for (int i = tid; i < here; i += kThreads) {
            const float l = to_f32(from[i]);
            if (l == l) s_list[atomicAdd(&s_count, 1)] = key_of(l, first + i);
        }
    __syncthreads();
    if (tid == 0) {
        float all = s_sum[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) all += s_sum[i];
        sums[wg] = PieceSum{all != all ? all : m, all};
    }
    const int count = s_count;
    if ((picky || few) && count <= kList) {
        for (int i = tid; i < count; i += kThreads) {
            const uint64_t k = s_list[i];
            int rank = 0;
            for (int q = 0; q < count; ++q) rank += s_list[q] > k;
            if (rank < W) out[rank] = k;
        }
        if (tid >= count && tid < W) out[tid] = 0;
    } else if (!some) {
        if (tid < W) out[tid] = tid < here ? key_of(-__builtin_inff(), first + tid) : 0;
    } else {  // W rounds, each the best key below the last one; the logits from memory again
        uint64_t last = ~(uint64_t)0;
        for (int k = 0; k < W; ++k) {
            uint64_t c = 0;
            for (int i = tid; i < here; i += kThreads) {
                const float l = to_f32(from[i]);
                const uint64_t x = key_of(l, first + i);
                if (l == l && x < last && x > c) c = x;
            }
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const uint64_t x = __shfl_xor(c, o);
                c = x > c ? x : c;
            }
            __syncthreads();  // the list and the round in front are read
            if (lane == 0) s_list[wave] = c;
            __syncthreads();
            c = s_list[0];
#pragma unroll
            for (int i = 1; i < kWaves; ++i) c = s_list[i] > c ? s_list[i] : c;
            if (tid == 0) out[k] = c;  // 0: none left
            last = c;
        }
    }
}

struct Cand {
    double score;
    int64_t place;  // w 2^32 + v, in the order of w V + v; -1: none
};
__device__ __forceinline__ int64_t place_of(int w, int64_t v) { return (int64_t)w << 32 | v; }
__device__ __forceinline__ bool before(const Cand &a, const Cand &b) {
    if (b.place < 0) return a.place >= 0;
    if (a.place < 0) return false;
    return a.score > b.score || (a.score == b.score && a.place < b.place);
}
__device__ __forceinline__ Cand better(const Cand &a, const Cand &b) { return before(b, a) ? b : a; }

__device__ __forceinline__ Cand wave_best(Cand c) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        Cand d;
        d.score = __shfl_xor(c.score, o);
        d.place = __shfl_xor(c.place, o);
        c = better(c, d);
    }
    return c;
}

// What a beam offers, by the join kernel's shared arrays.
struct BeamRow {
    double logsum;  // log of the sum of e^(l - m)
    float m, score;
    int done, live;
};

// Candidate q of beam w (of npieces * W): a piece's key, or what a beam that
// has ended or is dead offers in its place.
__device__ __forceinline__ Cand candidate(const BeamRow &r, int w, int q, int W, int64_t V,
                                          int32_t eos, uint64_t key) {
    Cand d{-__builtin_inf(), -1};
    if (!r.live) {  // its tokens in order at -inf
        if (q < W && q < V) d.place = place_of(w, q);
    } else if (r.done) {  // itself, then its other tokens in order at -inf
        const int64_t v = q == 0 ? eos : (q - 1 < eos ? q - 1 : q);
        if (q == 0) d.score = r.score;
        if (q < W && v < V) d.place = place_of(w, v);
    } else if (key >> 32) {
        const float l = unordered((uint32_t)(key >> 32));
        d.score = (double)r.score + (((double)l - (double)r.m) - r.logsum);
        d.place = place_of(w, (uint32_t)~(uint32_t)key);
    }
    return d;
}

// A score in 32 ordered bits, rounded down: a >= b keeps its order or ties.
// 0 for no candidate.
__device__ __forceinline__ uint32_t score_bits(const Cand &c) {
    return c.place < 0 ? 0u : ordered(__double2float_rd(c.score));
}

// One workgroup per batch item: the logsumexp of its beams, then the W best of
// the pieces' candidates, found as in a piece (a bound from the scores rounded
// down to 32 bits, then a ranking in fp64).
// A thread holds up to HELD candidates. A chain of latencies: 5 us for one item of
// 4 beams and 16 pieces, 9 for 32 items of 8 beams and 16 pieces. Where W^2 pieces
// are more than 8,192 all is done by rounds over them, by the one workgroup of the
// item. One item: 9 beams from 206,849 to 229,376 tokens, 12 from 114,689 to
// 172,032, 16 from 65,537 to 122,880 and from 262,145 on, 32 nearly always from
// 16,385 on (pieces are 8,192 tokens long where that gives 256 workgroups, else
// 2,048). A call takes 80 us for W = 9 and 220,000 tokens, where W = 8 takes 24 to
// 29; 165 for 16 and 100,352; 390 for 32 and 32,000; 447 for 32 and 151,936.
template <int THREADS, int HELD>
__global__ __launch_bounds__(THREADS) void beam_join_kernel(BeamParams p, int npieces,
                                                            const PieceSum *sums,
                                                            const uint64_t *best) {
    constexpr int kWaves = THREADS / 64;
    __shared__ BeamRow s_row[kMaxW];
    __shared__ int32_t s_slot[kMaxW];
    __shared__ Cand s_list[kList];
    __shared__ uint32_t s_bound[kWaves];
    __shared__ int s_count;

    if (workgroup() >= (uint32_t)p.B) return;
    const int b = workgroup(), W = p.W, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t V = p.V;
    const int per = npieces * W, n = W * per;  // candidates of a beam, and all
    const uint64_t *keys = best + (int64_t)b * n;
    const bool held = n <= HELD * THREADS;
    uint64_t key[HELD];
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
        const int i = j * THREADS + tid;
        key[j] = held && i < n ? keys[i] : 0;
    }
    if (tid == 0) s_count = 0;
    for (int w = wave; w < W; w += kWaves) {
        const int64_t row = (int64_t)b * W + w;
        const PieceSum *ps = sums + row * npieces;
        const float s = p.scores[row];
        const bool done = p.finished && p.finished[row];
        if (p.src_slots && lane == 0) s_slot[w] = p.slots[row];
        PieceSum own{-__builtin_inff(), 0.f};  // the lane's first piece, and often its only one
        if (lane < npieces) own = ps[lane];
        float m = own.m;
        bool nan = own.m != own.m;
        for (int i = lane + 64; i < npieces; i += 64) {
            nan |= ps[i].m != ps[i].m;
            m = fmaxf(m, ps[i].m);
        }
        m = wave_max(m);
        nan = __ballot(nan) != 0;
        double sum = 0.0;
        if (m > -__builtin_inff()) {
            if (own.m > -__builtin_inff()) sum = (double)own.sum * exp((double)own.m - (double)m);
            for (int i = lane + 64; i < npieces; i += 64)
                if (ps[i].m > -__builtin_inff())
                    sum += (double)ps[i].sum * exp((double)ps[i].m - (double)m);
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
        if (lane == 0) {
            const bool live = fabsf(s) < __builtin_inff() &&
                              (done || (!nan && m > -__builtin_inff()));
            s_row[w] = BeamRow{live && !done ? log(sum) : 0.0, m, s, done, live};
        }
    }
    __syncthreads();

    const auto write = [&](int k, const Cand &c) {
        const int w = (int)(c.place >> 32);
        const int32_t v = (int32_t)c.place;
        const int64_t to = (int64_t)b * W + k;
        p.new_scores[to] = (float)c.score;
        p.tokens[to] = v;
        p.parents[to] = w;
        if (p.new_finished) p.new_finished[to] = s_row[w].done || v == p.eos;
        if (p.src_slots) p.src_slots[to] = s_slot[w];
    };

    if (held) {
        Cand c[HELD];
        uint32_t bits[HELD], top = 0;
#pragma unroll
        for (int j = 0; j < HELD; ++j) {
            const int i = j * THREADS + tid;
            c[j].place = -1;
            if (i < n) {
                const int w = i / per;
                c[j] = candidate(s_row[w], w, i - w * per, W, V, p.eos, key[j]);
            }
            bits[j] = score_bits(c[j]);
            top = max(top, bits[j]);
        }
        const uint32_t wb = wave_bound(top, W, 0);
        if (lane == 0) s_bound[wave] = wb;
        __syncthreads();
        uint32_t bound = s_bound[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) bound = max(bound, s_bound[i]);
#pragma unroll
        for (int j = 0; j < HELD; ++j)
            if (c[j].place >= 0 && bits[j] >= bound) {
                const int i = atomicAdd(&s_count, 1);
                if (i < kList) s_list[i] = c[j];
            }
        __syncthreads();
        const int count = s_count;
        if (count <= kList) {  // at least W: every beam offers min(W, V)
            for (int i = tid; i < count; i += THREADS) {
                const Cand x = s_list[i];
                int rank = 0;
                for (int q = 0; q < count; ++q) rank += before(s_list[q], x);
                if (rank < W) write(rank, x);
            }
            return;
        }
    }

    // W rounds, each the best candidate behind the last one taken
    Cand last{0.0, -1};
    for (int k = 0; k < W; ++k) {
        Cand c{0.0, -1};
        for (int i = tid; i < n; i += THREADS) {
            const int w = i / per;
            const Cand d = candidate(s_row[w], w, i - w * per, W, V, p.eos, keys[i]);
            if (d.place >= 0 && (k == 0 || before(last, d))) c = better(c, d);
        }
        c = wave_best(c);
        __syncthreads();  // the round in front is read
        if (lane == 0) s_list[wave] = c;
        __syncthreads();
        c = s_list[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) c = better(c, s_list[i]);
        last = c;
        if (tid == 0) write(k, c);
    }
}

// 16 KiB of one row per workgroup: a copy, 32 states of 3 MiB in 22.5 us (8.9 TB/s
// read and written, parents that several beams share coming from cache). A short
// row leaves most of its workgroup idle: 65,536 rows of 256 bytes 31 us (1.1 TB/s).
__global__ __launch_bounds__(256) void gather_kernel(const u32x4 *src, int64_t num_src,
                                                     const int32_t *index, u32x4 *dst,
                                                     int64_t row_vecs, int parts, uint32_t total) {
    const uint32_t wg = workgroup();
    if (wg >= total) return;
    const int64_t row = wg / parts;
    const int part = wg - (int)(row * parts);
    const int64_t from = index[row];
    const int64_t v0 = (int64_t)part * 1024 + threadIdx.x;
    u32x4 *to = dst + row * row_vecs;
    if (from >= 0 && from < num_src) {
        const u32x4 *s = src + from * row_vecs;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (v0 + 256 * i < row_vecs)
                __builtin_nontemporal_store(s[v0 + 256 * i], to + v0 + 256 * i);
    } else {
        const uint32_t f = from < 0 ? 0u : 0xFFFFFFFFu;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (v0 + 256 * i < row_vecs) to[v0 + 256 * i] = u32x4{f, f, f, f};
    }
}

// 8 logits per thread where a piece of 32 per thread would leave CUs without a
// workgroup, else 32.
int piece_vecs(int64_t rows, int64_t V) {
    return rows * ((V + 8191) / 8192) < 256 ? 1 : 4;
}

int64_t pieces_of(int64_t rows, int64_t V) {
    const int64_t piece = piece_vecs(rows, V) * 8 * kThreads;
    return (V + piece - 1) / piece;
}

size_t keys_offset(int64_t pieces) { return ((size_t)pieces * sizeof(PieceSum) + 255) / 256 * 256; }

}  // namespace

size_t beam_workspace_bytes(int32_t B, int32_t W, int64_t V, int) {
    const int64_t rows = (int64_t)B * W, pieces = rows * pieces_of(rows, V);
    return keys_offset(pieces) + (size_t)pieces * W * 8;
}

hipError_t launch_beam(const BeamParams &p, int dtype, void *ws, hipStream_t stream) {
    const int64_t rows = (int64_t)p.B * p.W, np = pieces_of(rows, p.V), pieces = rows * np;
    PieceSum *sums = static_cast<PieceSum *>(ws);
    uint64_t *best = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) + keys_offset(pieces));
    const bool few = piece_vecs(rows, p.V) == 1;
#define GDN_BEAM_LAUNCH(DT, VECS)                                                              \
    hipLaunchKernelGGL((beam_piece_kernel<DT, VECS>), grid_of(pieces, kThreads), dim3(kThreads), 0, \
                       stream, static_cast<const DT *>(p.logits), p.V, p.W, (int)np,              \
                       (uint32_t)pieces, sums, best)
    if (dtype == 1) {
        if (few)
            GDN_BEAM_LAUNCH(__bf16, 1);
        else
            GDN_BEAM_LAUNCH(__bf16, 4);
    } else {
        if (few)
            GDN_BEAM_LAUNCH(float, 1);
        else
            GDN_BEAM_LAUNCH(float, 4);
    }
#undef GDN_BEAM_LAUNCH
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // a wave per beam where that is enough of them: their sums take the longest
    if (p.W > 4 && p.W <= 8 && np * p.W * p.W <= 2048)
        hipLaunchKernelGGL((beam_join_kernel<512, 4>), grid_of(p.B, 512), dim3(512), 0, stream,
                           p, (int)np, sums, best);
    else if (np * p.W * p.W <= 1024)
        hipLaunchKernelGGL((beam_join_kernel<256, 4>), grid_of(p.B, 256), dim3(256), 0, stream,
                           p, (int)np, sums, best);
    else
        hipLaunchKernelGGL((beam_join_kernel<1024, 8>), grid_of(p.B, 1024), dim3(1024), 0,
                           stream, p, (int)np, sums, best);
    return hipGetLastError();
}

hipError_t launch_gather(const void *src, int64_t num_src, const int32_t *index, void *dst,
                         int64_t rows, int64_t row_bytes, hipStream_t stream) {
    if (rows == 0 || row_bytes == 0) return hipSuccess;
    const int parts = (int)((row_bytes + 16383) / 16384);
    hipLaunchKernelGGL(gather_kernel, grid_of(rows * parts, 256), dim3(256), 0, stream,
                       static_cast<const u32x4 *>(src), num_src, index, static_cast<u32x4 *>(dst),
                       row_bytes / 16, parts, (uint32_t)(rows * parts));
    return hipGetLastError();
}

}  // namespace gdn
