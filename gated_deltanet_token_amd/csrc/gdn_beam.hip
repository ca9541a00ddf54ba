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
// The best W of a piece: every thread keeps its best (value, place); the W-th
// best of those is a bound that at least W elements reach and that at most W
// threads have anything above of, so the elements that reach it are few and
// fit a fixed buffer; they are ranked against each other. Keys hold the place
// too, so they all differ, and neither ties nor the order of the buffer's
// filling change the result.
#include "gdn_device.hpp"
#include "gdn_ops_launch.hpp"

namespace gdn {

namespace {

constexpr int kThreads = 256;
constexpr int kPiece = 8192;                 // logits per workgroup
constexpr int kPer = kPiece / kThreads;      // per thread
constexpr int kMaxW = 32;
constexpr float kLog2e = 0x1.715476p+0f;

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

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x = fmaxf(x, __shfl_xor(x, o));
    return x;
}
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
    return x;
}

struct PieceSum {
    float m, sum;  // sum of e^(l - m) over the piece; m NaN: a NaN or +inf was there
};

__host__ __device__ inline int64_t pieces_of(int64_t V) { return (V + kPiece - 1) / kPiece; }

// 8 logits from any element on: rows of an odd V start off 16 bytes, and a
// thread's share is counted from its row's start all the same, so that equal
// rows give equal sums bit by bit and their candidates tie.
template <typename DT> struct __attribute__((packed, aligned(sizeof(DT)))) Eight {
    DT v[8];
};

template <typename DT>
__global__ __launch_bounds__(kThreads) void beam_piece_kernel(const DT *logits, int64_t V,
                                                              int W, int npieces,
                                                              PieceSum *sums, uint64_t *best) {
    __shared__ uint64_t s_key[kThreads];
    __shared__ uint64_t s_list[kMaxW * kPer];
    __shared__ float s_red[2][4];
    __shared__ uint64_t s_bound;
    __shared__ int s_count;

    const int64_t row = blockIdx.x / npieces;
    const int piece = blockIdx.x - (int)(row * npieces);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const DT *from = logits + row * V + (int64_t)piece * kPiece;
    const uint32_t first = (uint32_t)piece * kPiece;  // the piece's first token
    const int here = (int)(V - first < kPiece ? V - first : kPiece);
    if (tid == 0) s_count = 0;

    // element e of vector j: the piece's (j * 256 + tid) * 8 + e
    float v[kPer / 8][8];
    float top = -__builtin_inff();
    bool bad = false;
#pragma unroll
    for (int j = 0; j < kPer / 8; ++j) {
        const int at = (j * kThreads + tid) * 8;
        if (at + 8 <= here) {
            const Eight<DT> q = *reinterpret_cast<const Eight<DT> *>(from + at);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = to_f32(q.v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[j][e] = at + e < here ? to_f32(from[at + e]) : -__builtin_inff();
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            bad |= !(v[j][e] < __builtin_inff());  // NaN or +inf: the row is dead
            if (v[j][e] != v[j][e]) v[j][e] = -__builtin_inff();
            top = fmaxf(top, v[j][e]);
        }
    }
    top = wave_max(top);
    const uint64_t anybad = __ballot(bad);
    if (lane == 0) s_red[0][wave] = anybad ? __builtin_nanf("") : top;
    __syncthreads();
    float m = -__builtin_inff();
    bool dead = false;
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) {
        dead |= s_red[0][i] != s_red[0][i];
        m = fmaxf(m, s_red[0][i]);
    }
    // l - m first: the terms that count are near 0 there, so that no rounding is
    // common to all of them, and the lowest finite values neither overflow nor
    // drop out of a row that holds nothing else
    float sum = 0.f;
    if (m > -__builtin_inff()) {
#pragma unroll
        for (int j = 0; j < kPer / 8; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sum += __builtin_amdgcn_exp2f((v[j][e] - m) * kLog2e);  // -inf: 0
            }
    }
    sum = wave_sum(sum);

    // the thread's best; places rise with j and e, so the first of equals stays
    float bv = 0.f;
    int bp = -1;
#pragma unroll
    for (int j = 0; j < kPer / 8; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int at = (j * kThreads + tid) * 8 + e;
            if (at < here && (bp < 0 || v[j][e] > bv)) {
                bv = v[j][e];
                bp = at;
            }
        }
    // a thread without elements: a key below all real ones, its own
    const uint64_t mine = bp < 0 ? (uint64_t)tid : key_of(bv, first + bp);
    s_key[tid] = mine;
    if (lane == 0) s_red[1][wave] = sum;
    __syncthreads();
    int above = 0;
    for (int i = 0; i < kThreads; ++i) above += s_key[i] > mine;
    if (above == W - 1) s_bound = mine;
    __syncthreads();
    const uint64_t bound = s_bound;
    if (mine >= bound && bp >= 0) {
#pragma unroll
        for (int j = 0; j < kPer / 8; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = (j * kThreads + tid) * 8 + e;
                if (at < here) {
                    const uint64_t k = key_of(v[j][e], first + at);
                    if (k >= bound) s_list[atomicAdd(&s_count, 1)] = k;
                }
            }
    }
    __syncthreads();
    const int count = s_count;
    uint64_t *out = best + (int64_t)blockIdx.x * W;
    for (int i = tid; i < count; i += kThreads) {
        const uint64_t k = s_list[i];
        int rank = 0;
        for (int q = 0; q < count; ++q) rank += s_list[q] > k;
        if (rank < W) out[rank] = k;
    }
    if (tid >= count && tid < W) out[tid] = 0;  // fewer elements than W
    if (tid == 0) {
        float all = 0.f;
        for (int i = 0; i < kThreads / 64; ++i) all += s_red[1][i];
        sums[blockIdx.x] = PieceSum{dead ? __builtin_nanf("") : m, all};
    }
}

struct Cand {
    double score;
    int64_t place;  // w V + v; -1: none
};
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

// One workgroup per batch item: the logsumexp of its beams, then W rounds that
// each take the best candidate behind the last one taken.
__global__ __launch_bounds__(kThreads) void beam_join_kernel(BeamParams p, int npieces,
                                                             const PieceSum *sums,
                                                             const uint64_t *best) {
    __shared__ double s_logsum[kMaxW];  // log of the sum of e^(l - m)
    __shared__ float s_m[kMaxW];
    __shared__ float s_score[kMaxW];
    __shared__ int s_done[kMaxW], s_live[kMaxW];
    __shared__ Cand s_pick[kThreads / 64];

    const int b = blockIdx.x, W = p.W, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t V = p.V;
    for (int w = wave; w < W; w += kThreads / 64) {
        const int64_t row = (int64_t)b * W + w;
        const PieceSum *ps = sums + row * npieces;
        float m = -__builtin_inff();
        bool nan = false;
        for (int i = lane; i < npieces; i += 64) {
            nan |= ps[i].m != ps[i].m;
            m = fmaxf(m, ps[i].m);
        }
        m = wave_max(m);
        nan = __ballot(nan) != 0;
        double sum = 0.0;
        if (m > -__builtin_inff())
            for (int i = lane; i < npieces; i += 64)
                if (ps[i].m > -__builtin_inff())
                    sum += (double)ps[i].sum * exp((double)ps[i].m - (double)m);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
        if (lane == 0) {
            const float s = p.scores[row];
            const bool done = p.finished && p.finished[row];
            const bool live = fabsf(s) < __builtin_inff() &&
                              (done || (!nan && m > -__builtin_inff()));
            s_m[w] = m;
            s_logsum[w] = live && !done ? log(sum) : 0.0;
            s_score[w] = s;
            s_done[w] = done;
            s_live[w] = live;
        }
    }
    __syncthreads();

    const int per = npieces * W;  // candidates of a beam
    Cand last{__builtin_inf(), -1};
    bool any = false;
    for (int k = 0; k < W; ++k) {
        Cand c{0.0, -1};
        for (int i = tid; i < W * per; i += kThreads) {
            const int w = i / per, q = i - w * per;
            const int64_t row = (int64_t)b * W + w;
            Cand d{-__builtin_inf(), -1};
            if (!s_live[w]) {  // its tokens in order at -inf
                if (q < W && q < V) d.place = w * V + q;
            } else if (s_done[w]) {  // itself, then its other tokens in order at -inf
                const int64_t v = q == 0 ? p.eos : (q - 1 < p.eos ? q - 1 : q);
                if (q == 0) d.score = s_score[w];
                if (q < W && v < V) d.place = w * V + v;
            } else {
                const uint64_t key = best[row * per + q];
                if (key >> 32) {
                    const float l = unordered((uint32_t)(key >> 32));
                    d.score = (double)s_score[w] + (((double)l - (double)s_m[w]) - s_logsum[w]);
                    d.place = w * V + (uint32_t)~(uint32_t)key;
                }
            }
            if (d.place >= 0 && (!any || before(last, d))) c = better(c, d);
        }
        c = wave_best(c);
        if (lane == 0) s_pick[wave] = c;
        __syncthreads();
        c = s_pick[0];
#pragma unroll
        for (int i = 1; i < kThreads / 64; ++i) c = better(c, s_pick[i]);
        last = c;
        any = true;
        if (tid == 0) {
            const int w = (int)(c.place / V);
            const int32_t v = (int32_t)(c.place - w * V);
            const int64_t to = (int64_t)b * W + k;
            p.new_scores[to] = (float)c.score;
            p.tokens[to] = v;
            p.parents[to] = w;
            if (p.new_finished) p.new_finished[to] = s_done[w] || v == p.eos;
            if (p.src_slots) p.src_slots[to] = p.slots[(int64_t)b * W + w];
        }
        __syncthreads();
    }
}

// 16 KiB of one row per workgroup.
__global__ __launch_bounds__(256) void gather_kernel(const u32x4 *src, int64_t num_src,
                                                     const int32_t *index, u32x4 *dst,
                                                     int64_t row_vecs, int parts) {
    const int64_t row = blockIdx.x / parts;
    const int part = blockIdx.x - (int)(row * parts);
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

size_t keys_offset(int64_t pieces) { return ((size_t)pieces * sizeof(PieceSum) + 255) / 256 * 256; }

}  // namespace

size_t beam_workspace_bytes(int32_t B, int32_t W, int64_t V, int) {
    const int64_t pieces = (int64_t)B * W * pieces_of(V);
    return keys_offset(pieces) + (size_t)pieces * W * 8;
}

hipError_t launch_beam(const BeamParams &p, int dtype, void *ws, hipStream_t stream) {
    const int64_t np = pieces_of(p.V), pieces = (int64_t)p.B * p.W * np;
    PieceSum *sums = static_cast<PieceSum *>(ws);
    uint64_t *best = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) + keys_offset(pieces));
    if (dtype == 1)
        hipLaunchKernelGGL(beam_piece_kernel<__bf16>, dim3((unsigned)pieces), dim3(kThreads), 0,
                           stream, static_cast<const __bf16 *>(p.logits), p.V, p.W, (int)np, sums,
                           best);
    else
        hipLaunchKernelGGL(beam_piece_kernel<float>, dim3((unsigned)pieces), dim3(kThreads), 0,
                           stream, static_cast<const float *>(p.logits), p.V, p.W, (int)np, sums,
                           best);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(beam_join_kernel, dim3((unsigned)p.B), dim3(kThreads), 0, stream, p,
                       (int)np, sums, best);
    return hipGetLastError();
}

hipError_t launch_gather(const void *src, int64_t num_src, const int32_t *index, void *dst,
                         int64_t rows, int64_t row_bytes, hipStream_t stream) {
    if (rows == 0 || row_bytes == 0) return hipSuccess;
    const int parts = (int)((row_bytes + 16383) / 16384);
    hipLaunchKernelGGL(gather_kernel, dim3((unsigned)(rows * parts)), dim3(256), 0, stream,
                       static_cast<const u32x4 *>(src), num_src, index, static_cast<u32x4 *>(dst),
                       row_bytes / 16, parts);
    return hipGetLastError();
}

}  // namespace gdn
