// gdn_scan.hip -- the gated linear recurrence (gfx950): h_t = alpha_t h_{t-1}
// + beta_t x_t per channel, forward, backward and single tokens.
//
// Each element is read once and written once for a handful of operations, so
// the bound is HBM traffic: 4 elements per token and channel forward (3 with
// tied gates), 7 backward (5).
//
// The recurrence is affine, so a run of tokens is summed up by two numbers per
// channel: with A the product of its decays and H its result from a zero
// state, it maps h to A h + H. A workgroup takes tiles of 128 tokens; every
// thread sums up its few tokens, one thread per channel chains the groups of
// threads, and each thread then walks its tokens from its true state. The
// backward pass is the same chain from the end: with c_t = alpha_t (dout_t +
// c_{t+1}) the gradient that reaches h_{t-1}, a run maps c to A c + K.
#include <type_traits>

#include "gdn_scan.hpp"

namespace gdn {

namespace {

// The tile that a workgroup of a SPLIT launch takes: its sequence (-1: no tile),
// column block and tile, which may lie past the sequence's last one.
struct ScanTile {
    int n, cb;
    int64_t slot, tile;
};
template <bool BACK>
__device__ __forceinline__ ScanTile take_tile(const ScanParams &p, const ScanSplit &sp, int ncb,
                                              int *s_take) {
    const int chain = sp.runs.chain(workgroup() % sp.runs.grid);
    if (chain < 0) return ScanTile{-1, 0, 0, 0};
    if (threadIdx.x == 0) {
        s_take[0] = (int)__hip_atomic_fetch_add(sp.ticket + chain, 1u, __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT);
        s_take[1] = 0;
    }
    __syncthreads();
    // uniform, and known to be
    const int64_t k = counted_tile(__builtin_amdgcn_readfirstlane(s_take[0]), sp.per_chain, BACK);
    if (k < 0) return ScanTile{-1, 0, 0, 0};
    ScanTile t;
    if (p.cu) {
        t.cb = chain;
        t.slot = k;
        t.n = scan_slot_sequence(p, k, s_take + 1);
        t.tile = k - scan_first_slot(p, t.n);
    } else {
        t.n = chain / ncb;
        t.cb = chain - t.n * ncb;
        t.tile = k;
        t.slot = k * p.N + t.n;
    }
    return t;
}

// SPLIT > 0: one tile per workgroup (gdn_scan.hpp). Else one workgroup per
// (sequence, column block), its tiles in order: enough where that alone fills
// the device, and without a workspace.
//
// Bound by HBM: 65,536 x 6,144 bf16 610 us (5.3 TB/s, the reads and writes
// counted at 1.01 times the tensors), 20,011 x 2,048 fp32 packed 130 us. Two
// workgroups of 512 threads per CU (4 waves per SIMD) hold 196 KiB of loads in
// flight; those of 1,024 threads (pairs and single columns) share a CU up to 64
// registers only, which the bf16 pairs pass with SPLIT 4 and 0 (79 and 94).
// Gates are formed once and kept with the products beta x as fp32.
template <typename DT, int VEC, bool TIED, bool LOGITS, int SPLIT>
__global__ __launch_bounds__((ScanShape<DT, VEC>::kThreads)) void scan_forward_kernel(
    ScanParams p, int ncb, ScanSplit sp) {
    using Sh = ScanShape<DT, VEC>;
    constexpr int G = Sh::kGroups, C = Sh::kCols, R = Sh::kPer;
    __shared__ float s_a[G][C], s_h[G][C];

    __shared__ int s_take[3];
    const int pair = SPLIT > 0 ? 0 : sp.runs.chain(workgroup());
    ScanTile mine{pair / ncb, pair % ncb, 0, 0};
    if constexpr (SPLIT > 0) mine = take_tile<false>(p, sp, ncb, s_take);
    if (SPLIT > 0 ? mine.n < 0 : pair < 0) return;
    const int n = mine.n, cb = mine.cb;
    const int tid = threadIdx.x, g = tid / Sh::kLanes, l = tid % Sh::kLanes;
    const int D = p.D, c0 = cb * C + l * VEC;
    const bool on = c0 < D;
    const int col = on ? c0 : 0;  // lanes past the last column read the first, and write nothing
    const int ch = cb * C + tid;  // the channel that this thread chains
    const bool chain = tid < C && ch < D;
    int64_t base, len;
    scan_bounds(p, n, base, len);
    float carry = 0.f;  // the state in front of the tile, once it is known
    if (chain && p.h0 && mine.tile == 0) carry = p.h0[(int64_t)n * D + ch];
    if (mine.tile < 0 || mine.tile * Sh::kRows >= len) {  // (below 0: malformed offsets)
        if (mine.tile == 0 && chain && p.hT) p.hT[(int64_t)n * D + ch] = carry;
        if constexpr (SPLIT > 0)
            if (tid < C) publish_state(sp, mine.slot, ch, 0.f);
        return;
    }
    const int64_t prow = p.prefix_out ? scan_prefix_row(p, n, base) : 0;

    int64_t t0 = mine.tile * Sh::kRows;
    do {
        const int left = (int)(len - t0 < Sh::kRows ? len - t0 : Sh::kRows);  // tokens here
        const int64_t tile = (base + t0) * D;
        const DT *xt = as<DT>(p.x, tile), *at = as<DT>(p.a, tile);
        const DT *bt = TIED ? at : as<DT>(p.b, tile);
        Raw<DT, VEC> x[R], a[R], b[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {  // rows past the end read the last one
            const uint32_t i = ((uint32_t)min(g * R + r, left - 1) * D + col) * sizeof(DT);
            x[r] = load_raw<VEC>(xt, i);
            a[r] = load_raw<VEC>(at, i);
            b[r] = TIED ? a[r] : load_raw<VEC>(bt, i);
        }
        float al[R][VEC], u[R][VEC];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = g * R + r < left;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float alpha, keep, beta;
                gates<DT, TIED, LOGITS>(a[r][e], b[r][e], alpha, keep, beta);
                al[r][e] = in ? alpha : 1.f;  // past the end: the identity
                u[r][e] = in ? beta * x[r][e] : 0.f;
            }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float A = 1.f, H = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                H = fmaf(al[r][e], H, u[r][e]);
                A *= al[r][e];
            }
            s_a[g][l * VEC + e] = A;
            s_h[g][l * VEC + e] = H;
        }
        __syncthreads();
        if (tid < C) {
            float A = 1.f, H = 0.f;
#pragma unroll 8
            for (int i = 0; i < G; ++i) {
                H = fmaf(s_a[i][tid], H, s_h[i][tid]);
                A *= s_a[i][tid];
            }
            if constexpr (SPLIT > 0) {
                if (mine.tile > 0) {
                    if constexpr (SPLIT > 1) publish_map(sp, mine.slot, ch, A, H);
                    const int64_t step = p.cu ? -1 : -(int64_t)p.N;
                    carry = find_state<SPLIT>(sp, mine.slot + step, step, (int32_t)mine.tile, ch);
                }
                publish_state(sp, mine.slot, ch, fmaf(A, carry, H));
            }
            float h = carry;
#pragma unroll 8
            for (int i = 0; i < G; ++i) {
                const float gh = s_h[i][tid];
                s_h[i][tid] = h;  // the state in front of group i
                h = fmaf(s_a[i][tid], h, gh);
            }
            carry = fmaf(A, carry, H);
        }
        __syncthreads();
        // a thread reads and rewrites its own places only: no third barrier
        float h[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] = s_h[g][l * VEC + e];
        DT *ot = as<DT>(p.out, tile);
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) h[e] = fmaf(al[r][e], h[e], u[r][e]);
            if (on && g * R + r < left)
                store_raw(ot, ((uint32_t)(g * R + r) * D + c0) * sizeof(DT), pack<DT>(h));
        }
        // past the end h stays the last token's state
        if (on && p.prefix_out && ((g + 1) * R & 63) == 0 && (g + 1) * R <= left) {
            const int64_t blk = scan_block_ending(p, t0 + (g + 1) * R);
            if (blk >= 0) store_raw(p.prefix_out + (prow + blk) * D, c0 * 4, pack<float>(h));
        }
        if (on && p.hT && t0 + left == len && g == (left - 1) / R)
            store_raw(p.hT + (int64_t)n * D, c0 * 4, pack<float>(h));
        t0 += Sh::kRows;
    } while (SPLIT == 0 && t0 < len);
}

// The tiles from the last to the first. The states inside a tile are formed anew
// in fp32 from the prefix state in front of it, so that no output is read and
// the decay's gradient does not inherit a rounding of one.
//
// 7 elements of traffic per token and channel against 49 vector instructions
// (780 per wave of 1,024 elements, which fill 43 us of the SIMDs): 4 x 4,097 x
// 2,048 bf16 101 us, 4.7 TB/s. Registers decide: at most 128, for two workgroups
// of 512 threads per CU, so a thread holds 4 columns of bf16 (not 8: 143 us
// against 117 when that was chosen), the raw words rather than their values, and
// one pair of columns' gradients at a time. The pairs and single columns of other
// widths have 1,024 threads and, but for fp32 without SPLIT 4, more than 64
// registers: one workgroup per CU, whose loads, chaining and gradients do not
// overlap (4 x 4,097 x 2,056 148 to 158 us).
template <typename DT, int VEC, bool TIED, bool LOGITS, int SPLIT>
__global__ __launch_bounds__((ScanShape<DT, VEC>::kThreads), 4) void scan_backward_kernel(
    ScanParams p, int ncb, ScanSplit sp) {
    using Sh = ScanShape<DT, VEC>;
    constexpr int G = Sh::kGroups, C = Sh::kCols, R = Sh::kPer;
    __shared__ float s_a[G][C], s_h[G][C], s_k[G][C];

    __shared__ int s_take[3];
    const int pair = SPLIT > 0 ? 0 : sp.runs.chain(workgroup());
    ScanTile mine{pair / ncb, pair % ncb, 0, 0};
    if constexpr (SPLIT > 0) mine = take_tile<true>(p, sp, ncb, s_take);
    if (SPLIT > 0 ? mine.n < 0 : pair < 0) return;
    const int n = mine.n, cb = mine.cb;
    const int tid = threadIdx.x, g = tid / Sh::kLanes, l = tid % Sh::kLanes;
    const int D = p.D, c0 = cb * C + l * VEC;
    const bool on = c0 < D;
    const int col = on ? c0 : 0;
    const int ch = cb * C + tid;
    const bool chain = tid < C && ch < D;
    int64_t base, len;
    scan_bounds(p, n, base, len);
    const int64_t last = len > 0 ? (len - 1) / Sh::kRows : 0;
    if constexpr (SPLIT == 0) mine.tile = last;
    float carry = 0.f;  // what reaches the tile from behind, once it is known
    if (chain && p.dhT && mine.tile == last) carry = p.dhT[(int64_t)n * D + ch];
    if (mine.tile < 0 || mine.tile * Sh::kRows >= len) {  // (below 0: malformed offsets)
        if (mine.tile == 0 && chain && p.dh0) p.dh0[(int64_t)n * D + ch] = carry;
        if constexpr (SPLIT > 0)
            if (tid < C) publish_state(sp, mine.slot, ch, 0.f);
        return;
    }
    const int64_t prow = p.prefix_in ? scan_prefix_row(p, n, base) : 0;

    int64_t t0 = mine.tile * Sh::kRows;
    const auto run_tile = [&](auto full, const int left) {
        constexpr bool FULL = decltype(full)::value;
        const int64_t tile = (base + t0) * D;
        const DT *xt = as<DT>(p.x, tile), *at = as<DT>(p.a, tile), *yt = as<DT>(p.dout, tile);
        const DT *bt = TIED ? at : as<DT>(p.b, tile);
        Raw<DT, VEC> x[R], a[R], b[R], dy[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = FULL ? g * R + r : min(g * R + r, left - 1);
            const uint32_t i = ((uint32_t)row * D + col) * sizeof(DT);
            x[r] = load_raw<VEC>(xt, i);
            a[r] = load_raw<VEC>(at, i);
            b[r] = TIED ? a[r] : load_raw<VEC>(bt, i);
            dy[r] = load_raw<VEC>(yt, i);
        }
        float h_in = 0.f;  // the state in front of the tile
        if (chain) {
            if (t0 > 0)
                h_in = p.prefix_in[(prow + scan_block_ending(p, t0)) * D + ch];
            else if (p.h0)
                h_in = p.h0[(int64_t)n * D + ch];
        }
        // alpha and beta as fp32 for both sweeps, where they fit the registers of
        // two workgroups per CU; else they are formed twice
        constexpr bool HOLD = SPLIT > 0 && sizeof(DT) == 2 && R * VEC <= 16;
        float al[HOLD ? R : 1][VEC], be[HOLD ? R : 1][VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float A = 1.f, H = 0.f, K = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool in = FULL || g * R + r < left;
                float alpha, keep, beta;
                gates<DT, TIED, LOGITS>(a[r][e], b[r][e], alpha, keep, beta);
                if constexpr (HOLD) {
                    al[r][e] = alpha;
                    be[r][e] = beta;
                }
                alpha = in ? alpha : 1.f;
                H = fmaf(alpha, H, in ? beta * x[r][e] : 0.f);
                // rows join at the far end: K = sum of dy_r times the decays up to it
                A *= alpha;
                K = fmaf(A, in ? dy[r][e] : 0.f, K);
            }
            s_a[g][l * VEC + e] = A;
            s_h[g][l * VEC + e] = H;
            s_k[g][l * VEC + e] = K;
            __builtin_amdgcn_sched_barrier(0);  // one column's gates in registers at a time
        }
        __syncthreads();
        if (tid < C) {
            float A = 1.f, K = 0.f;
#pragma unroll 8
            for (int i = G - 1; i >= 0; --i) {
                K = fmaf(s_a[i][tid], K, s_k[i][tid]);
                A *= s_a[i][tid];
            }
            if constexpr (SPLIT > 1) {
                if (mine.tile < last) publish_map(sp, mine.slot, ch, A, K);
            }
            float h = h_in;
#pragma unroll 8
            for (int i = 0; i < G; ++i) {
                const float gh = s_h[i][tid];
                s_h[i][tid] = h;
                h = fmaf(s_a[i][tid], h, gh);
            }
            if constexpr (SPLIT > 0) {
                if (mine.tile < last) {
                    const int64_t step = p.cu ? 1 : p.N;
                    carry = find_state<SPLIT>(sp, mine.slot + step, step,
                                              (int32_t)(last - mine.tile), ch);
                }
                publish_state(sp, mine.slot, ch, fmaf(A, carry, K));
            }
            float c = carry;
#pragma unroll 8
            for (int i = G - 1; i >= 0; --i) {
                const float gk = s_k[i][tid];
                s_k[i][tid] = c;  // what reaches group i from behind
                c = fmaf(s_a[i][tid], c, gk);
            }
            carry = fmaf(A, carry, K);
        }
        __syncthreads();
        forget(x);
        forget(a);
        if constexpr (!TIED) forget(b);
        forget(dy);
        float ox[R][2], oa[R][2], ob[R][2];  // gradients of a pair of columns
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float alpha[R], keep[R], beta[R], rest[R], before[R];
            float h = s_h[g][l * VEC + e], c = s_k[g][l * VEC + e];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                before[r] = h;
                if constexpr (HOLD) {
                    alpha[r] = al[r][e];
                    beta[r] = be[r][e];
                    if constexpr (LOGITS) {
                        keep[r] = TIED ? beta[r] : exp_logit(a[r][e], DT()) * alpha[r];
                        if constexpr (!TIED) rest[r] = write_rest(b[r][e], beta[r]);
                    }
                } else {
                    gates<DT, TIED, LOGITS>(a[r][e], b[r][e], alpha[r], keep[r], beta[r]);
                    if constexpr (!TIED && LOGITS) write_pair(b[r][e], beta[r], rest[r], DT());
                }
                h = fmaf(alpha[r], h, beta[r] * x[r][e]);
            }
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                const bool in = FULL || g * R + r < left;  // past the end c passes through
                const float gr = (in ? dy[r][e] : 0.f) + c;
                c = (in ? alpha[r] : 1.f) * gr;
                // alpha' = -alpha (1 - alpha), beta' = beta (1 - beta) of the logits
                const float xe = x[r][e];
                float da = gr * (TIED ? before[r] - xe : before[r]);
                if constexpr (LOGITS) da *= -alpha[r] * keep[r];
                if constexpr (!TIED) {
                    float db = gr * xe;
                    if constexpr (LOGITS) db *= beta[r] * rest[r];
                    ob[r][e & 1] = db;
                }
                oa[r][e & 1] = da;
                ox[r][e & 1] = gr * beta[r];
            }
            if ((e & 1) || VEC == 1) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    x[r].set(e & ~1, ox[r][0], ox[r][VEC > 1]);
                    a[r].set(e & ~1, oa[r][0], oa[r][VEC > 1]);
                    if constexpr (!TIED) b[r].set(e & ~1, ob[r][0], ob[r][VEC > 1]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        DT *dxt = as<DT>(p.dx, tile), *dat = as<DT>(p.da, tile), *dbt = as<DT>(p.db, TIED ? 0 : tile);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!on || (!FULL && g * R + r >= left)) continue;
            const uint32_t i = ((uint32_t)(g * R + r) * D + c0) * sizeof(DT);
            store_raw(dxt, i, x[r]);
            store_raw(dat, i, a[r]);
            if constexpr (!TIED) store_raw(dbt, i, b[r]);
        }
    };
    do {
        // code apart for whole tiles where the registers allow it (-1 %)
        constexpr bool APART = SPLIT > 0 && sizeof(DT) == 2;
        if (APART && len - t0 >= Sh::kRows)
            run_tile(std::true_type(), Sh::kRows);
        else
            run_tile(std::false_type(), (int)(len - t0 < Sh::kRows ? len - t0 : Sh::kRows));
        t0 -= Sh::kRows;
    } while (SPLIT == 0 && t0 >= 0);
    if (SPLIT > 0 && mine.tile > 0) return;
    if (chain && p.dh0) p.dh0[(int64_t)n * D + ch] = carry;
}

// K tokens per sequence against a pool of state slots: VEC channels of one
// sequence per thread, the state in registers in between. Every byte once;
// at serving sizes bound by latency (64 x 1 x 6,144 bf16, 6.3 MB: 3.3 us).
template <typename DT, int VEC, bool TIED, bool LOGITS>
__global__ __launch_bounds__(256) void scan_decode_kernel(ScanDecodeParams p) {
    const int per = (p.D + VEC - 1) / VEC;
    const int64_t i = (int64_t)workgroup() * 256 + threadIdx.x;
    const int64_t b = i / per;
    if (b >= p.B) return;
    const int c0 = (int)(i - b * per) * VEC;
    const int src = p.src[b], dst = p.dst[b];
    const bool bad = src >= p.num_slots || dst >= p.num_slots;
    float h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = bad ? __builtin_nanf("") : 0.f;
    if (!bad && src >= 0) {
        const auto s = load_raw<VEC>(p.pool + (int64_t)src * p.D, c0 * 4);
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] = s[e];
    }
    for (int k = 0; k < p.K; ++k) {
        const int64_t at = (b * p.K + k) * p.D;
        const uint32_t i = c0 * sizeof(DT);
        const auto x = load_raw<VEC>(as<DT>(p.x, at), i), a = load_raw<VEC>(as<DT>(p.a, at), i);
        const auto w = TIED ? a : load_raw<VEC>(as<DT>(p.b, at), i);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float alpha, keep, beta;
            gates<DT, TIED, LOGITS>(a[e], w[e], alpha, keep, beta);
            h[e] = fmaf(alpha, h[e], beta * x[e]);
        }
        store_raw(as<DT>(p.out, at), i, pack<DT>(h));
    }
    if (!bad && dst >= 0) store_raw(p.pool + (int64_t)dst * p.D, c0 * 4, pack<float>(h));
}

// Calls f with the kernel's element type, columns per thread and gate form as types.
template <typename DT, int VEC, typename F>
hipError_t with_scan_gates(bool tied, bool logits, F &&f) {
    if (tied)
        return logits ? f.template run<DT, VEC, true, true>() : f.template run<DT, VEC, true, false>();
    return logits ? f.template run<DT, VEC, false, true>() : f.template run<DT, VEC, false, false>();
}
// Columns per thread, for the workspace's layout and the kernel alike: 16-byte
// accesses where every row starts on 16 bytes, else pairs of bf16, else single
// columns. The bf16 backward kernel takes 4, in segments of 128 bytes, where rows
// start on 64 bytes, and else pairs in segments of 256, of which fewer straddle
// cache lines (4 x 4,097 x 2,056, both directions: 232 us against 282; 2,080 189
// in fours and 190).
enum ScanPass { kForward, kBackward, kDecode };
constexpr int kForVec = 8, kBackVec = 4, kBackRows = 32;

int scan_vec(int32_t D, int dtype, ScanPass pass) {
    if (dtype != 1) return D % 4 == 0 ? 4 : 1;
    if (pass == kBackward ? D % kBackRows == 0 : D % kForVec == 0)
        return pass == kBackward ? kBackVec : kForVec;
    return D % 2 == 0 ? 2 : 1;
}

template <ScanPass PASS, typename F>
hipError_t with_scan_types(int dtype, int32_t D, const void *b, uint32_t flags, F &&f) {
    constexpr int kWide = PASS == kBackward ? kBackVec : kForVec;
    const bool tied = b == nullptr, logits = flags & GDN_GATE_LOGITS;
    const int vec = scan_vec(D, dtype, PASS);
    if (dtype == 1)
        return vec == kWide ? with_scan_gates<__bf16, kWide>(tied, logits, f)
               : vec == 2   ? with_scan_gates<__bf16, 2>(tied, logits, f)
                            : with_scan_gates<__bf16, 1>(tied, logits, f);
    return vec == 4 ? with_scan_gates<float, 4>(tied, logits, f)
                    : with_scan_gates<float, 1>(tied, logits, f);
}

template <typename DT, int VEC> int column_blocks(int32_t D) {
    return (D + ScanShape<DT, VEC>::kCols - 1) / ScanShape<DT, VEC>::kCols;
}

// Sets a SPLIT launch's workspace: counters to 0, words to absent. A kernel and
// not a memset, whose node in a replayed graph is not to be relied on. 12.6 MB
// for 65,536 x 6,144: 6 us beside 608.
__global__ __launch_bounds__(256) void scan_clear_kernel(u32x4 *ws, int64_t zero, int64_t total) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * 256) {
        const uint32_t v = i < zero ? 0u : kAbsent;
        ws[i] = u32x4{v, v, v, v};
    }
}

// The workspace of a SPLIT launch: counters, then maps (SPLIT > 1), then states.
struct ScanLayout {
    int64_t chains, slots, width, words_at, bytes;
    int deep;
};

// How far the tiles of few chains look. The more tiles of a chain are under way
// at once, the further back it pays to look, as long as the looking stays small:
// with 4 chains (32,768 tokens of 512 bf16 channels) 4 deep takes 66 us and 1
// deep 131, with 16 120 and 160, with 48 (65,536 x 6,144) 618 and 612. These are
// long chains, most of whose tiles wait to be launched; short ones whose tiles
// all run at once (2 x 1,000 x 1,111 has 36 of 8) follow the rule unmeasured.
constexpr int kDeep = 4;
constexpr int64_t kDeepChains = 24;

ScanLayout scan_layout(int64_t nseq, int64_t tokens, int32_t D, int cols, bool packed) {
    ScanLayout l;
    const int64_t ncb = (D + cols - 1) / cols;
    l.width = ncb * cols;
    l.chains = packed ? ncb : nseq * ncb;
    l.slots = packed ? tokens / GDN_SCAN_TILE + nseq
                     : nseq * ((tokens + GDN_SCAN_TILE - 1) / GDN_SCAN_TILE);
    l.words_at = (l.chains * 4 + 255) / 256 * 256;
    l.deep = l.chains <= kDeepChains ? kDeep : 1;
    l.bytes = l.words_at + l.slots * l.width * (l.deep > 1 ? 12 : 4);
    return l;
}

// Whether a call is cut along time: sequences of more than one tile, and either
// not enough (sequence, column block) pairs to fill the device with one
// workgroup each (128 x 512 x 2,048 bf16, 16 pairs per CU: 194 us uncut, 197
// cut; 33 packed sequences of 20,011 x 2,048 fp32, 4 pairs: 227 and 136), or a
// packed batch of a tile per sequence or more on average, whose longest
// sequence may be most of it (128 sequences, 24,576 x 4,096: 221 uncut, 215 cut;
// shorter ones lose, 300 sequences, 24,576 x 2,048: 138 and 172).
bool scan_wants_split(int64_t nseq, int64_t tokens, int64_t ncb, bool packed, int cus) {
    if (tokens <= GDN_SCAN_TILE) return false;
    return nseq * ncb < 8 * (int64_t)cus || (packed && tokens >= nseq * GDN_SCAN_TILE);
}

// Channels of a tile.
int scan_cols(int32_t D, int dtype, bool back) {
    const int vec = scan_vec(D, dtype, back ? kBackward : kForward);
    if (dtype == 1)
        return vec == kForVec    ? ScanShape<__bf16, kForVec>::kCols
               : vec == kBackVec ? ScanShape<__bf16, kBackVec>::kCols
               : vec == 2        ? ScanShape<__bf16, 2>::kCols
                                 : ScanShape<__bf16, 1>::kCols;
    return vec == 4 ? ScanShape<float, 4>::kCols : ScanShape<float, 1>::kCols;
}

}  // namespace

size_t scan_workspace_bytes(int64_t nseq, int64_t tokens, int32_t D, int dtype, bool packed,
                            int cus) {
    int64_t most = 0;  // of the forward and the backward call
    for (const bool back : {false, true}) {
        const int cols = scan_cols(D, dtype, back);
        const ScanLayout l = scan_layout(nseq, tokens, D, cols, packed);
        if (scan_wants_split(nseq, tokens, l.width / cols, packed, cus) && l.bytes > most)
            most = l.bytes;
    }
    return (size_t)most;
}

namespace {

// Fills sp and clears the workspace when the call is to be cut; sp.slots is 0
// when not.
hipError_t prepare_split(const ScanParams &p, int dtype, int cus, void *ws, size_t ws_bytes,
                         bool back, ScanSplit &sp, hipStream_t stream) {
    sp = ScanSplit{};
    const bool packed = p.cu != nullptr;
    const int64_t tokens = packed ? p.total : p.T;
    const int cols = scan_cols(p.D, dtype, back);
    const ScanLayout l = scan_layout(p.N, tokens, p.D, cols, packed);
    const int64_t ncb = l.width / cols;
    sp.runs = XcdRuns::make(p.N * ncb, ncb);  // one workgroup each, unless cut
    if (!ws || ws_bytes < scan_workspace_bytes(p.N, tokens, p.D, dtype, packed, cus) ||
        !scan_wants_split(p.N, tokens, ncb, packed, cus))
        return hipSuccess;
    sp.runs = XcdRuns::make(l.chains, ncb);
    sp.per_chain = l.slots * ncb / l.chains;
    char *base = static_cast<char *>(ws);
    sp.ticket = reinterpret_cast<uint32_t *>(base);
    sp.map = reinterpret_cast<uint64_t *>(base + l.words_at);
    sp.state = reinterpret_cast<uint32_t *>(base + l.words_at) +
               (l.deep > 1 ? 2 * l.slots * l.width : 0);
    sp.deep = l.deep;
    sp.slots = (int32_t)l.slots;
    sp.width = (int32_t)l.width;
    const int64_t total = (l.bytes + 15) / 16, wgs = (total + 255) / 256;
    hipLaunchKernelGGL(scan_clear_kernel, dim3((unsigned)(wgs < 8192 ? wgs : 8192)), dim3(256), 0,
                       stream, static_cast<u32x4 *>(ws), l.words_at / 16, total);
    return hipGetLastError();
}

struct RunForward {
    const ScanParams &p;
    const ScanSplit &sp;
    hipStream_t stream;
    template <typename DT, int VEC, bool TIED, bool LOGITS> hipError_t run() const {
        const int ncb = column_blocks<DT, VEC>(p.D);
        const dim3 block(ScanShape<DT, VEC>::kThreads);
        const dim3 grid = grid_of((sp.slots > 0 ? sp.per_chain : 1) * sp.runs.grid, block.x);
        if (sp.slots > 0 && sp.deep > 1)
            hipLaunchKernelGGL((scan_forward_kernel<DT, VEC, TIED, LOGITS, kDeep>), grid, block, 0,
                               stream, p, ncb, sp);
        else if (sp.slots > 0)
            hipLaunchKernelGGL((scan_forward_kernel<DT, VEC, TIED, LOGITS, 1>), grid, block, 0,
                               stream, p, ncb, sp);
        else
            hipLaunchKernelGGL((scan_forward_kernel<DT, VEC, TIED, LOGITS, 0>), grid, block, 0,
                               stream, p, ncb, sp);
        return hipGetLastError();
    }
};

struct RunBackward {
    const ScanParams &p;
    const ScanSplit &sp;
    hipStream_t stream;
    template <typename DT, int VEC, bool TIED, bool LOGITS> hipError_t run() const {
        const int ncb = column_blocks<DT, VEC>(p.D);
        const dim3 block(ScanShape<DT, VEC>::kThreads);
        const dim3 grid = grid_of((sp.slots > 0 ? sp.per_chain : 1) * sp.runs.grid, block.x);
        if (sp.slots > 0 && sp.deep > 1)
            hipLaunchKernelGGL((scan_backward_kernel<DT, VEC, TIED, LOGITS, kDeep>), grid, block, 0,
                               stream, p, ncb, sp);
        else if (sp.slots > 0)
            hipLaunchKernelGGL((scan_backward_kernel<DT, VEC, TIED, LOGITS, 1>), grid, block, 0,
                               stream, p, ncb, sp);
        else
            hipLaunchKernelGGL((scan_backward_kernel<DT, VEC, TIED, LOGITS, 0>), grid, block, 0,
                               stream, p, ncb, sp);
        return hipGetLastError();
    }
};

struct RunDecode {
    const ScanDecodeParams &p;
    hipStream_t stream;
    template <typename DT, int VEC, bool TIED, bool LOGITS> hipError_t run() const {
        const int64_t threads = (int64_t)p.B * ((p.D + VEC - 1) / VEC);
        hipLaunchKernelGGL((scan_decode_kernel<DT, VEC, TIED, LOGITS>),
                           grid_of((threads + 255) / 256, 256), dim3(256), 0, stream, p);
        return hipGetLastError();
    }
};

}  // namespace

hipError_t launch_scan(const ScanParams &p, int dtype, int cus, void *ws, size_t ws_bytes,
                       hipStream_t stream) {
    ScanSplit sp;
    const hipError_t e = prepare_split(p, dtype, cus, ws, ws_bytes, false, sp, stream);
    if (e != hipSuccess) return e;
    return with_scan_types<kForward>(dtype, p.D, p.b, p.flags, RunForward{p, sp, stream});
}

hipError_t launch_scan_backward(const ScanParams &p, int dtype, int cus, void *ws,
                                size_t ws_bytes, hipStream_t stream) {
    ScanSplit sp;
    const hipError_t e = prepare_split(p, dtype, cus, ws, ws_bytes, true, sp, stream);
    if (e != hipSuccess) return e;
    return with_scan_types<kBackward>(dtype, p.D, p.b, p.flags, RunBackward{p, sp, stream});
}

hipError_t launch_scan_decode(const ScanDecodeParams &p, int dtype, hipStream_t stream) {
    return with_scan_types<kDecode>(dtype, p.D, p.b, p.flags, RunDecode{p, stream});
}

}  // namespace gdn
