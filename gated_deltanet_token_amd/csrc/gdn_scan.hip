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
#include "gdn_scan.hpp"

namespace gdn {

namespace {

// One workgroup per (sequence, column block), its tiles in order.
template <typename DT, int VEC, bool TIED, bool LOGITS>
__global__ __launch_bounds__((ScanShape<DT, VEC>::kThreads)) void scan_forward_kernel(
    ScanParams p, int ncb) {
    using Sh = ScanShape<DT, VEC>;
    constexpr int G = Sh::kGroups, C = Sh::kCols, R = Sh::kPer;
    __shared__ float s_a[G][C], s_h[G][C];

    const int n = blockIdx.x / ncb, cb = blockIdx.x - n * ncb;
    const int tid = threadIdx.x, g = tid / Sh::kLanes, l = tid % Sh::kLanes;
    const int D = p.D, c0 = cb * C + l * VEC;
    const bool on = c0 < D;
    const int col = on ? c0 : 0;  // lanes past the last column read the first, and write nothing
    const int ch = cb * C + tid;  // the channel that this thread chains
    const bool chain = tid < C && ch < D;
    int64_t base, len;
    scan_bounds(p, n, base, len);
    float carry = 0.f;
    if (chain && p.h0) carry = p.h0[(int64_t)n * D + ch];
    if (len == 0) {
        if (chain && p.hT) p.hT[(int64_t)n * D + ch] = carry;
        return;
    }
    const int64_t prow = p.prefix_out ? scan_prefix_row(p, n, base) : 0;

    for (int64_t t0 = 0; t0 < len; t0 += Sh::kRows) {
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
                gates<TIED, LOGITS>(a[r][e], b[r][e], alpha, keep, beta);
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
            float A = 1.f, H = 0.f, h = carry;
#pragma unroll 4
            for (int i = 0; i < G; ++i) {
                const float ga = s_a[i][tid], gh = s_h[i][tid];
                s_h[i][tid] = h;  // the state in front of group i
                h = fmaf(ga, h, gh);
                H = fmaf(ga, H, gh);
                A *= ga;
            }
            carry = fmaf(A, carry, H);
        }
        __syncthreads();
        // a thread reads and rewrites its own places only: no third barrier
        Raw<float, VEC> h;
#pragma unroll
        for (int e = 0; e < VEC; ++e) h.v[e] = s_h[g][l * VEC + e];
        DT *ot = as<DT>(p.out, tile);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            Raw<DT, VEC> o;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                h.v[e] = fmaf(al[r][e], h[e], u[r][e]);
                o.set(e, h[e]);
            }
            if (on && g * R + r < left)
                store_raw(ot, ((uint32_t)(g * R + r) * D + c0) * sizeof(DT), o);
        }
        // past the end h stays the last token's state
        if (on && p.prefix_out && ((g + 1) * R & 63) == 0 && (g + 1) * R <= left) {
            const int64_t blk = scan_block_ending(p, t0 + (g + 1) * R);
            if (blk >= 0) store_raw(p.prefix_out + (prow + blk) * D, c0 * 4, h);
        }
        if (on && p.hT && t0 + left == len && g == (left - 1) / R)
            store_raw(p.hT + (int64_t)n * D, c0 * 4, h);
    }
}

template <typename DT, int VEC, bool TIED, bool LOGITS>
__global__ __launch_bounds__((ScanShape<DT, VEC>::kThreads)) void scan_backward_kernel(
    ScanParams p, int ncb) {
    using Sh = ScanShape<DT, VEC>;
    constexpr int G = Sh::kGroups, C = Sh::kCols, R = Sh::kPer;
    __shared__ float s_a[G][C], s_h[G][C], s_k[G][C];

    const int n = blockIdx.x / ncb, cb = blockIdx.x - n * ncb;
    const int tid = threadIdx.x, g = tid / Sh::kLanes, l = tid % Sh::kLanes;
    const int D = p.D, c0 = cb * C + l * VEC;
    const bool on = c0 < D;
    const int col = on ? c0 : 0;
    const int ch = cb * C + tid;
    const bool chain = tid < C && ch < D;
    int64_t base, len;
    scan_bounds(p, n, base, len);
    float carry = 0.f;
    if (chain && p.dhT) carry = p.dhT[(int64_t)n * D + ch];
    const int64_t prow = p.prefix_in ? scan_prefix_row(p, n, base) : 0;

    for (int64_t t0 = (len - 1) / Sh::kRows * Sh::kRows; len > 0 && t0 >= 0; t0 -= Sh::kRows) {
        const int left = (int)(len - t0 < Sh::kRows ? len - t0 : Sh::kRows);
        const int64_t tile = (base + t0) * D;
        const DT *xt = as<DT>(p.x, tile), *at = as<DT>(p.a, tile), *yt = as<DT>(p.dout, tile);
        const DT *bt = TIED ? at : as<DT>(p.b, tile);
        Raw<DT, VEC> x[R], a[R], b[R], dy[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t i = ((uint32_t)min(g * R + r, left - 1) * D + col) * sizeof(DT);
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
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float A = 1.f, H = 0.f, K = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const bool in = g * R + r < left;
                float alpha, keep, beta;
                gates<TIED, LOGITS>(a[r][e], b[r][e], alpha, keep, beta);
                alpha = in ? alpha : 1.f;
                H = fmaf(alpha, H, in ? beta * x[r][e] : 0.f);
                // rows join at the far end: K = sum of dy_r times the decays up to it
                A *= alpha;
                K = fmaf(A, in ? dy[r][e] : 0.f, K);
            }
            s_a[g][l * VEC + e] = A;
            s_h[g][l * VEC + e] = H;
            s_k[g][l * VEC + e] = K;
        }
        __syncthreads();
        if (tid < C) {
            float h = h_in;
#pragma unroll 4
            for (int i = 0; i < G; ++i) {
                const float gh = s_h[i][tid];
                s_h[i][tid] = h;
                h = fmaf(s_a[i][tid], h, gh);
            }
            float A = 1.f, K = 0.f, c = carry;
#pragma unroll 4
            for (int i = G - 1; i >= 0; --i) {
                const float ga = s_a[i][tid], gk = s_k[i][tid];
                s_k[i][tid] = c;  // what reaches group i from behind
                c = fmaf(ga, c, gk);
                K = fmaf(ga, K, gk);
                A *= ga;
            }
            carry = fmaf(A, carry, K);
        }
        __syncthreads();
        forget_all(a);
        if constexpr (!TIED) forget_all(b);
        Raw<float, VEC> before[R];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float h = s_h[g][l * VEC + e];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float alpha, keep, beta;
                before[r].v[e] = h;
                gates<TIED, LOGITS>(a[r][e], b[r][e], alpha, keep, beta);
                h = fmaf(alpha, h, beta * x[r][e]);
            }
        }
        if constexpr (R > 4) {  // more rows than registers for their gates
            forget_all(a);
            if constexpr (!TIED) forget_all(b);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float c = s_k[g][l * VEC + e];
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                const bool in = g * R + r < left;  // past the end c passes through
                float alpha, keep, beta, rest = 0.f;
                gates<TIED, LOGITS>(a[r][e], b[r][e], alpha, keep, beta);
                if constexpr (!TIED && LOGITS) sigmoid_pair(-b[r][e], beta, rest);
                const float gr = (in ? dy[r][e] : 0.f) + c;
                c = (in ? alpha : 1.f) * gr;
                // alpha' = -alpha (1 - alpha), beta' = beta (1 - beta) of the logits
                const float xe = x[r][e];
                float da = gr * (TIED ? before[r][e] - xe : before[r][e]);
                if constexpr (LOGITS) da *= -alpha * keep;
                if constexpr (!TIED) {
                    float db = gr * xe;
                    if constexpr (LOGITS) db *= beta * rest;
                    b[r].set(e, db);
                }
                a[r].set(e, da);
                x[r].set(e, gr * beta);
            }
        }
        DT *dxt = as<DT>(p.dx, tile), *dat = as<DT>(p.da, tile), *dbt = as<DT>(p.db, TIED ? 0 : tile);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!on || g * R + r >= left) continue;
            const uint32_t i = ((uint32_t)(g * R + r) * D + c0) * sizeof(DT);
            store_raw(dxt, i, x[r]);
            store_raw(dat, i, a[r]);
            if constexpr (!TIED) store_raw(dbt, i, b[r]);
        }
    }
    if (chain && p.dh0) p.dh0[(int64_t)n * D + ch] = carry;
}

// K tokens per sequence against a pool of state slots: VEC channels of one
// sequence per thread, the state in registers in between.
template <typename DT, int VEC, bool TIED, bool LOGITS>
__global__ __launch_bounds__(256) void scan_decode_kernel(ScanDecodeParams p) {
    const int per = (p.D + VEC - 1) / VEC;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t b = i / per;
    if (b >= p.B) return;
    const int c0 = (int)(i - b * per) * VEC;
    const int src = p.src[b], dst = p.dst[b];
    const bool bad = src >= p.num_slots || dst >= p.num_slots;
    Raw<float, VEC> h;
#pragma unroll
    for (int e = 0; e < VEC; ++e) h.v[e] = bad ? __builtin_nanf("") : 0.f;
    if (!bad && src >= 0) h = load_raw<VEC>(p.pool + (int64_t)src * p.D, c0 * 4);
    for (int k = 0; k < p.K; ++k) {
        const int64_t at = (b * p.K + k) * p.D;
        const uint32_t i = c0 * sizeof(DT);
        const auto x = load_raw<VEC>(as<DT>(p.x, at), i), a = load_raw<VEC>(as<DT>(p.a, at), i);
        const auto w = TIED ? a : load_raw<VEC>(as<DT>(p.b, at), i);
        Raw<DT, VEC> o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float alpha, keep, beta;
            gates<TIED, LOGITS>(a[e], w[e], alpha, keep, beta);
            h.v[e] = fmaf(alpha, h[e], beta * x[e]);
            o.set(e, h[e]);
        }
        store_raw(as<DT>(p.out, at), i, o);
    }
    if (!bad && dst >= 0) store_raw(p.pool + (int64_t)dst * p.D, c0 * 4, h);
}

// Calls f with the kernel's element type, vector width and gate form as types:
// 16-byte accesses where every row starts on 16 bytes.
template <typename DT, int VEC, typename F>
hipError_t with_scan_gates(bool tied, bool logits, F &&f) {
    if (tied)
        return logits ? f.template run<DT, VEC, true, true>() : f.template run<DT, VEC, true, false>();
    return logits ? f.template run<DT, VEC, false, true>() : f.template run<DT, VEC, false, false>();
}
template <typename F>
hipError_t with_scan_types(int dtype, int32_t D, const void *b, uint32_t flags, F &&f) {
    const bool tied = b == nullptr, logits = flags & GDN_GATE_LOGITS;
    if (dtype == 1)
        return D % 8 == 0 ? with_scan_gates<__bf16, 8>(tied, logits, f)
                          : with_scan_gates<__bf16, 1>(tied, logits, f);
    return D % 4 == 0 ? with_scan_gates<float, 4>(tied, logits, f)
                      : with_scan_gates<float, 1>(tied, logits, f);
}

template <typename DT, int VEC> int column_blocks(int32_t D) {
    return (D + ScanShape<DT, VEC>::kCols - 1) / ScanShape<DT, VEC>::kCols;
}

struct RunForward {
    const ScanParams &p;
    hipStream_t stream;
    template <typename DT, int VEC, bool TIED, bool LOGITS> hipError_t run() const {
        const int ncb = column_blocks<DT, VEC>(p.D);
        hipLaunchKernelGGL((scan_forward_kernel<DT, VEC, TIED, LOGITS>), dim3((unsigned)(p.N * ncb)),
                           dim3(ScanShape<DT, VEC>::kThreads), 0, stream, p, ncb);
        return hipGetLastError();
    }
};

struct RunBackward {
    const ScanParams &p;
    hipStream_t stream;
    template <typename DT, int VEC, bool TIED, bool LOGITS> hipError_t run() const {
        const int ncb = column_blocks<DT, VEC>(p.D);
        hipLaunchKernelGGL((scan_backward_kernel<DT, VEC, TIED, LOGITS>), dim3((unsigned)(p.N * ncb)),
                           dim3(ScanShape<DT, VEC>::kThreads), 0, stream, p, ncb);
        return hipGetLastError();
    }
};

struct RunDecode {
    const ScanDecodeParams &p;
    hipStream_t stream;
    template <typename DT, int VEC, bool TIED, bool LOGITS> hipError_t run() const {
        const int64_t threads = (int64_t)p.B * ((p.D + VEC - 1) / VEC);
        hipLaunchKernelGGL((scan_decode_kernel<DT, VEC, TIED, LOGITS>),
                           dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream, p);
        return hipGetLastError();
    }
};

}  // namespace

size_t scan_workspace_bytes(int64_t, int64_t, int32_t, int, bool, int) { return 0; }

hipError_t launch_scan(const ScanParams &p, int dtype, int, void *, size_t, hipStream_t stream) {
    return with_scan_types(dtype, p.D, p.b, p.flags, RunForward{p, stream});
}

hipError_t launch_scan_backward(const ScanParams &p, int dtype, int, void *, size_t,
                                hipStream_t stream) {
    return with_scan_types(dtype, p.D, p.b, p.flags, RunBackward{p, stream});
}

hipError_t launch_scan_decode(const ScanDecodeParams &p, int dtype, hipStream_t stream) {
    return with_scan_types(dtype, p.D, p.b, p.flags, RunDecode{p, stream});
}

}  // namespace gdn
