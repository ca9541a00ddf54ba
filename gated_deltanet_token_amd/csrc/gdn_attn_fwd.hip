// gdn_attn_fwd.hip -- causal softmax attention with grouped heads over whole
// prompts (gfx950), dense and packed.
//
//   o_t = sum_{j <= t} p_tj v_j,  p_tj = exp(scale q_t . k_j - lse_t),
//   lse_t = log sum_{j <= t} exp(scale q_t . k_j)
//
// One pass over the keys with a running reference and sum per query
// (gdn_attn.hpp). Bound by the matrix instructions, beside them by LDS reads (a
// fragment of keys or values feeds CT products) and the vector instructions of
// the exponentials. 8,192 tokens of 24/4 heads of 256: 779 to 808 us, 1,020 to
// 1,058 TFLOP/s, matrix instructions busy 49 % of the time; 2 x 8,192 of 16/4
// heads of 128 500 to 525 us (1,047 to 1,099), of 64 312 to 327 us (840 to 882: more
// exponentials per product). fp32, 4,096 of 16/4 heads of 128: 662 us, 104 TFLOP/s.
#include "gdn_attn.hpp"

namespace gdn {

namespace {

template <typename DT, int D, int CT, int NW, int BK, int PER_SIMD>
__global__ __launch_bounds__(64 * NW, PER_SIMD) void attn_kernel(AttnParams p, HeadOrder order) {
    using Tiles = KeyTiles<DT, D, CT, NW, BK>;
    constexpr int BM = NW * CT * 16;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const int lane = threadIdx.x & 63, c = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int unit, slot;
    if (!order.pick(workgroup(), unit, slot)) return;
    const SeqTile s = seq_tile<BM>(p.cu, p.N, p.T, p.total, unit, slot, order.tiles, p.Hq, lane);
    if (s.tile >= s.tiles) return;
    const int64_t tok0 = s.tok0;
    const int len = s.len, head = s.head, tile = s.tiles - 1 - s.tile;  // long tiles first
    const int q0 = tile * BM, w0 = q0 + wave * CT * 16;
    const int kh = head / (p.Hq / p.Hk);

    const DT *q = static_cast<const DT *>(p.q);
    Frag<DT> qf[D / 32][CT];
    int lim[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int row = min(w0 + 16 * ct + c, len - 1);
        lim[ct] = row + 1;
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
            qf[kk][ct] = Rows<DT, D>::load(q + ((tok0 + row) * p.Hq + head) * D, kk, g4);
    }
    const int64_t stride = (int64_t)p.Hk * D * sizeof(DT);
    DenseKeys src;
    src.k = static_cast<const unsigned char *>(p.k) + tok0 * stride + kh * Rows<DT, D>::kPitch;
    src.v = static_cast<const unsigned char *>(p.v) + tok0 * stride + kh * Rows<DT, D>::kPitch;
    src.stride = stride;
    src.len = len;
    Attend<DT, D, CT> st;
    st.clear();
    const int hi = w0 < len ? min(w0 + CT * 16, len) : 0;
    Tiles::template run<false>(st, qf, src, 0, min(q0 + BM, len), lim, q0 + 1, min(w0, len) + 1,
                               hi, (uint32_t)stride, p.scale * kLog2e, lds);
    st.finish();
    DT *out = static_cast<DT *>(p.out);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int row = w0 + 16 * ct + c;
        if (row >= len) continue;
        const float inv = st.l[ct] == 0.f ? 0.f : 1.f / st.l[ct];
        DT *o = out + ((tok0 + row) * p.Hq + head) * D + 4 * g4;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) store4(o + 16 * dt, st.acc[dt][ct] * inv);
        if (p.lse && g4 == 0) p.lse[(tok0 + row) * p.Hq + head] = st.lse(ct);
    }
}

template <typename DT, int D, int CT, int NW, int BK, int PER_SIMD>
hipError_t launch(const AttnParams &p, hipStream_t stream) {
    using Tiles = KeyTiles<DT, D, CT, NW, BK>;
    constexpr int BM = NW * CT * 16;
    const HeadOrder order =
        p.cu ? HeadOrder::make(p.Hq, p.total / BM + p.N)
             : HeadOrder::make((int64_t)p.N * p.Hq, (p.T + BM - 1) / BM);
    const auto kernel = attn_kernel<DT, D, CT, NW, BK, PER_SIMD>;
    const hipError_t e = with_lds(kernel, Tiles::kLds);
    if (e != hipSuccess) return e;
    kernel<<<grid_of(order.grid(), 64 * NW), 64 * NW, Tiles::kLds, stream>>>(p, order);
    return hipGetLastError();
}

}  // namespace

// Workgroups of BIG waves, or of SMALL where there would not be one for every CU: a wave has as
// many products, but fewer neighbours on its SIMD and in LDS (1,000 tokens of 24/4 heads of 256:
// 49 against 66 us; 3 x 331 of 6/2 fp32 heads of 64, with gradients, 88 against 109). bf16 heads
// up to 128 gain nothing from 2 waves instead of 4 (1,000 tokens of 16/4 heads, with
// gradients: 134 against 129).
template <typename DT, int D, int CT, int BIG, int SMALL, int BK>
hipError_t by_size(const AttnParams &p, int cus, hipStream_t stream) {
    constexpr int BM = BIG * CT * 16;
    const int64_t tiles = p.cu ? p.total / BM + 1 : p.N * ((p.T + BM - 1) / BM);
    return tiles * p.Hq >= cus ? launch<DT, D, CT, BIG, BK, 2>(p, stream)
                               : launch<DT, D, CT, SMALL, BK, 2>(p, stream);
}

hipError_t launch_attn(const AttnParams &p, int dtype, int D, int cus, hipStream_t stream) {
    if (dtype == 1) {
        if (D == 64) return launch<__bf16, 64, 2, 4, 64, 2>(p, stream);
        if (D == 128) return launch<__bf16, 128, 2, 4, 64, 2>(p, stream);
        return by_size<__bf16, 256, 2, 8, 4, 64>(p, cus, stream);
    }
    if (D == 64) return by_size<float, 64, 1, 8, 2, 64>(p, cus, stream);
    if (D == 128) return by_size<float, 128, 1, 8, 2, 64>(p, cus, stream);
    return by_size<float, 256, 1, 8, 4, 32>(p, cus, stream);
}

}  // namespace gdn
