// gdn_ops_validate.hpp -- host-side argument checks of the scan, norm and beam
// calls of the C ABI (include/gdn.h).
//
// Plain C++ with no HIP runtime call, like gdn_validate.hpp, so that the same
// code is compiled into the library and into a host-only test program built
// with sanitizers. Every function returns a status and has no side effects.
#pragma once
#include "gdn_validate.hpp"

namespace gdn {
namespace val {

constexpr int64_t kMaxGrid = 0x7FFFFFFF;
constexpr int32_t kMaxScanWidth = 1 << 22;  // 128 tokens of fp32 within 32-bit offsets
constexpr int32_t kMaxNormWidth = 16384;
constexpr int32_t kMaxBeams = 32;

// a * b * c, or -1 when it does not fit in int64 (factors >= 0).
static inline int64_t bytes_of(int64_t a, int64_t b, int64_t c) {
    return mul_ok(a, b) && mul_ok(a, c) ? a : -1;
}

// Every output apart from every input and from every other output.
template <int NI, int NO>
static inline bool any_overlap(const Range (&in)[NI], const Range (&out)[NO]) {
    for (int i = 0; i < NO; ++i) {
        for (const Range &r : in)
            if (overlap(out[i], r)) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

template <int N> static inline bool all_aligned(const void *const (&ptrs)[N], uintptr_t to) {
    for (const void *p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & (to - 1)) return false;
    return true;
}

// The calls of the gated linear recurrence. `tokens` is B * T or total_T,
// `nstates` B or N, `longest` the most tokens one sequence can have.
struct ScanArgs {
    const void *x, *a, *b;
    const float *h0;
    const int32_t *cu;
    int64_t cu_count;
    int64_t tokens, nstates, longest;
    int32_t D;
    gdn_dtype_t dtype;
    uint32_t flags;
    const float *prefix;
    int32_t prefix_interval;
    int64_t prefix_rows;
    const void *ws;
    size_t ws_bytes;
};

// Workgroups of a scan call: a tile of tokens by at least 64 channels each.
static inline bool scan_fits(int64_t tokens, int64_t nstates, int32_t D) {
    int64_t wgs = tokens / GDN_SCAN_TILE + nstates;
    return mul_ok(wgs, (D + (int64_t)63) / 64 + 8) && wgs <= kMaxGrid;
}

static inline gdn_status_t check_scan_common(const ScanArgs &s, int64_t &nx, int64_t &nst,
                                             int64_t &npre) {
    if (s.nstates < 1 || s.tokens < 0 || s.D < 1) return GDN_ERR_BAD_SHAPE;
    if (!known_dtype(s.dtype) || s.D > kMaxScanWidth) return GDN_ERR_UNSUPPORTED;
    if (s.flags & ~(uint32_t)GDN_GATE_LOGITS) return GDN_ERR_UNSUPPORTED;
    if (s.prefix && s.prefix_interval < 1) return GDN_ERR_BAD_SHAPE;
    nx = bytes_of(s.tokens, s.D, s.dtype == GDN_BF16 ? 2 : 4);
    nst = bytes_of(s.nstates, s.D, 4);
    npre = s.prefix ? bytes_of(s.prefix_rows, s.D, 4) : 0;
    if (nx < 0 || nst < 0 || npre < 0) return GDN_ERR_BAD_SHAPE;
    if (!scan_fits(s.tokens, s.nstates, s.D)) return GDN_ERR_BAD_SHAPE;
    if (s.tokens > 0 && (!s.x || !s.a)) return GDN_ERR_NULL_POINTER;
    if (s.cu_count > 0 && !s.cu) return GDN_ERR_NULL_POINTER;
    if (s.ws_bytes > (size_t)INT64_MAX) return GDN_ERR_BAD_SHAPE;
    return GDN_OK;
}

static inline gdn_status_t check_scan(const ScanArgs &s, const void *out, const float *hT) {
    int64_t nx, nst, npre;
    const gdn_status_t st = check_scan_common(s, nx, nst, npre);
    if (st != GDN_OK) return st;
    if (s.tokens > 0 && !out) return GDN_ERR_NULL_POINTER;
    const void *ptrs[] = {s.x, s.a, s.b, s.h0, s.cu, s.prefix, s.ws, out, hT};
    if (!all_aligned(ptrs, 16)) return GDN_ERR_MISALIGNED;
    // final_state may be initial_state itself
    const Range rh0 = range_of(s.h0, s.h0 == hT ? 0 : nst);
    const Range in[] = {range_of(s.x, nx), range_of(s.a, nx), range_of(s.b, nx), rh0,
                        range_of(s.cu, s.cu_count * 4)};
    const Range ro[] = {range_of(out, nx), range_of(hT, nst), range_of(s.prefix, npre),
                        range_of(s.ws, (int64_t)s.ws_bytes)};
    return any_overlap(in, ro) ? GDN_ERR_ALIAS : GDN_OK;
}

static inline gdn_status_t check_scan_backward(const ScanArgs &s, const void *dout,
                                               const float *dfinal, const void *dx,
                                               const void *da, const void *db,
                                               const float *dh0) {
    int64_t nx, nst, npre;
    const gdn_status_t st = check_scan_common(s, nx, nst, npre);
    if (st != GDN_OK) return st;
    if (s.prefix && GDN_SCAN_TILE % (64 * (int64_t)s.prefix_interval) != 0)
        return GDN_ERR_UNSUPPORTED;
    if (s.tokens > 0 && (!dout || !dx || !da || (s.b && !db))) return GDN_ERR_NULL_POINTER;
    if (!s.b && db) return GDN_ERR_BAD_SHAPE;
    if (!s.prefix && s.longest > GDN_SCAN_TILE) return GDN_ERR_NULL_POINTER;
    const void *ptrs[] = {s.x, s.a, s.b, s.h0, s.cu, s.prefix, s.ws, dout, dfinal, dx, da, db,
                          dh0};
    if (!all_aligned(ptrs, 16)) return GDN_ERR_MISALIGNED;
    const Range in[] = {range_of(s.x, nx),      range_of(s.a, nx),    range_of(s.b, nx),
                        range_of(s.h0, nst),    range_of(dout, nx),   range_of(dfinal, nst),
                        range_of(s.prefix, npre), range_of(s.cu, s.cu_count * 4)};
    const Range ro[] = {range_of(dx, nx), range_of(da, nx), range_of(db, nx),
                        range_of(dh0, nst), range_of(s.ws, (int64_t)s.ws_bytes)};
    return any_overlap(in, ro) ? GDN_ERR_ALIAS : GDN_OK;
}

static inline gdn_status_t check_scan_decode(const void *x, const void *a, const void *b,
                                             const float *pool, int32_t num_slots,
                                             const int32_t *src, const int32_t *dst,
                                             const void *out, int32_t B, int32_t K, int32_t D,
                                             gdn_dtype_t dtype, uint32_t flags) {
    if (B < 1 || K < 0 || D < 1 || num_slots < 1) return GDN_ERR_BAD_SHAPE;
    if (!known_dtype(dtype) || D > kMaxScanWidth) return GDN_ERR_UNSUPPORTED;
    if (flags & ~(uint32_t)GDN_GATE_LOGITS) return GDN_ERR_UNSUPPORTED;
    int64_t tok = B;
    if (!mul_ok(tok, K)) return GDN_ERR_BAD_SHAPE;
    const int64_t nx = bytes_of(tok, D, dtype == GDN_BF16 ? 2 : 4);
    const int64_t npool = bytes_of(num_slots, D, 4);
    if (nx < 0 || npool < 0) return GDN_ERR_BAD_SHAPE;
    if ((int64_t)B * ((D + 63) / 64) > kMaxGrid) return GDN_ERR_BAD_SHAPE;
    if (!pool || !src || !dst) return GDN_ERR_NULL_POINTER;
    if (K > 0 && (!x || !a || !out)) return GDN_ERR_NULL_POINTER;
    const void *ptrs[] = {x, a, b, pool, out};
    if (!all_aligned(ptrs, 16)) return GDN_ERR_MISALIGNED;
    const void *slots[] = {src, dst};
    if (!all_aligned(slots, 4)) return GDN_ERR_MISALIGNED;
    const Range in[] = {range_of(x, nx), range_of(a, nx), range_of(b, nx),
                        range_of(src, (int64_t)B * 4), range_of(dst, (int64_t)B * 4)};
    const Range ro[] = {range_of(out, nx), range_of(pool, npool)};
    return any_overlap(in, ro) ? GDN_ERR_ALIAS : GDN_OK;
}

static inline int64_t norm_groups(int32_t D, int32_t group) {
    return group == 0 ? 1 : (D + group - 1) / group;
}

static inline gdn_status_t check_norm_shape(int64_t rows, int32_t D, gdn_dtype_t dtype,
                                            float eps, int64_t &n) {
    if (rows < 0 || rows > kMaxGrid || D < 1) return GDN_ERR_BAD_SHAPE;
    if (!(eps >= 0x1p-126f) || eps > 3.0e38f) return GDN_ERR_BAD_SHAPE;  // no denormals
    if (D > kMaxNormWidth || !known_dtype(dtype)) return GDN_ERR_UNSUPPORTED;
    n = bytes_of(rows, D, dtype == GDN_BF16 ? 2 : 4);
    return n < 0 ? GDN_ERR_BAD_SHAPE : GDN_OK;
}

static inline gdn_status_t check_norm(const void *x, const void *res, const void *w,
                                      const void *res_out, const void *out, const void *out8,
                                      const float *scales, int32_t group, int64_t rows,
                                      int32_t D, gdn_dtype_t dtype, float eps) {
    int64_t n;
    const gdn_status_t st = check_norm_shape(rows, D, dtype, eps, n);
    if (st != GDN_OK) return st;
    if (group != 0 && group != 128) return GDN_ERR_UNSUPPORTED;
    if (rows > 0) {
        if (!x || !w || (!out && !out8)) return GDN_ERR_NULL_POINTER;
        if ((out8 != nullptr) != (scales != nullptr)) return GDN_ERR_NULL_POINTER;
        if (res_out && !res) return GDN_ERR_NULL_POINTER;
    }
    const void *ptrs[] = {x, res, w, res_out, out, out8, scales};
    if (!all_aligned(ptrs, 16)) return GDN_ERR_MISALIGNED;
    // residual_out may be residual or x itself: each element is read before it
    // is written, by the same thread
    const int64_t es = dtype == GDN_BF16 ? 2 : 4;
    const Range rx = range_of(x, n), rr = range_of(res, n), rw = range_of(w, D * es);
    const Range in[] = {rx, rr, rw};
    const Range ro[] = {range_of(out, n), range_of(out8, rows * D),
                        range_of(scales, rows * norm_groups(D, group) * 4)};
    if (any_overlap(in, ro)) return GDN_ERR_ALIAS;
    const Range in2[] = {range_of(x, res_out == x ? 0 : n),
                         range_of(res, res_out == res ? 0 : n), rw, ro[0], ro[1], ro[2]};
    const Range ro2[] = {range_of(res_out, n)};
    return any_overlap(in2, ro2) ? GDN_ERR_ALIAS : GDN_OK;
}

static inline gdn_status_t check_norm_backward(const void *dout, const void *r, const void *w,
                                               const void *dres, const void *dx,
                                               const float *dw, int64_t rows, int32_t D,
                                               gdn_dtype_t dtype, float eps, const void *ws,
                                               size_t ws_bytes, size_t ws_needed) {
    int64_t n;
    const gdn_status_t st = check_norm_shape(rows, D, dtype, eps, n);
    if (st != GDN_OK) return st;
    if (rows > 0 && (!dout || !r || !w || !dx)) return GDN_ERR_NULL_POINTER;
    if (ws_bytes > (size_t)INT64_MAX) return GDN_ERR_BAD_SHAPE;
    if (dw && rows > 0) {
        if (!ws) return GDN_ERR_NULL_POINTER;
        if (ws_bytes < ws_needed) return GDN_ERR_BAD_SHAPE;
    }
    const void *ptrs[] = {dout, r, w, dres, dx, dw, ws};
    if (!all_aligned(ptrs, 16)) return GDN_ERR_MISALIGNED;
    const int64_t es = dtype == GDN_BF16 ? 2 : 4;
    // dx may be dresidual itself
    const Range in[] = {range_of(dout, n), range_of(r, n), range_of(w, D * es),
                        range_of(dres, dres == dx ? 0 : n)};
    const Range ro[] = {range_of(dx, n), range_of(dw, (int64_t)D * 4),
                        range_of(ws, (int64_t)ws_bytes)};
    return any_overlap(in, ro) ? GDN_ERR_ALIAS : GDN_OK;
}

static inline gdn_status_t check_beam_shape(int32_t B, int32_t W, int64_t V,
                                            gdn_dtype_t dtype) {
    if (B < 1 || W < 1 || V < 1) return GDN_ERR_BAD_SHAPE;
    if (W > kMaxBeams || !known_dtype(dtype)) return GDN_ERR_UNSUPPORTED;
    const int64_t rows = (int64_t)B * W;
    if (V > 0x7FFFFFFF || rows > ((int64_t)1 << 40) / V) return GDN_ERR_BAD_SHAPE;
    if (rows * (V / 8192 + 2) > kMaxGrid) return GDN_ERR_BAD_SHAPE;  // workgroups
    return GDN_OK;
}

static inline gdn_status_t check_beam(const void *logits, const float *scores,
                                      const uint8_t *fin, const int32_t *slots,
                                      const float *new_scores, const int32_t *tokens,
                                      const int32_t *parents, const uint8_t *new_fin,
                                      const int32_t *src_slots, int32_t B, int32_t W, int64_t V,
                                      int32_t eos, gdn_dtype_t dtype, const void *ws,
                                      size_t ws_bytes, size_t ws_needed) {
    const gdn_status_t st = check_beam_shape(B, W, V, dtype);
    if (st != GDN_OK) return st;
    if (eos < -1 || eos >= V) return GDN_ERR_BAD_SHAPE;
    if (eos < 0 && (fin || new_fin)) return GDN_ERR_BAD_SHAPE;
    if (!logits || !scores || !new_scores || !tokens || !parents || !ws)
        return GDN_ERR_NULL_POINTER;
    if ((slots != nullptr) != (src_slots != nullptr)) return GDN_ERR_NULL_POINTER;
    if (ws_bytes > (size_t)INT64_MAX || ws_bytes < ws_needed) return GDN_ERR_BAD_SHAPE;
    const void *big[] = {logits, ws};
    if (!all_aligned(big, 16)) return GDN_ERR_MISALIGNED;
    const void *small[] = {scores, slots, new_scores, tokens, parents, src_slots};
    if (!all_aligned(small, 4)) return GDN_ERR_MISALIGNED;
    const int64_t bw = (int64_t)B * W, es = dtype == GDN_BF16 ? 2 : 4;
    const Range in[] = {range_of(logits, bw * V * es), range_of(scores, bw * 4),
                        range_of(fin, bw), range_of(slots, bw * 4)};
    const Range ro[] = {range_of(new_scores, bw * 4), range_of(tokens, bw * 4),
                        range_of(parents, bw * 4),    range_of(new_fin, bw),
                        range_of(src_slots, bw * 4),  range_of(ws, (int64_t)ws_bytes)};
    return any_overlap(in, ro) ? GDN_ERR_ALIAS : GDN_OK;
}

static inline gdn_status_t check_gather(const void *src, int64_t num_src, const int32_t *index,
                                        const void *dst, int64_t rows, int64_t row_bytes) {
    if (num_src < 0 || num_src > 0x7FFFFFFF || rows < 0 || row_bytes < 0)
        return GDN_ERR_BAD_SHAPE;
    if (row_bytes % 16 != 0) return GDN_ERR_UNSUPPORTED;
    const int64_t ns = bytes_of(num_src, row_bytes, 1), nd = bytes_of(rows, row_bytes, 1);
    const int64_t ni = bytes_of(rows, 4, 1);
    if (ns < 0 || nd < 0 || ni < 0) return GDN_ERR_BAD_SHAPE;
    // workgroups copy at least 16 KiB of a row each
    int64_t wgs = rows;
    if (!mul_ok(wgs, (row_bytes + 16383) / 16384) || wgs > kMaxGrid) return GDN_ERR_BAD_SHAPE;
    if (nd > 0 && (!index || !dst || (num_src > 0 && !src))) return GDN_ERR_NULL_POINTER;
    const void *big[] = {src, dst};
    if (!all_aligned(big, 16)) return GDN_ERR_MISALIGNED;
    const void *small[] = {index};
    if (!all_aligned(small, 4)) return GDN_ERR_MISALIGNED;
    const Range in[] = {range_of(src, ns), range_of(index, ni)};
    const Range ro[] = {range_of(dst, nd)};
    return any_overlap(in, ro) ? GDN_ERR_ALIAS : GDN_OK;
}

}  // namespace val
}  // namespace gdn
