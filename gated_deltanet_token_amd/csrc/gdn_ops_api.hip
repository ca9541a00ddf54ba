// gdn_ops_api.hip -- the C ABI of the scan, norm and beam calls (include/gdn.h):
// argument validation and launch, as in gdn_api.hip.
#include "gdn_ops_launch.hpp"
#include "gdn_ops_validate.hpp"

namespace {

using namespace gdn::val;

int code(gdn_dtype_t dtype) { return dtype == GDN_BF16 ? 1 : 0; }

// Rows of the prefix states: B * floor(T / L), or floor(total / L) + N packed.
int64_t prefix_rows(bool packed, int64_t n, int64_t tokens, int32_t interval) {
    const int64_t L = 64 * (int64_t)(interval < 1 ? 1 : interval);
    return packed ? tokens / L + n : n * (tokens / L);
}

// The scan calls' arguments as both the checks and the kernels want them.
// tokens: T (dense) or total_T (packed). False: B * T overflows.
bool scan_args(ScanArgs &s, gdn::ScanParams &p, const void *x, const void *a, const void *b,
               const float *h0, const int32_t *cu, bool packed, int32_t n, int64_t tokens,
               int32_t D, gdn_dtype_t dtype, uint32_t flags, const float *prefix,
               int32_t interval, const void *ws, size_t ws_bytes) {
    int64_t total = packed ? tokens : (n < 0 ? 0 : n);
    if (tokens < 0 || n < 1 || (!packed && !mul_ok(total, tokens))) return false;
    if (packed && tokens > 0x7FFFFFFF) return false;
    s = ScanArgs{x, a, b, h0, cu, packed ? (int64_t)n + 1 : 0, total, n, tokens, D, dtype, flags,
                 prefix, interval, prefix_rows(packed, n, tokens, interval), ws, ws_bytes};
    p = gdn::ScanParams{};
    p.x = x;
    p.a = a;
    p.b = b;
    p.h0 = h0;
    p.prefix_len = 64 * (int64_t)(interval < 1 ? 1 : interval);
    p.cu = packed ? cu : nullptr;
    p.T = packed ? 0 : tokens;
    p.total = total;
    p.N = n;
    p.D = D;
    p.flags = flags;
    return true;
}

gdn_status_t scan_forward(const void *x, const void *a, const void *b, const int32_t *cu,
                          bool packed, int32_t n, int64_t tokens, const float *h0, void *out,
                          float *hT, float *prefix, int32_t interval, int32_t D,
                          gdn_dtype_t dtype, uint32_t flags, void *ws, size_t ws_bytes,
                          hipStream_t stream, const char *where) {
    ScanArgs s;
    gdn::ScanParams p;
    if (!scan_args(s, p, x, a, b, h0, cu, packed, n, tokens, D, dtype, flags, prefix, interval,
                   ws, ws_bytes))
        return GDN_ERR_BAD_SHAPE;
    gdn_status_t st = check_scan(s, out, hT);
    if (st != GDN_OK) return st;
    if (s.tokens == 0 && !hT) return GDN_OK;
    if (packed && gdn::debug_checks(stream) &&
        (st = gdn::debug_cu_seqlens(cu, n, tokens, stream)) != GDN_OK)
        return st;
    int cus = 0;
    if ((st = gdn::device_cus(&cus)) != GDN_OK) return st;
    p.out = out;
    p.hT = hT;
    p.prefix_out = s.prefix_rows > 0 ? prefix : nullptr;
    const hipError_t e = gdn::launch_scan(p, code(dtype), cus, ws, ws_bytes, stream);
    return e == hipSuccess ? GDN_OK : gdn::hip_fail(e, where);
}

gdn_status_t scan_backward(const void *dout, const void *x, const void *a, const void *b,
                           const int32_t *cu, bool packed, int32_t n, int64_t tokens,
                           const float *h0, const float *prefix, int32_t interval,
                           const float *dhT, void *dx, void *da, void *db, float *dh0, int32_t D,
                           gdn_dtype_t dtype, uint32_t flags, void *ws, size_t ws_bytes,
                           hipStream_t stream, const char *where) {
    ScanArgs s;
    gdn::ScanParams p;
    if (!scan_args(s, p, x, a, b, h0, cu, packed, n, tokens, D, dtype, flags, prefix, interval,
                   ws, ws_bytes))
        return GDN_ERR_BAD_SHAPE;
    gdn_status_t st = check_scan_backward(s, dout, dhT, dx, da, db, dh0);
    if (st != GDN_OK) return st;
    if (s.tokens == 0 && !dh0) return GDN_OK;
    if (packed && gdn::debug_checks(stream) &&
        (st = gdn::debug_cu_seqlens(cu, n, tokens, stream)) != GDN_OK)
        return st;
    int cus = 0;
    if ((st = gdn::device_cus(&cus)) != GDN_OK) return st;
    p.prefix_in = s.prefix_rows > 0 ? prefix : nullptr;
    p.dout = dout;
    p.dhT = dhT;
    p.dx = dx;
    p.da = da;
    p.db = db;
    p.dh0 = dh0;
    const hipError_t e = gdn::launch_scan_backward(p, code(dtype), cus, ws, ws_bytes, stream);
    return e == hipSuccess ? GDN_OK : gdn::hip_fail(e, where);
}

}  // namespace

extern "C" {

gdn_status_t gdn_scan_prefill(const void *x, const void *alpha, const void *beta,
                              const float *initial_state, void *out, float *final_state,
                              float *prefix_states, int32_t prefix_interval, int32_t B,
                              int64_t T, int32_t D, gdn_dtype_t dtype, uint32_t flags,
                              void *workspace, size_t workspace_bytes, hipStream_t stream) {
    return scan_forward(x, alpha, beta, nullptr, false, B, T, initial_state, out, final_state,
                        prefix_states, prefix_interval, D, dtype, flags, workspace,
                        workspace_bytes, stream, "gdn_scan_prefill launch");
}

gdn_status_t gdn_scan_varlen_prefill(const void *x, const void *alpha, const void *beta,
                                     const int32_t *cu_seqlens, int32_t N, int64_t total_T,
                                     const float *initial_state, void *out, float *final_state,
                                     float *prefix_states, int32_t prefix_interval, int32_t D,
                                     gdn_dtype_t dtype, uint32_t flags, void *workspace,
                                     size_t workspace_bytes, hipStream_t stream) {
    return scan_forward(x, alpha, beta, cu_seqlens, true, N, total_T, initial_state, out,
                        final_state, prefix_states, prefix_interval, D, dtype, flags, workspace,
                        workspace_bytes, stream, "gdn_scan_varlen_prefill launch");
}

gdn_status_t gdn_scan_backward(const void *dout, const void *x, const void *alpha,
                               const void *beta, const float *initial_state,
                               const float *prefix_states, int32_t prefix_interval,
                               const float *dfinal, void *dx, void *dalpha, void *dbeta,
                               float *dinitial, int32_t B, int64_t T, int32_t D,
                               gdn_dtype_t dtype, uint32_t flags, void *workspace,
                               size_t workspace_bytes, hipStream_t stream) {
    return scan_backward(dout, x, alpha, beta, nullptr, false, B, T, initial_state,
                         prefix_states, prefix_interval, dfinal, dx, dalpha, dbeta, dinitial, D,
                         dtype, flags, workspace, workspace_bytes, stream,
                         "gdn_scan_backward launch");
}

gdn_status_t gdn_scan_varlen_backward(const void *dout, const void *x, const void *alpha,
                                      const void *beta, const int32_t *cu_seqlens, int32_t N,
                                      int64_t total_T, const float *initial_state,
                                      const float *prefix_states, int32_t prefix_interval,
                                      const float *dfinal, void *dx, void *dalpha, void *dbeta,
                                      float *dinitial, int32_t D, gdn_dtype_t dtype,
                                      uint32_t flags, void *workspace, size_t workspace_bytes,
                                      hipStream_t stream) {
    return scan_backward(dout, x, alpha, beta, cu_seqlens, true, N, total_T, initial_state,
                         prefix_states, prefix_interval, dfinal, dx, dalpha, dbeta, dinitial, D,
                         dtype, flags, workspace, workspace_bytes, stream,
                         "gdn_scan_varlen_backward launch");
}

gdn_status_t gdn_scan_decode(const void *x, const void *alpha, const void *beta,
                             float *state_pool, int32_t num_slots, const int32_t *src_slot,
                             const int32_t *dst_slot, void *out, int32_t B, int32_t K,
                             int32_t D, gdn_dtype_t dtype, uint32_t flags, hipStream_t stream) {
    const gdn_status_t st = check_scan_decode(x, alpha, beta, state_pool, num_slots, src_slot,
                                              dst_slot, out, B, K, D, dtype, flags);
    if (st != GDN_OK) return st;
    gdn::ScanDecodeParams p{x, alpha, beta, state_pool, src_slot, dst_slot, out, num_slots,
                            B, K, D, flags};
    const hipError_t e = gdn::launch_scan_decode(p, code(dtype), stream);
    return e == hipSuccess ? GDN_OK : gdn::hip_fail(e, "gdn_scan_decode launch");
}

size_t gdn_scan_workspace_size(int32_t num_seqs, int64_t tokens, int32_t D, gdn_dtype_t dtype,
                               int32_t packed) {
    if (num_seqs < 1 || tokens < 1 || D < 1 || !known_dtype(dtype)) return 0;
    if (packed && tokens > 0x7FFFFFFF) return 0;
    int64_t total = packed ? tokens : num_seqs;
    if (!packed && !mul_ok(total, tokens)) return 0;
    if (D > kMaxScanWidth || bytes_of(total, D, 4) < 0 || !scan_fits(total, num_seqs, D)) return 0;
    int cus = 0;
    if (gdn::device_cus(&cus) != GDN_OK) return 0;
    return gdn::scan_workspace_bytes(num_seqs, tokens, D, code(dtype), packed != 0, cus);
}

gdn_status_t gdn_rms_norm(const void *x, const void *residual, const void *weight,
                          void *residual_out, void *out, void *out8, float *scales,
                          int32_t group, int64_t rows, int32_t D, gdn_dtype_t dtype, float eps,
                          hipStream_t stream) {
    const gdn_status_t st = check_norm(x, residual, weight, residual_out, out, out8, scales,
                                       group, rows, D, dtype, eps);
    if (st != GDN_OK || rows == 0) return st;
    gdn::NormParams p{x, residual, weight, residual_out, out, static_cast<uint8_t *>(out8),
                      scales, group, rows, D, eps, 1.f / (float)D};
    const hipError_t e = gdn::launch_norm(p, code(dtype), stream);
    return e == hipSuccess ? GDN_OK : gdn::hip_fail(e, "gdn_rms_norm launch");
}

size_t gdn_rms_norm_workspace_size(int64_t rows, int32_t D) {
    if (rows < 1 || rows > kMaxGrid || D < 1 || D > kMaxNormWidth) return 0;
    return (size_t)gdn::norm_partials(rows, D) * gdn::norm_partial_width(D) * 4;
}

gdn_status_t gdn_rms_norm_backward(const void *dout, const void *r, const void *weight,
                                   const void *dresidual, void *dx, float *dweight,
                                   int64_t rows, int32_t D, gdn_dtype_t dtype, float eps,
                                   void *workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
    const gdn_status_t st =
        check_norm_backward(dout, r, weight, dresidual, dx, dweight, rows, D, dtype, eps,
                            workspace, workspace_bytes, gdn_rms_norm_workspace_size(rows, D));
    if (st != GDN_OK || (rows == 0 && !dweight)) return st;
    gdn::NormBackwardParams p{dout, r, weight, dresidual, dx, dweight,
                              static_cast<float *>(workspace), rows, D, eps, 1.f / (float)D};
    const hipError_t e = gdn::launch_norm_backward(p, code(dtype), stream);
    return e == hipSuccess ? GDN_OK : gdn::hip_fail(e, "gdn_rms_norm_backward launch");
}

size_t gdn_beam_workspace_size(int32_t B, int32_t W, int64_t V, gdn_dtype_t dtype) {
    if (check_beam_shape(B, W, V, dtype) != GDN_OK) return 0;
    return gdn::beam_workspace_bytes(B, W, V, code(dtype));
}

gdn_status_t gdn_beam_select(const void *logits, const float *scores, const uint8_t *finished,
                             const int32_t *beam_slots, float *new_scores, int32_t *tokens,
                             int32_t *parents, uint8_t *new_finished, int32_t *src_slots,
                             int32_t B, int32_t W, int64_t V, int32_t eos, gdn_dtype_t dtype,
                             void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const gdn_status_t st =
        check_beam(logits, scores, finished, beam_slots, new_scores, tokens, parents,
                   new_finished, src_slots, B, W, V, eos, dtype, workspace, workspace_bytes,
                   gdn_beam_workspace_size(B, W, V, dtype));
    if (st != GDN_OK) return st;
    gdn::BeamParams p{logits, scores, finished, beam_slots, new_scores, tokens, parents,
                      new_finished, src_slots, B, W, V, eos};
    const hipError_t e = gdn::launch_beam(p, code(dtype), workspace, stream);
    return e == hipSuccess ? GDN_OK : gdn::hip_fail(e, "gdn_beam_select launch");
}

gdn_status_t gdn_gather_states(const void *src, int64_t num_src, const int32_t *index, void *dst,
                               int64_t rows, int64_t row_bytes, hipStream_t stream) {
    const gdn_status_t st = check_gather(src, num_src, index, dst, rows, row_bytes);
    if (st != GDN_OK) return st;
    const hipError_t e = gdn::launch_gather(src, num_src, index, dst, rows, row_bytes, stream);
    return e == hipSuccess ? GDN_OK : gdn::hip_fail(e, "gdn_gather_states launch");
}

}  // extern "C"
