// gdn_attn_api.hip -- the C ABI of the attention, cache and rotary calls
// (include/gdn.h): argument validation and launch, as in gdn_api.hip.
#include "gdn_attn_launch.hpp"
#include "gdn_attn_validate.hpp"

namespace {

using namespace gdn::val;

int code(gdn_dtype_t dtype) { return dtype == GDN_BF16 ? 1 : 0; }

int log2_of(int32_t x) {  // a power of two
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

// Tokens in all; false: they overflow. tokens: T (dense) or total_T (packed).
bool prompt_args(PromptArgs &a, const void *q, const void *k, const void *v, const int32_t *cu,
                 bool packed, int32_t n, int64_t tokens, int32_t Hq, int32_t Hk, int32_t D,
                 gdn_dtype_t dtype, float scale) {
    int64_t total = packed ? tokens : (n < 0 ? 0 : n);
    if (tokens < 0 || n < 1 || (!packed && !mul_ok(total, tokens))) return false;
    a = PromptArgs{q, k, v, cu, packed ? (int64_t)n + 1 : 0, n, total, tokens, Hq, Hk, D, dtype,
                   scale};
    return true;
}

gdn_status_t attn_forward(const PromptArgs &a, void *out, float *lse, hipStream_t stream,
                          const char *where) {
    gdn_status_t st = check_prompt(a, out, lse);
    if (st != GDN_OK || a.tokens == 0) return st;
    const bool packed = a.cu_count > 0;
    if (packed && gdn::debug_checks(stream) &&
        (st = gdn::debug_cu_seqlens(a.cu, (int32_t)a.n, a.tokens, stream)) != GDN_OK)
        return st;
    int cus = 0;
    if ((st = gdn::device_cus(&cus)) != GDN_OK) return st;
    const gdn::AttnParams p{a.q, a.k, a.v, out, lse, packed ? a.cu : nullptr,
                            packed ? 0 : a.longest, a.tokens, (int32_t)a.n, a.Hq, a.Hk, a.scale};
    const hipError_t e = gdn::launch_attn(p, code(a.dtype), a.D, cus, stream);
    return e == hipSuccess ? GDN_OK : gdn::hip_fail(e, where);
}

size_t stats_bytes(const PromptArgs &a) {
    return ((size_t)3 * a.Hq * a.tokens * 4 + 255) / 256 * 256;
}
int32_t head_split(const PromptArgs &a, int cus) {
    return gdn::attn_backward_split(a.n, a.longest, a.tokens, a.Hq, a.Hk, a.D, code(a.dtype),
                                    a.cu_count > 0, cus);
}
size_t backward_bytes(const PromptArgs &a, int cus) {
    const int32_t split = head_split(a, cus);
    return stats_bytes(a) + (split > 1 ? (size_t)split * 2 * a.tokens * a.Hk * a.D * 4 : 0);
}

gdn_status_t attn_backward(const PromptArgs &a, const void *dout, const void *out,
                           const float *lse, void *dq, void *dk, void *dv, void *ws,
                           size_t ws_bytes, hipStream_t stream, const char *where) {
    // the arguments apart from the workspace's size, which needs the device
    gdn_status_t st = check_prompt_backward(a, dout, out, lse, dq, dk, dv, ws, ws_bytes, 0);
    if (st != GDN_OK || a.tokens == 0) return st;
    const bool packed = a.cu_count > 0;
    int cus = 0;
    if ((st = gdn::device_cus(&cus)) != GDN_OK) return st;
    st = check_prompt_backward(a, dout, out, lse, dq, dk, dv, ws, ws_bytes, backward_bytes(a, cus));
    if (st != GDN_OK) return st;
    if (packed && gdn::debug_checks(stream) &&
        (st = gdn::debug_cu_seqlens(a.cu, (int32_t)a.n, a.tokens, stream)) != GDN_OK)
        return st;
    unsigned char *w = static_cast<unsigned char *>(ws);
    const gdn::AttnBackwardParams p{dout, a.q, a.k, a.v, out, lse, dq, dk, dv,
                                    packed ? a.cu : nullptr, packed ? 0 : a.longest, a.tokens,
                                    (int32_t)a.n, a.Hq, a.Hk, a.scale,
                                    reinterpret_cast<float *>(w),
                                    reinterpret_cast<float *>(w + stats_bytes(a)),
                                    head_split(a, cus)};
    const hipError_t e = gdn::launch_attn_backward(p, code(a.dtype), a.D, cus, stream);
    return e == hipSuccess ? GDN_OK : gdn::hip_fail(e, where);
}

gdn::AttnDecodeParams decode_params(const DecodeArgs &a, void *out, float *lse) {
    return gdn::AttnDecodeParams{a.q, a.kc, a.vc, a.table, a.lengths, a.ptable, a.plengths,
                                 a.pgroups, out, lse, a.B, a.K, a.Hq, a.Hk, a.G, a.num_pages,
                                 log2_of(a.page_size), a.max_pages, a.max_ppages, a.scale};
}

}  // namespace

extern "C" {

gdn_status_t gdn_attn_prefill(const void *q, const void *k, const void *v, void *out, float *lse,
                              int32_t B, int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                              gdn_dtype_t dtype, float scale, hipStream_t stream) {
    PromptArgs a;
    if (!prompt_args(a, q, k, v, nullptr, false, B, T, Hq, Hk, D, dtype, scale))
        return GDN_ERR_BAD_SHAPE;
    return attn_forward(a, out, lse, stream, "gdn_attn_prefill launch");
}

gdn_status_t gdn_attn_varlen_prefill(const void *q, const void *k, const void *v,
                                     const int32_t *cu_seqlens, int32_t N, int64_t total_T,
                                     void *out, float *lse, int32_t Hq, int32_t Hk, int32_t D,
                                     gdn_dtype_t dtype, float scale, hipStream_t stream) {
    PromptArgs a;
    if (!prompt_args(a, q, k, v, cu_seqlens, true, N, total_T, Hq, Hk, D, dtype, scale))
        return GDN_ERR_BAD_SHAPE;
    return attn_forward(a, out, lse, stream, "gdn_attn_varlen_prefill launch");
}

gdn_status_t gdn_attn_backward(const void *dout, const void *q, const void *k, const void *v,
                               const void *out, const float *lse, void *dq, void *dk, void *dv,
                               int32_t B, int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                               gdn_dtype_t dtype, float scale, void *workspace,
                               size_t workspace_bytes, hipStream_t stream) {
    PromptArgs a;
    if (!prompt_args(a, q, k, v, nullptr, false, B, T, Hq, Hk, D, dtype, scale))
        return GDN_ERR_BAD_SHAPE;
    return attn_backward(a, dout, out, lse, dq, dk, dv, workspace, workspace_bytes, stream,
                         "gdn_attn_backward launch");
}

gdn_status_t gdn_attn_varlen_backward(const void *dout, const void *q, const void *k,
                                      const void *v, const void *out, const float *lse,
                                      const int32_t *cu_seqlens, int32_t N, int64_t total_T,
                                      void *dq, void *dk, void *dv, int32_t Hq, int32_t Hk,
                                      int32_t D, gdn_dtype_t dtype, float scale, void *workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
    PromptArgs a;
    if (!prompt_args(a, q, k, v, cu_seqlens, true, N, total_T, Hq, Hk, D, dtype, scale))
        return GDN_ERR_BAD_SHAPE;
    return attn_backward(a, dout, out, lse, dq, dk, dv, workspace, workspace_bytes, stream,
                         "gdn_attn_varlen_backward launch");
}

size_t gdn_attn_backward_workspace_size(int32_t num_seqs, int64_t tokens, int32_t Hq, int32_t Hk,
                                        int32_t D, gdn_dtype_t dtype, int32_t packed) {
    PromptArgs a;
    static const int32_t none = 0;
    int64_t nq, nk, nl;
    if (!prompt_args(a, &none, &none, &none, packed ? &none : nullptr, packed != 0, num_seqs,
                     tokens, Hq, Hk, D, dtype, 1.f) ||
        check_prompt_common(a, nq, nk, nl) != GDN_OK || a.tokens == 0)
        return 0;
    int cus = 0;
    if (gdn::device_cus(&cus) != GDN_OK) return 0;
    return backward_bytes(a, cus);
}

gdn_status_t gdn_attn_decode(const void *q, const void *k_cache, const void *v_cache,
                             int32_t num_pages, int32_t page_size, const int32_t *page_table,
                             int32_t max_pages, const int32_t *lengths,
                             const int32_t *prefix_table, int32_t max_prefix_pages,
                             const int32_t *prefix_lengths, const int32_t *prefix_groups,
                             int32_t G, void *out, float *lse, int32_t B, int32_t K, int32_t Hq,
                             int32_t Hk, int32_t D, gdn_dtype_t dtype, float scale,
                             void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const DecodeArgs a{q, k_cache, v_cache, num_pages, page_size, max_pages,
                       prefix_table ? max_prefix_pages : 0, prefix_table ? G : 0, page_table,
                       lengths, prefix_table, prefix_lengths, prefix_groups, out, lse, B, K, Hq,
                       Hk, D, dtype, scale};
    gdn_status_t st = check_decode(a, workspace, workspace_bytes, 0);
    if (st != GDN_OK) return st;
    int cus = 0;
    if ((st = gdn::device_cus(&cus)) != GDN_OK) return st;
    const gdn::AttnDecodeParams p = decode_params(a, out, lse);
    const size_t need = gdn::attn_decode_workspace_bytes(p, code(dtype), D, cus);
    if ((st = check_decode(a, workspace, workspace_bytes, need)) != GDN_OK) return st;
    if (prefix_groups && gdn::debug_checks(stream) &&
        (st = gdn::debug_cu_seqlens(prefix_groups, G, B, stream)) != GDN_OK)
        return st;
    const hipError_t e = gdn::launch_attn_decode(p, code(dtype), D, cus, workspace, stream);
    return e == hipSuccess ? GDN_OK : gdn::hip_fail(e, "gdn_attn_decode launch");
}

size_t gdn_attn_decode_workspace_size(int32_t B, int32_t K, int32_t Hq, int32_t Hk, int32_t D,
                                      int32_t page_size, int32_t max_pages, int32_t G,
                                      int32_t max_prefix_pages, gdn_dtype_t dtype) {
    static const int32_t none = 0;
    DecodeArgs a{};
    a.num_pages = 1;
    a.page_size = page_size;
    a.max_pages = max_pages;
    a.max_ppages = max_prefix_pages;
    a.G = G;
    a.ptable = G != 0 ? &none : nullptr;
    a.B = B;
    a.K = K;
    a.Hq = Hq;
    a.Hk = Hk;
    a.D = D;
    a.dtype = dtype;
    a.scale = 1.f;
    if (check_decode_shape(a, G != 0) != GDN_OK) return 0;
    int cus = 0;
    if (gdn::device_cus(&cus) != GDN_OK) return 0;
    return gdn::attn_decode_workspace_bytes(decode_params(a, nullptr, nullptr), code(dtype), D,
                                            cus);
}

gdn_status_t gdn_rotary(const void *q, const void *k, void *q_out, void *k_out,
                        const int32_t *positions, int32_t axes, const float *inv_freq,
                        const int32_t *pair_axis, int32_t R, int64_t tokens, int32_t Hq,
                        int32_t Hk, int32_t D, gdn_dtype_t dtype, uint32_t flags,
                        hipStream_t stream) {
    const RotaryArgs a{q, k, q_out, k_out, positions, inv_freq, pair_axis, axes, R, tokens, Hq,
                       k ? Hk : 0, D, dtype, flags};
    const gdn_status_t st = check_rotary(a);
    if (st != GDN_OK || tokens == 0) return st;
    gdn::RotaryParams p{};
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    p.freq = inv_freq;
    p.pos = positions;
    p.axis = pair_axis;
    p.tokens = tokens;
    p.T = tokens;
    p.N = 1;
    p.Hq = Hq;
    p.Hk = Hk;
    p.D = D;
    p.R = R;
    p.axes = axes;
    p.pairs = (flags & GDN_ROPE_PAIRS) != 0;
    p.inverse = (flags & GDN_ROPE_INVERSE) != 0;
    const hipError_t e = gdn::launch_rotary(p, code(dtype), stream);
    return e == hipSuccess ? GDN_OK : gdn::hip_fail(e, "gdn_rotary launch");
}

gdn_status_t gdn_kv_append(const void *k, const void *v, void *k_cache, void *v_cache,
                           int32_t num_pages, int32_t page_size, const int32_t *page_table,
                           int32_t max_pages, const int32_t *lengths, const int32_t *cu_seqlens,
                           const void *q, void *q_out, void *k_out, const float *inv_freq,
                           int32_t R, const int32_t *positions, int32_t axes,
                           const int32_t *pair_axis, int32_t N, int64_t tokens, int32_t Hq,
                           int32_t Hk, int32_t D, gdn_dtype_t dtype, uint32_t flags,
                           hipStream_t stream) {
    int64_t total = cu_seqlens ? tokens : (N < 0 ? 0 : N);
    if (tokens < 0 || (!cu_seqlens && !mul_ok(total, tokens))) return GDN_ERR_BAD_SHAPE;
    const AppendArgs a{RotaryArgs{q, k, q_out, k_out, positions, inv_freq, pair_axis, axes,
                                  inv_freq ? R : 0, total, q ? Hq : 0, Hk, D, dtype, flags},
                       v, k_cache, v_cache, num_pages, page_size, max_pages, page_table, lengths,
                       cu_seqlens, N, tokens};
    gdn_status_t st = check_append(a);
    if (st != GDN_OK || total == 0) return st;
    if (inv_freq && R < 2) return GDN_ERR_BAD_SHAPE;
    if (cu_seqlens && gdn::debug_checks(stream) &&
        (st = gdn::debug_cu_seqlens(cu_seqlens, N, total, stream)) != GDN_OK)
        return st;
    const gdn::RotaryParams p{q, k, v, q_out, k_out, k_cache, v_cache, inv_freq, positions,
                              pair_axis, cu_seqlens, lengths, page_table, total, tokens, N,
                              q ? Hq : 0, Hk, D, a.r.R, axes, num_pages, log2_of(page_size),
                              max_pages, (flags & GDN_ROPE_PAIRS) != 0,
                              (flags & GDN_ROPE_INVERSE) != 0};
    const hipError_t e = gdn::launch_rotary(p, code(dtype), stream);
    return e == hipSuccess ? GDN_OK : gdn::hip_fail(e, "gdn_kv_append launch");
}

}  // extern "C"
