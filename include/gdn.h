/*
 * gdn.h -- C ABI of the MI355X (gfx950) Gated DeltaNet token mixer.
 *
 * The layer: the Gated DeltaNet blocks that fill 48 of the 64 layers of the
 * hybrid stack in "The Hybrid Attention in Qwen3.8-27B" (section "Why 27B
 * parameters can carry 262K tokens": layout 16 x (3 x (Gated DeltaNet ->
 * FFN) -> 1 x (Gated Attention -> FFN)); section "Grouped-query attention
 * multiplies on top of that": 16 query/key heads, 48 value heads, head
 * dimension 128). Each value head keeps one fixed-size state whatever the
 * context length ("The economics of hybrid attention", TL;DR: the 48 blocks
 * hold a fixed ~150 MiB, i.e. 48 x 48 x 128 x 128 fp32).
 *
 * The pages name the layer but do not print its recurrence; this library
 * computes the published gated delta rule, for each sequence and value head
 * h (S in R^{Dv x Dk}, row-major; q/k head g = h / (Hv / Hk)):
 *
 *     S_t = alpha_t * S_{t-1} * (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *     o_t = scale * S_t q_t
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All tensor pointers are DEVICE pointers, contiguous, in the layouts
 *    stated per call, and 16-byte aligned. q, k, v and out have the element
 *    type `dtype` (GDN_BF16 or GDN_F32); alpha, beta and states are fp32.
 *  - Ownership: the caller owns every buffer. The library allocates and
 *    frees no memory, creates no stream or event, keeps no pointer after the
 *    call returns and holds no mutable global state; calls are re-entrant
 *    and thread-safe (two calls that share a workspace must not overlap in
 *    time on the device, like any two users of one buffer).
 *  - Asynchrony: each call validates its arguments on the host, enqueues
 *    kernels on `stream` and returns without synchronising. Results are
 *    ready when the stream reaches that point.
 *  - Validation happens before any HIP call; a call that fails validation
 *    has no side effects. GDN_ERR_HIP reports a failure of the HIP runtime
 *    (no device, launch error); gdn_status_string() then gives the detail
 *    for the calling thread.
 *  - Values are not validated: NaN or Inf inputs propagate. alpha and beta
 *    are meant to lie in [0, 1]; alpha is clamped to >= FLT_MIN before its
 *    logarithm is taken.
 *  - Debug checks: with GDN_DEBUG=1 in the environment, the prefill calls
 *    also run synchronous checks (they synchronise `stream`, and are skipped
 *    while the stream is being captured into a graph): the contents of
 *    cu_seqlens (GDN_ERR_BAD_SHAPE before any launch when malformed), and,
 *    after a call that used a workspace, its status word (GDN_ERR_HIP when a
 *    kernel's bounded wait for another wave of its workgroup ran out, which
 *    a correct run never does).
 *  - `out` must not overlap any input. `final_state` must either be the same
 *    pointer as `initial_state` (in-place update) or not overlap it, and it
 *    must not overlap any other argument.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GDN_OK = 0,
    GDN_ERR_NULL_POINTER = 1, /* a required pointer is NULL */
    GDN_ERR_BAD_SHAPE = 2,    /* a size is out of range or inconsistent */
    GDN_ERR_UNSUPPORTED = 3,  /* a valid shape the library has no kernel for */
    GDN_ERR_MISALIGNED = 4,   /* a pointer is not 16-byte aligned */
    GDN_ERR_ALIAS = 5,        /* forbidden overlap between buffers */
    GDN_ERR_HIP = 6           /* HIP runtime error; see gdn_status_string */
} gdn_status_t;

typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype_t; /* type of q, k, v, out */

/*
 * Input preparation done inside the kernels: the `flags` argument of the
 * compute calls (bitwise OR; 0 = inputs used as given). The pages name the
 * layer but not these steps; they are the ones just before the recurrence in
 * the published Gated DeltaNet (Yang, Kautz & Hatamizadeh, ICLR 2025): q and k
 * L2-normalised per head, the write strength a sigmoid and the decay the
 * exponential of a negative softplus of per-token projections.
 *   GDN_QK_L2NORM    q and k hold raw rows; each row x is used as
 *                    x / sqrt(sum(x^2) + 1e-6) (fp32 arithmetic)
 *   GDN_GATE_LOGITS  alpha holds a, beta holds b (fp32 logits); the kernels
 *                    use alpha = exp(-softplus(a)), beta = sigmoid(b), taking
 *                    log(alpha) = -softplus(a) directly for the decay
 *   GDN_ROPE_PAIRS, GDN_ROPE_INVERSE   the rotary calls' (see there)
 * Any other bit, or one of another family's: GDN_ERR_UNSUPPORTED.
 */
enum { GDN_QK_L2NORM = 1, GDN_GATE_LOGITS = 2, GDN_ROPE_PAIRS = 4, GDN_ROPE_INVERSE = 8 };

/*
 * gdn_prefill_chunked -- chunked prefill of B equal-length sequences.
 *
 *   q, k          [B, T, Hk, Dk]  dtype
 *   v             [B, T, Hv, Dv]  dtype
 *   alpha, beta   [B, T, Hv]      fp32   per-token decay and write strength
 *   initial_state [B, Hv, Dv, Dk] fp32   S_0 per (sequence, value head);
 *                                        NULL means a zero state
 *   out           [B, T, Hv, Dv]  dtype  o_t (fp32 -> bf16 rounds to nearest even)
 *   final_state   [B, Hv, Dv, Dk] fp32   S_T; NULL means not written;
 *                                        may equal initial_state
 *   prefix_states [B, floor(T / L), Hv, Dv, Dk] fp32, or NULL: the state
 *                 after every block of L = 64 * prefix_interval tokens,
 *                 row i of sequence b holding S_{L (i + 1)} (whole blocks
 *                 only; the state after a partial last block is final_state).
 *                 These are the block-aligned prefix states of "PHBA:
 *                 Prefix-State Hybrid Block Attention" (Abstract, Figure 1),
 *                 formed by the gated recurrence at block boundaries, and the
 *                 states a prefix cache keeps. prefix_interval >= 1 when
 *                 prefix_states is set (ignored otherwise); must not overlap
 *                 any other argument.
 *
 * Sizes: B >= 1, T >= 0, Hk >= 1, Hv a multiple of Hk, Dk == Dv in {64, 128}.
 * T == 0 writes the initial state (or zeros) to final_state.
 * The sequence is processed in chunks of 64 tokens; the result equals the
 * token recurrence up to rounding (the chunked form is an exact rewrite).
 *
 * workspace: optional device scratch of workspace_bytes bytes (16-byte
 * aligned, disjoint from every other argument, contents ignored and
 * overwritten; the caller keeps ownership). Its first 256 bytes hold a status
 * word (see "Debug checks" above). When it holds at least
 * gdn_prefill_workspace_size() bytes the call may run in two passes: the
 * state-independent per-chunk factors of all chunks first, then the
 * sequential state chain. NULL (or too small) selects the single-pass
 * kernel. Both give the same result up to rounding. With few (sequence,
 * value head) chains, bf16 and no prefix states, a workspace of the size
 * query's answer also allows the segmented arrangement: each sequence is
 * split into segments run in parallel from zero and from the identity
 * state, joined by a scan of the segment maps and an output correction
 * (same result up to rounding).
 */
gdn_status_t gdn_prefill_chunked(const void *q, const void *k, const void *v,
                                 const float *alpha, const float *beta,
                                 const float *initial_state, void *out,
                                 float *final_state, float *prefix_states,
                                 int32_t prefix_interval, int32_t B, int64_t T,
                                 int32_t Hk, int32_t Hv, int32_t Dk, int32_t Dv,
                                 gdn_dtype_t dtype, float scale, uint32_t flags,
                                 void *workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/*
 * gdn_prefill_chunked_noalloc -- gdn_prefill_chunked for callers that cannot
 * allocate device memory (code under graph capture, tight serving loops,
 * harnesses that forbid allocation). Same arguments and results as
 * gdn_prefill_chunked without the workspace pair: the call uses the
 * library's own static device scratch of 64 MiB per device (allocated when
 * the library's code is loaded on that device, held until the process ends)
 * as the workspace that gdn_prefill_workspace_size() names, and calls no
 * allocating routine. Shapes that need more scratch than 64 MiB are
 * rejected with GDN_ERR_UNSUPPORTED and no side effects (the scratch covers,
 * for example, one 4,096-token sequence at 16 q/k and 48 value heads of
 * dimension 128). Every call on a device shares that device's scratch, which
 * keeps the last call's contents: calls that may overlap in time on one
 * device (different streams, or threads) race and must be serialised by the
 * caller.
 */
gdn_status_t gdn_prefill_chunked_noalloc(const void *q, const void *k, const void *v,
                                         const float *alpha, const float *beta,
                                         const float *initial_state, void *out,
                                         float *final_state, float *prefix_states,
                                         int32_t prefix_interval, int32_t B, int64_t T,
                                         int32_t Hk, int32_t Hv, int32_t Dk, int32_t Dv,
                                         gdn_dtype_t dtype, float scale, uint32_t flags,
                                         hipStream_t stream);

/*
 * gdn_decode_step -- one new token per sequence, state updated in place.
 *
 *   q, k         [B, Hk, Dk]     dtype
 *   v            [B, Hv, Dv]     dtype
 *   alpha, beta  [B, Hv]         fp32
 *   state        [B, Hv, Dv, Dk] fp32   read as S_{t-1}, overwritten with S_t
 *   out          [B, Hv, Dv]     dtype  o_t = scale * S_t q_t
 *
 * Sizes: B >= 1, Hk >= 1, Hv a multiple of Hk, Dk == Dv in {64, 128}.
 * This is the fixed-cost step the pages point to when they note that decode
 * speed stays flat as the context grows ("The economics of hybrid
 * attention", section "Where the constraint moved").
 */
gdn_status_t gdn_decode_step(const void *q, const void *k, const void *v,
                             const float *alpha, const float *beta, float *state,
                             void *out, int32_t B, int32_t Hk, int32_t Hv,
                             int32_t Dk, int32_t Dv, gdn_dtype_t dtype,
                             float scale, uint32_t flags, hipStream_t stream);

/*
 * gdn_decode_multi -- K new tokens per sequence against a pool of state
 * slots, for checking several drafted tokens in one call. "The economics of
 * hybrid attention" names the model's multi-token prediction head (section
 * "The stack, verified") and the speculation head's draft buffers served at
 * two slots (section "Where the constraint moved"); this call is the mixer's
 * side of that: the K tokens of each sequence run in order on one state that
 * crosses HBM once per call instead of once per token.
 *
 *   q, k         [B, K, Hk, Dk]      dtype
 *   v            [B, K, Hv, Dv]      dtype
 *   alpha, beta  [B, K, Hv]          fp32
 *   state_pool   [num_slots, Hv, Dv, Dk] fp32, DEVICE memory
 *   src_slot     [B] int32, DEVICE memory: sequence b starts from the state
 *                in slot src_slot[b]; a negative value means a zero state
 *   dst_slot     [B] int32, DEVICE memory: S_K of sequence b is written to
 *                slot dst_slot[b]; a negative value means it is not written
 *   out          [B, K, Hv, Dv]      dtype  o_t = scale * S_t q_t
 *   step_states  [B, K, Hv, Dv, Dk]  fp32 or NULL: S_t after each token t
 *                (for rolling back to any accepted prefix); NULL skips them
 *
 * Sizes: B >= 1, K >= 0, num_slots >= 1, Hk >= 1, Hv a multiple of Hk,
 * Dk == Dv in {64, 128}. K == 0 copies slot src_slot[b] (or zeros) to slot
 * dst_slot[b]. A token with alpha = 1 and beta = 0 leaves the state unchanged,
 * so a batch with fewer real tokens in some sequences can be padded with such
 * tokens.
 *
 * The slot indices are read on the device. An index >= num_slots is not
 * an error the call can return: that sequence touches no slot and its
 * outputs (and step states) are set to NaN. The caller guarantees that the
 * non-negative dst_slot values are distinct and that no sequence's dst slot
 * is another sequence's src slot (src_slot[b] == dst_slot[b] updates in
 * place); otherwise workgroups race and the result is unspecified. Slots not
 * named in dst_slot are left untouched. state_pool, out, step_states and the
 * slot arrays must not overlap each other or the inputs (GDN_ERR_ALIAS).
 */
gdn_status_t gdn_decode_multi(const void *q, const void *k, const void *v,
                              const float *alpha, const float *beta,
                              float *state_pool, int32_t num_slots,
                              const int32_t *src_slot, const int32_t *dst_slot,
                              void *out, float *step_states, int32_t B, int32_t K,
                              int32_t Hk, int32_t Hv, int32_t Dk, int32_t Dv,
                              gdn_dtype_t dtype, float scale, uint32_t flags,
                              hipStream_t stream);

/*
 * gdn_varlen_prefill -- chunked prefill of N packed sequences.
 *
 *   q, k          [total_T, Hk, Dk] dtype
 *   v, out        [total_T, Hv, Dv] dtype
 *   alpha, beta   [total_T, Hv]     fp32
 *   cu_seqlens    [N + 1] int32, DEVICE memory: sequence n spans tokens
 *                 cu_seqlens[n] .. cu_seqlens[n+1]-1; cu_seqlens[0] = 0,
 *                 non-decreasing, cu_seqlens[N] = total_T. Its contents are
 *                 checked only under GDN_DEBUG=1. Otherwise the kernels clamp
 *                 each sequence's start and end into [0, total_T] (end >=
 *                 start), so malformed offsets give meaningless results but
 *                 no access outside the caller's buffers.
 *   initial_state [N, Hv, Dv, Dk] fp32 or NULL (zero states)
 *   final_state   [N, Hv, Dv, Dk] fp32 or NULL; may equal initial_state
 *   prefix_states [floor(total_T / L) + N, Hv, Dv, Dk] fp32 or NULL, with
 *                 L = 64 * prefix_interval: as for gdn_prefill_chunked, the
 *                 state after each whole block of L tokens of a sequence;
 *                 block i of sequence n goes to row
 *                 floor(cu_seqlens[n] / L) + n + i (rows that no block maps
 *                 to are left untouched)
 *
 * Sizes: N >= 1, 0 <= total_T < 2^31, Hv a multiple of Hk, Dk == Dv in
 * {64, 128}. Chunks restart at every sequence boundary. workspace: as for
 * gdn_prefill_chunked.
 */
gdn_status_t gdn_varlen_prefill(const void *q, const void *k, const void *v,
                                const float *alpha, const float *beta,
                                const int32_t *cu_seqlens, int32_t N,
                                int64_t total_T, const float *initial_state,
                                void *out, float *final_state,
                                float *prefix_states, int32_t prefix_interval,
                                int32_t Hk,
                                int32_t Hv, int32_t Dk, int32_t Dv,
                                gdn_dtype_t dtype, float scale, uint32_t flags,
                                void *workspace, size_t workspace_bytes,
                                hipStream_t stream);

/*
 * gdn_prefill_workspace_size -- bytes of workspace the prefill calls can use.
 *
 *   packed = 0: gdn_prefill_chunked with num_seqs = B and tokens = T;
 *   packed = 1: gdn_varlen_prefill with num_seqs = N and tokens = total_T.
 *
 * Returns 0 when the library would not use a workspace for this shape on the
 * current device (enough (sequence, value head) pairs to fill it in one
 * pass), when an argument is invalid, or when no device is available. The
 * size is 256 bytes (the status word) plus 17,152 bytes (bf16) or 33,536
 * bytes (fp32) per (64-token chunk, value head): B * ceil(T/64) chunks, or
 * ceil(total_T/64) + N for packed batches. It is larger where
 * gdn_prefill_chunked would run segmented (the segment end states, maps,
 * start states and the identity-start outputs).
 */
size_t gdn_prefill_workspace_size(int32_t num_seqs, int64_t tokens, int32_t Hk,
                                  int32_t Hv, int32_t Dk, int32_t Dv,
                                  gdn_dtype_t dtype, int32_t packed);

/*
 * Gated linear recurrence (the scan calls)
 * ----------------------------------------
 * The vector-state sibling of the gated delta rule: one state value per
 * channel instead of a matrix per head. Per sequence and channel
 *
 *     h_t = alpha_t * h_{t-1} + beta_t * x_t,      out_t = h_t
 *
 * with a decay and a write strength of its own for every token and channel.
 * x, alpha, beta and out have the element type `dtype`; states are fp32 [D]
 * per sequence. beta == NULL ties the gates: beta_t = 1 - alpha_t. `flags`
 * accepts GDN_GATE_LOGITS: alpha holds a, beta holds b, and the kernels use
 * alpha = exp(-softplus(a)) = sigmoid(-a), beta = sigmoid(b) (tied:
 * beta = sigmoid(a), formed without cancellation). Any other bit:
 * GDN_ERR_UNSUPPORTED. Unlike the delta-rule calls, alpha is used as given
 * (not clamped). 1 <= D <= 2^22.
 *
 * A NaN or infinity (in an input or a state) reaches no other channel or
 * sequence and no earlier token; from its token on, out and the states of its
 * channel are not finite, as the recurrence has it. Which of the two they are
 * may differ from walking the tokens one by one: the product of the decays of
 * a run of tokens may be 0 in fp32, and 0 times infinity is NaN. Gradients are
 * the same towards earlier tokens.
 */

/* Tokens per tile of the scan kernels: block starts at multiples of this are
 * where gdn_scan_backward picks up prefix states. */
enum { GDN_SCAN_TILE = 128 };

/*
 * gdn_scan_prefill -- the recurrence over B equal-length sequences.
 *
 *   x, alpha, beta, out [B, T, D] dtype   (beta may be NULL: tied gates)
 *   initial_state [B, D] fp32 or NULL (zero)
 *   final_state   [B, D] fp32 or NULL; may equal initial_state
 *   prefix_states [B * floor(T / L), D] fp32 or NULL: the state after every
 *                 whole block of L = 64 * prefix_interval tokens, in the rows
 *                 of gdn_prefill_chunked's prefix_states
 *
 * Sizes: B >= 1, T >= 0, D >= 1. T == 0 writes the initial state (or zeros) to
 * final_state. workspace: optional device scratch (16-byte aligned, disjoint
 * from every other argument, contents ignored and overwritten). With at least
 * gdn_scan_workspace_size() bytes the call may cut the sequences along time
 * and run the pieces side by side; NULL or less runs each sequence's tiles one
 * after the other. Both give the same bits. Calls that may run at the same
 * time need a workspace each: two that overlap on one neither hang nor leave
 * their buffers, but their results are undefined (NaN, values left as they
 * were, or finite wrong ones). Aliasing rules as for gdn_prefill_chunked.
 */
gdn_status_t gdn_scan_prefill(const void *x, const void *alpha, const void *beta,
                              const float *initial_state, void *out, float *final_state,
                              float *prefix_states, int32_t prefix_interval, int32_t B,
                              int64_t T, int32_t D, gdn_dtype_t dtype, uint32_t flags,
                              void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * gdn_scan_varlen_prefill -- the recurrence over N packed sequences.
 *
 *   x, alpha, beta, out [total_T, D] dtype
 *   cu_seqlens          [N + 1] int32, DEVICE memory, as for
 *                       gdn_varlen_prefill (clamped, checked under GDN_DEBUG=1)
 *   initial_state, final_state [N, D] fp32 or NULL
 *   prefix_states       [floor(total_T / L) + N, D] fp32 or NULL, in the rows
 *                       of gdn_varlen_prefill's prefix_states
 *
 * A sequence of length zero hands its initial state (or zeros) to final_state.
 * Each sequence's results have the same bits as gdn_scan_prefill's on it alone.
 */
gdn_status_t gdn_scan_varlen_prefill(const void *x, const void *alpha, const void *beta,
                                     const int32_t *cu_seqlens, int32_t N, int64_t total_T,
                                     const float *initial_state, void *out, float *final_state,
                                     float *prefix_states, int32_t prefix_interval, int32_t D,
                                     gdn_dtype_t dtype, uint32_t flags, void *workspace,
                                     size_t workspace_bytes, hipStream_t stream);

/*
 * gdn_scan_backward -- gradients of gdn_scan_prefill.
 *
 *   dout                [B, T, D] dtype: gradient of out
 *   x, alpha, beta, initial_state: the forward call's inputs
 *   prefix_states       [B * floor(T / L), D] fp32: as the forward call wrote
 *                       them, with prefix_interval 1 or 2 (L = 64 or 128); the
 *                       states inside a tile of GDN_SCAN_TILE tokens are
 *                       recomputed from them in fp32. May be NULL when
 *                       T <= GDN_SCAN_TILE.
 *   dfinal              [B, D] fp32 or NULL (zero): gradient of final_state
 *   dx, dalpha, dbeta   [B, T, D] dtype; dbeta is NULL exactly when beta is.
 *                       With GDN_GATE_LOGITS dalpha and dbeta are the gradients
 *                       of the logits. Tied gates: dalpha holds both paths.
 *   dinitial            [B, D] fp32 or NULL: gradient of initial_state
 *
 * With g_t = dout_t + alpha_{t+1} g_{t+1} (from dfinal at the end):
 *   dx_t = beta_t g_t, dbeta_t = g_t x_t, dalpha_t = g_t h_{t-1}
 *   (tied: g_t (h_{t-1} - x_t)), dinitial = alpha_1 g_1.
 * T == 0 copies dfinal (or zeros) to dinitial. Outputs overlap nothing.
 * workspace: as for gdn_scan_prefill.
 */
gdn_status_t gdn_scan_backward(const void *dout, const void *x, const void *alpha,
                               const void *beta, const float *initial_state,
                               const float *prefix_states, int32_t prefix_interval,
                               const float *dfinal, void *dx, void *dalpha, void *dbeta,
                               float *dinitial, int32_t B, int64_t T, int32_t D,
                               gdn_dtype_t dtype, uint32_t flags, void *workspace,
                               size_t workspace_bytes, hipStream_t stream);

/*
 * gdn_scan_varlen_backward -- gradients of gdn_scan_varlen_prefill: as above
 * with [total_T, D] tensors, cu_seqlens, states [N, D] and the packed call's
 * prefix rows (prefix_states may be NULL when total_T <= GDN_SCAN_TILE).
 */
gdn_status_t gdn_scan_varlen_backward(const void *dout, const void *x, const void *alpha,
                                      const void *beta, const int32_t *cu_seqlens, int32_t N,
                                      int64_t total_T, const float *initial_state,
                                      const float *prefix_states, int32_t prefix_interval,
                                      const float *dfinal, void *dx, void *dalpha, void *dbeta,
                                      float *dinitial, int32_t D, gdn_dtype_t dtype,
                                      uint32_t flags, void *workspace, size_t workspace_bytes,
                                      hipStream_t stream);

/*
 * gdn_scan_decode -- K new tokens per sequence against a pool of state slots.
 *
 *   x, alpha, beta, out  [B, K, D] dtype (beta may be NULL)
 *   state_pool           [num_slots, D] fp32
 *   src_slot, dst_slot   [B] int32, DEVICE memory, with gdn_decode_multi's
 *                        meaning and rules (negative: zero state / not
 *                        written; past the pool: NaN outputs, no slot touched)
 *
 * Sizes: B >= 1, K >= 0, D >= 1. K == 0 copies slots.
 */
gdn_status_t gdn_scan_decode(const void *x, const void *alpha, const void *beta,
                             float *state_pool, int32_t num_slots, const int32_t *src_slot,
                             const int32_t *dst_slot, void *out, int32_t B, int32_t K,
                             int32_t D, gdn_dtype_t dtype, uint32_t flags, hipStream_t stream);

/*
 * gdn_scan_workspace_size -- bytes of workspace the scan calls can use:
 * packed = 0: num_seqs = B, tokens = T; packed = 1: num_seqs = N,
 * tokens = total_T. 0 when the call would not use one (sequences of one tile,
 * or enough equal ones to fill the device), when an argument is invalid, or when
 * no device is available.
 */
size_t gdn_scan_workspace_size(int32_t num_seqs, int64_t tokens, int32_t D, gdn_dtype_t dtype,
                               int32_t packed);

/*
 * gdn_rms_norm -- root-mean-square norm with the residual's addition and an
 * output in 8 bits with scales: the step in front of the mixer's projections
 * (with a residual) and behind the mixer per value head (rows of D = 128; in 8
 * bits where no output gate comes between the norm and the projection).
 *
 *   x        [rows, D] dtype
 *   residual [rows, D] dtype or NULL (none)
 *   weight   [D]       dtype
 *   residual_out [rows, D] dtype or NULL (not written): r = x + residual,
 *            rounded; may equal residual or x. Needs a residual.
 *   out      [rows, D] dtype or NULL: y = r / sqrt(mean(r^2) + eps) * weight
 *   out8     [rows, D] OCP e4m3 or NULL: y / scale, rounded to nearest even
 *   scales   [rows, G] fp32, set exactly when out8 is. scale = max |y| / 448
 *            over the group (at least 2^-100), so that out8 * scale stands
 *            for y. group 0: one scale per row (G = 1); group 128: one per 128
 *            columns (G = ceil(D / 128)); others: GDN_ERR_UNSUPPORTED.
 *
 * The sum, the mean and y are fp32; y is formed from the unrounded sum. out8 is
 * formed from r * weight, for the row's factor cancels in y / scale: where fp32
 * holds those products (without a residual those of bf16), every value is the
 * one of exact arithmetic, ties to even. Sizes: rows >= 0, 1 <= D <= 16384, eps a
 * normal fp32 number. At least one of out and out8. A NaN or Inf in a row, or
 * squares whose sum passes fp32's range, make NaN of that row.
 */
gdn_status_t gdn_rms_norm(const void *x, const void *residual, const void *weight,
                          void *residual_out, void *out, void *out8, float *scales,
                          int32_t group, int64_t rows, int32_t D, gdn_dtype_t dtype, float eps,
                          hipStream_t stream);

/*
 * gdn_rms_norm_backward -- gradients of gdn_rms_norm's y at a stored row sum.
 *
 *   dout      [rows, D] dtype: gradient of y
 *   r         [rows, D] dtype: the row sums (residual_out; x without a residual)
 *   weight    [D] dtype
 *   dresidual [rows, D] dtype or NULL: gradient arriving at residual_out
 *   dx        [rows, D] dtype: gradient of x and of residual alike; may equal
 *             dresidual
 *   dweight   [D] fp32 or NULL (not wanted)
 *
 * With s = 1 / sqrt(mean(r^2) + eps):
 *   dx = s w dout - r s^3 mean(w dout r) + dresidual,
 *   dweight = sum over rows of dout r s (fp32, in a fixed order).
 * workspace: gdn_rms_norm_workspace_size(rows, D) bytes, required with dweight
 * (GDN_ERR_BAD_SHAPE when too small), unused without; for one call at a time.
 */
gdn_status_t gdn_rms_norm_backward(const void *dout, const void *r, const void *weight,
                                   const void *dresidual, void *dx, float *dweight,
                                   int64_t rows, int32_t D, gdn_dtype_t dtype, float eps,
                                   void *workspace, size_t workspace_bytes,
                                   hipStream_t stream);
size_t gdn_rms_norm_workspace_size(int64_t rows, int32_t D);

/*
 * gdn_beam_select -- beam search's selection over beams and vocabulary.
 *
 *   logits   [B, W, V] dtype: next-token logits of every beam
 *   scores   [B, W] fp32: summed log-probability of every beam
 *   finished [B, W] uint8 or NULL: nonzero beams have ended and offer only
 *            themselves (token eos, score unchanged)
 *   beam_slots [B, W] int32 or NULL: the state slot of every beam
 *   new_scores [B, W] fp32, tokens [B, W] int32, parents [B, W] int32 (beam
 *            index in its batch item): the W best candidates, best first
 *   new_finished [B, W] uint8 or NULL: the parent's flag, or token == eos
 *   src_slots [B, W] int32, set exactly when beam_slots is:
 *            beam_slots[b][parent], the src_slot of the next
 *            gdn_decode_multi or gdn_scan_decode call (states are reordered by
 *            reading the parent's slot; give every beam a dst_slot that is no
 *            beam's source), or the index of gdn_gather_states
 *
 * A live beam w offers every token v at score_w + logit - logsumexp(logits_w),
 * compared in fp64 (within a beam the W largest logits compete); ties go to the
 * lowest w * V + v. A beam whose score or logsumexp is not finite (all logits
 * -inf, any NaN or +inf) offers its tokens at -inf, as does a logit of -inf;
 * finite logits of any size are masks or scores like others. Sizes: B >= 1, 1 <= W <= 32, V >= 1,
 * B * W * V < 2^40; eos in [0, V), or -1 for none (then finished and
 * new_finished are NULL). Results are the same from call to call.
 * workspace: gdn_beam_workspace_size() bytes, required; for one call at a time.
 */
gdn_status_t gdn_beam_select(const void *logits, const float *scores, const uint8_t *finished,
                             const int32_t *beam_slots, float *new_scores, int32_t *tokens,
                             int32_t *parents, uint8_t *new_finished, int32_t *src_slots,
                             int32_t B, int32_t W, int64_t V, int32_t eos, gdn_dtype_t dtype,
                             void *workspace, size_t workspace_bytes, hipStream_t stream);
size_t gdn_beam_workspace_size(int32_t B, int32_t W, int64_t V, gdn_dtype_t dtype);

/*
 * gdn_gather_states -- rows of a state buffer in a new order: row i of dst is
 * row index[i] of src. For callers whose states are not addressed by slots.
 *
 *   src [num_src, row_bytes], dst [rows, row_bytes], index [rows] int32 in
 *   DEVICE memory. row_bytes: a multiple of 16. A negative index writes zeros,
 *   one past the end writes bytes of 0xff (NaN as fp32 or bf16). src and dst
 *   must not overlap (an in-place permutation would need a copy).
 */
gdn_status_t gdn_gather_states(const void *src, int64_t num_src, const int32_t *index, void *dst,
                               int64_t rows, int64_t row_bytes, hipStream_t stream);

/*
 * Softmax attention (the attn, cache and rotary calls)
 * ----------------------------------------------------
 * The stack's other token mixer: every fourth block is attention with grouped
 * heads ("The Hybrid Attention in Qwen3.8-27B", section "Grouped-query attention
 * multiplies on top of that": 24 query heads on 4 key heads of dimension 256),
 * whose cache of keys and values grows with the context. Query head i reads key
 * head i / (Hq / Hk). q, k, v, out, the caches and the gradients have the
 * element type `dtype`; sums, softmax statistics and lse are fp32; in bf16 the
 * weights (and the gradients' inner terms) are rounded to bf16 as operands of
 * the matrix products (not so in gdn_attn_decode for a sequence's own tokens
 * where K Hq / Hk <= 32: there they are two bf16 terms). Hq a multiple of Hk, D
 * in {64, 128, 256}, Hq * D <= 2^24, scale positive and finite (1 / sqrt(D) as a
 * rule).
 *
 * A query without any key has out = 0 and lse = -infinity; one whose scores
 * are all -infinity counts as one. An infinity or NaN in a key or value that a
 * query does not see (a later token, another sequence, the rest of a page)
 * does not reach it; what it reaches is not finite. Scores (scale q . k) beyond
 * 2^28 in magnitude may give NaN.
 */

/*
 * gdn_attn_prefill -- causal attention over B prompts of T tokens.
 *
 *   q, out [B, T, Hq, D] dtype,  k, v [B, T, Hk, D] dtype
 *   lse    [B, T, Hq] fp32 or NULL (not written): log of the sum of the
 *          exponentials of a query's scores; the backward call takes it
 *
 *   out_t = sum_{j <= t} exp(scale q_t . k_j - lse_t) v_j
 *
 * Sizes: B >= 1, 0 <= T <= 2^30, (B T / 16 + B) Hq <= 2^30. out and lse overlap
 * nothing.
 */
gdn_status_t gdn_attn_prefill(const void *q, const void *k, const void *v, void *out, float *lse,
                              int32_t B, int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                              gdn_dtype_t dtype, float scale, hipStream_t stream);

/*
 * gdn_attn_varlen_prefill -- the same over N packed prompts: tensors
 * [total_T, H, D], lse [total_T, Hq], cu_seqlens as for gdn_varlen_prefill
 * (clamped, checked under GDN_DEBUG=1). Tokens behind the last sequence are
 * left as they were.
 */
gdn_status_t gdn_attn_varlen_prefill(const void *q, const void *k, const void *v,
                                     const int32_t *cu_seqlens, int32_t N, int64_t total_T,
                                     void *out, float *lse, int32_t Hq, int32_t Hk, int32_t D,
                                     gdn_dtype_t dtype, float scale, hipStream_t stream);

/*
 * gdn_attn_backward -- gradients of gdn_attn_prefill.
 *
 *   dout    [B, T, Hq, D] dtype: gradient of out
 *   q, k, v, out, lse: the forward call's inputs and outputs
 *   dq      [B, T, Hq, D] dtype,  dk, dv [B, T, Hk, D] dtype (sums over the
 *           query heads of a key head)
 *
 * With p = exp(scale q_t . k_j - lse_t) and ds = p (dout_t . v_j - dout_t . out_t):
 *   dq_t = scale sum_j ds k_j,  dk_j = scale sum_t ds q_t,  dv_j = sum_t p dout_t.
 * out and lse may be over more keys than these (a prefix in front, say): the
 * results are then the part of these keys.
 * Results are the same from call to call. workspace:
 * gdn_attn_backward_workspace_size() bytes, required; for one call at a time.
 */
gdn_status_t gdn_attn_backward(const void *dout, const void *q, const void *k, const void *v,
                               const void *out, const float *lse, void *dq, void *dk, void *dv,
                               int32_t B, int64_t T, int32_t Hq, int32_t Hk, int32_t D,
                               gdn_dtype_t dtype, float scale, void *workspace,
                               size_t workspace_bytes, hipStream_t stream);

/* gdn_attn_varlen_backward -- gradients of gdn_attn_varlen_prefill. */
gdn_status_t gdn_attn_varlen_backward(const void *dout, const void *q, const void *k,
                                      const void *v, const void *out, const float *lse,
                                      const int32_t *cu_seqlens, int32_t N, int64_t total_T,
                                      void *dq, void *dk, void *dv, int32_t Hq, int32_t Hk,
                                      int32_t D, gdn_dtype_t dtype, float scale, void *workspace,
                                      size_t workspace_bytes, hipStream_t stream);

/* Workspace of the two on the current device: packed = 0: num_seqs = B, tokens = T;
 * packed = 1: num_seqs = N, tokens = total_T. 0 for invalid arguments, no tokens or
 * no device. */
size_t gdn_attn_backward_workspace_size(int32_t num_seqs, int64_t tokens, int32_t Hq, int32_t Hk,
                                        int32_t D, gdn_dtype_t dtype, int32_t packed);

/*
 * gdn_attn_decode -- K new tokens per sequence against a paged cache, for a batch
 * whose sequences may share long prefixes.
 *
 *   q, out     [B, K, Hq, D] dtype
 *   k_cache, v_cache [num_pages, page_size, Hk, D] dtype
 *   page_table [B, max_pages] int32: the pages of a sequence's own tokens, in order
 *   lengths    [B] int32: tokens of the sequence in these pages, the K new ones
 *              among them (gdn_kv_append comes before this call). Token t of the
 *              K sees the first lengths[b] - K + 1 + t of them
 *   prefix_table [G, max_prefix_pages], prefix_lengths [G], prefix_groups [G + 1]
 *              int32, or all NULL: sequences prefix_groups[g] .. [g + 1] - 1 share
 *              prefix g, whose tokens stand in front of their own and are not
 *              among lengths[b]. Every new token sees all of its prefix, which is
 *              read once for the group. prefix_groups[0] = 0, non-decreasing,
 *              prefix_groups[G] = B (clamped, checked under GDN_DEBUG=1)
 *   lse        [B, K, Hq] fp32 or NULL, over prefix and own tokens
 *
 * All index arrays are DEVICE memory. A page that is outside the pool (negative
 * ones too) makes NaN of the queries that see a token in it; a length past its
 * table's max_pages * page_size does so for the whole sequence; a negative
 * length counts as 0. Table entries behind the last token are not read.
 * Sizes: B, K >= 1, B K Hq <= 2^30, page_size a power of two from 16 to 2^20,
 * max_pages * page_size <= 2^31 - 2^21, 1 <= G <= B. K may be a whole piece of a
 * prompt. workspace: gdn_attn_decode_workspace_size() bytes, required where
 * that is not 0; for one call at a time.
 */
gdn_status_t gdn_attn_decode(const void *q, const void *k_cache, const void *v_cache,
                             int32_t num_pages, int32_t page_size, const int32_t *page_table,
                             int32_t max_pages, const int32_t *lengths,
                             const int32_t *prefix_table, int32_t max_prefix_pages,
                             const int32_t *prefix_lengths, const int32_t *prefix_groups,
                             int32_t G, void *out, float *lse, int32_t B, int32_t K, int32_t Hq,
                             int32_t Hk, int32_t D, gdn_dtype_t dtype, float scale,
                             void *workspace, size_t workspace_bytes, hipStream_t stream);
/* On the current device; G = 0: no prefixes. 0: none needed (or invalid arguments, or
 * no device). */
size_t gdn_attn_decode_workspace_size(int32_t B, int32_t K, int32_t Hq, int32_t Hk, int32_t D,
                                      int32_t page_size, int32_t max_pages, int32_t G,
                                      int32_t max_prefix_pages, gdn_dtype_t dtype);

/*
 * gdn_rotary -- rotary positions on one or several axes.
 *
 *   q, q_out [tokens, Hq, D] dtype;  k, k_out [tokens, Hk, D] dtype or both NULL
 *   positions [axes, tokens] int32: the tokens' places (time, height, width, say)
 *   inv_freq  [R / 2] fp32: radians per position of every pair
 *   pair_axis [R / 2] int32 or NULL (axis 0): the axis of every pair; a pair
 *             whose axis is outside [0, axes) becomes NaN
 *
 * The first R columns of a head are pairs (j, j + R / 2), or with GDN_ROPE_PAIRS
 * neighbours (2j, 2j + 1); the others are copied. A pair (x, y) becomes
 * (x cos - y sin, y cos + x sin) at the angle positions[axis][token] * inv_freq,
 * formed and reduced in 64 bits. GDN_ROPE_INVERSE turns back, which is the
 * gradient of the rotation. q_out may be q, k_out may be k. Sizes: tokens >= 0,
 * D a multiple of 8 up to 1024, R even, 2 <= R <= D, axes >= 1.
 */
gdn_status_t gdn_rotary(const void *q, const void *k, void *q_out, void *k_out,
                        const int32_t *positions, int32_t axes, const float *inv_freq,
                        const int32_t *pair_axis, int32_t R, int64_t tokens, int32_t Hq,
                        int32_t Hk, int32_t D, gdn_dtype_t dtype, uint32_t flags,
                        hipStream_t stream);

/*
 * gdn_kv_append -- new keys and values into a paged cache, rotated on the way.
 *
 *   k, v       [N, T, Hk, D] dtype, or [total_T, Hk, D] with cu_seqlens
 *   k_cache, v_cache, page_table [N, max_pages]: as for gdn_attn_decode
 *   lengths    [N] int32: tokens in the cache before this call. Token i of
 *              sequence n gets the place lengths[n] + i
 *   cu_seqlens [N + 1] int32 or NULL (T tokens per sequence): as for
 *              gdn_varlen_prefill, checked under GDN_DEBUG=1
 *   q, q_out   [.., Hq, D] dtype or both NULL: the new tokens' queries, rotated
 *   k_out      like k, or NULL: the rotated keys, for the prompts' own attention
 *   inv_freq, R, positions, axes, pair_axis, flags: as for gdn_rotary. inv_freq
 *              NULL: no rotation; positions NULL: the places in the cache
 *   tokens     T, or total_T
 *
 * All index arrays are DEVICE memory. A token whose place is negative or past the
 * table, or whose page is outside the pool (negative ones too), is not written to
 * the cache (q_out and k_out are); tokens outside every sequence are written
 * nowhere. No two tokens of a call may share a place. q_out may be q, k_out may
 * be k. D a multiple of 8 up to 1024; pages as for gdn_attn_decode.
 */
gdn_status_t gdn_kv_append(const void *k, const void *v, void *k_cache, void *v_cache,
                           int32_t num_pages, int32_t page_size, const int32_t *page_table,
                           int32_t max_pages, const int32_t *lengths, const int32_t *cu_seqlens,
                           const void *q, void *q_out, void *k_out, const float *inv_freq,
                           int32_t R, const int32_t *positions, int32_t axes,
                           const int32_t *pair_axis, int32_t N, int64_t tokens, int32_t Hq,
                           int32_t Hk, int32_t D, gdn_dtype_t dtype, uint32_t flags,
                           hipStream_t stream);

/* Static description of a status; for GDN_ERR_HIP, the calling thread's
 * last HIP error detail. The pointer stays valid until the thread's next
 * call into the library. */
const char *gdn_status_string(gdn_status_t s);

/* Library version, major * 10000 + minor * 100 + patch. */
int32_t gdn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
