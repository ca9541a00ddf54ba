// gdn_attn_launch.hpp -- host-side launchers of the attention, cache and rotary
// kernels (internal to the library).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_ops_launch.hpp"

namespace gdn {

// Attention over whole prompts. Dense batches pass cu == nullptr and T tokens
// per sequence; total = tokens in the batch.
struct AttnParams {
    const void *q, *k, *v;
    void *out;
    float *lse;  // [tokens, Hq] or nullptr
    const int32_t *cu;
    int64_t T, total;
    int32_t N, Hq, Hk;
    float scale;
};

struct AttnBackwardParams {
    const void *dout, *q, *k, *v, *out;
    const float *lse;
    void *dq, *dk, *dv;
    const int32_t *cu;
    int64_t T, total;
    int32_t N, Hq, Hk;
    float scale;
    float *stats;   // workspace: [3][Hq][total], log2-scaled lse, delta, 1 / sum of weights
    float *parts;   // workspace: [split][2][total][Hk][D] partial dk, dv (split > 1)
    int32_t split;  // workgroups that share the query heads of a key head
};

// dtype: 0 = fp32, 1 = bf16, here and below. D: 64, 128 or 256.
hipError_t launch_attn(const AttnParams &p, int dtype, int D, int cus, hipStream_t stream);
int32_t attn_backward_split(int64_t N, int64_t T, int64_t total, int32_t Hq, int32_t Hk, int D,
                            int dtype, bool packed, int cus);
hipError_t launch_attn_backward(const AttnBackwardParams &p, int dtype, int D, int cus,
                                hipStream_t stream);

// New tokens against a paged cache.
struct AttnDecodeParams {
    const void *q;
    const void *kc, *vc;
    const int32_t *table, *lengths;
    const int32_t *ptable, *plengths, *pgroups;  // shared prefixes, or nullptr
    void *out;
    float *lse;
    int32_t B, K, Hq, Hk, G;
    int32_t num_pages, page_shift, max_pages, max_ppages;
    float scale;
};

size_t attn_decode_workspace_bytes(const AttnDecodeParams &p, int dtype, int D, int cus);
hipError_t launch_attn_decode(const AttnDecodeParams &p, int dtype, int D, int cus, void *ws,
                              hipStream_t stream);

// Rotary positions, and appending to a paged cache. One launch turns q and k
// (either may be nullptr) and copies k and v into the cache (where kc is set).
struct RotaryParams {
    const void *q, *k, *v;
    void *q_out, *k_out;      // nullptr: not written
    void *kc, *vc;
    const float *freq;        // [R / 2], or nullptr: no rotation
    const int32_t *pos;       // [axes][tokens], or nullptr: the place in the sequence
    const int32_t *axis;      // [R / 2], or nullptr: axis 0
    const int32_t *cu, *lengths, *table;
    int64_t tokens, T;        // T: tokens per sequence of a dense batch
    int32_t N, Hq, Hk, D, R, axes;
    int32_t num_pages, page_shift, max_pages;
    bool pairs, inverse;
};
hipError_t launch_rotary(const RotaryParams &p, int dtype, hipStream_t stream);

}  // namespace gdn
