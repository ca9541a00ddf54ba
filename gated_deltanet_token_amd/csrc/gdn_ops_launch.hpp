// gdn_ops_launch.hpp -- host-side launchers of the scan, norm and beam kernels
// (internal to the library), and the status of a failed HIP call.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/gdn.h"
#include "gdn_grid.hpp"

namespace gdn {

// GDN_ERR_HIP, with the calling thread's detail text set (gdn_api.hip).
gdn_status_t hip_fail(hipError_t e, const char *where);
// Compute units of the current device (gdn_api.hip).
gdn_status_t device_cus(int *cus);
// GDN_DEBUG=1 and `stream` is not being captured (gdn_api.hip).
bool debug_checks(hipStream_t stream);
gdn_status_t debug_cu_seqlens(const int32_t *cu, int32_t N, int64_t total_T, hipStream_t stream);

// One call of the gated linear recurrence, forward or backward. Dense batches
// pass cu == nullptr and T tokens per sequence.
struct ScanParams {
    const void *x, *a, *b;  // b == nullptr: tied gates
    const float *h0;
    const float *prefix_in;  // backward: states at block ends
    float *prefix_out;       // forward: the same, written
    int64_t prefix_len;      // L, tokens per block
    void *out;               // forward
    float *hT;
    const void *dout;        // backward
    const float *dhT;
    void *dx, *da, *db;
    float *dh0;
    const int32_t *cu;
    int64_t T, total;
    int32_t N, D;
    uint32_t flags;
};

struct ScanDecodeParams {
    const void *x, *a, *b;
    float *pool;
    const int32_t *src, *dst;
    void *out;
    int32_t num_slots, B, K, D;
    uint32_t flags;
};

// dtype: 0 = fp32, 1 = bf16, here and below.
size_t scan_workspace_bytes(int64_t nseq, int64_t tokens, int32_t D, int dtype, bool packed,
                            int cus);
hipError_t launch_scan(const ScanParams &p, int dtype, int cus, void *ws, size_t ws_bytes,
                       hipStream_t stream);
hipError_t launch_scan_backward(const ScanParams &p, int dtype, int cus, void *ws,
                                size_t ws_bytes, hipStream_t stream);
hipError_t launch_scan_decode(const ScanDecodeParams &p, int dtype, hipStream_t stream);

struct NormParams {
    const void *x, *res, *w;
    void *res_out, *out;
    uint8_t *out8;
    float *scales;
    int32_t group;
    int64_t rows;
    int32_t D;
    float eps, inv_d;  // inv_d: 1 / D
};

struct NormBackwardParams {
    const void *dout, *r, *w, *dres;
    void *dx;
    float *dw;
    float *partial;  // [norm_partials(rows, D)][norm_partial_width(D)]
    int64_t rows;
    int32_t D;
    float eps, inv_d;  // inv_d: 1 / D
};

hipError_t launch_norm(const NormParams &p, int dtype, hipStream_t stream);
int norm_partials(int64_t rows, int32_t D);
constexpr int norm_partial_width(int D) { return (D + 7) / 8 * 8; }
hipError_t launch_norm_backward(const NormBackwardParams &p, int dtype, hipStream_t stream);

struct BeamParams {
    const void *logits;
    const float *scores;
    const uint8_t *finished;
    const int32_t *slots;
    float *new_scores;
    int32_t *tokens, *parents;
    uint8_t *new_finished;
    int32_t *src_slots;
    int32_t B, W;
    int64_t V;
    int32_t eos;
};

size_t beam_workspace_bytes(int32_t B, int32_t W, int64_t V, int dtype);
hipError_t launch_beam(const BeamParams &p, int dtype, void *ws, hipStream_t stream);

hipError_t launch_gather(const void *src, int64_t num_src, const int32_t *index, void *dst,
                         int64_t rows, int64_t row_bytes, hipStream_t stream);

}  // namespace gdn
