// gate_internal.h -- launcher interface of what stands in front of the
// dispatch (residual norm, choice of experts, balance loss) and of the
// gradients. Arguments are checked in epx_api.hip; launchers assume valid
// shapes and return the HIP launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace epx {

struct NormArgs {
    const uint16_t *x;         // [T, h] bf16
    const uint16_t *residual;  // [T, h] bf16, or null
    const void *w;             // [h] bf16 or fp32
    int T, h;
    float eps;
    uint16_t *res_out;  // [T, h] bf16 (with residual)
    uint16_t *out;      // [T, h] bf16, or null
    uint8_t *codes;     // [T, h] e4m3, or null
    float *scales;      // [T, scale_stride(h)] with codes
};

hipError_t launch_rms_norm(const NormArgs &a, bool w_f32, hipStream_t stream);

struct NormBwdArgs {
    const uint16_t *dout;  // [T, h] bf16
    const uint16_t *x;     // [T, h] bf16: what was normed
    const void *w;         // [h] bf16 or fp32
    const uint16_t *dres;  // [T, h] bf16, or null
    int T, h;
    float eps;
    uint16_t *dx;   // [T, h] bf16
    float *dw;      // [h]
    float *partial; // workspace [blocks, h]
};

// Rows of fp32 partial sums that the backward pass keeps in its workspace.
int norm_bwd_blocks(int T, int h);
hipError_t launch_rms_norm_backward(const NormBwdArgs &a, bool w_f32, hipStream_t stream);

struct RouteArgs {
    const float *logits;  // [T, E]
    const float *bias;    // [E], or null
    const uint8_t *mask;  // [T], or null
    int T, E, K, G, top_groups, group_size;
    uint32_t size_mul;    // div_magic(group_size)
    float scale;
    int64_t *topk_idx;    // [T, K]
    float *topk_w;        // [T, K]
    int *err;
};

hipError_t launch_route(const RouteArgs &a, bool sigmoid, bool normalize, hipStream_t stream);

// The balance loss's workspace.
struct BalanceWs {
    unsigned int *done;  // blocks of the second launch that have ended
    float *dot;          // [S, ceil(E / 64)]: sums of counts * probs
    int *seen;           // [rows]
    int *counts;         // [rows, E]
    float *probs;        // [rows, E]
};

struct BalanceArgs {
    const float *logits;      // [T, E]
    const int64_t *topk_idx;  // [T, K]
    const int32_t *seq_off;   // [S + 1], or null (one sequence of all tokens)
    int T, E, K, S;
    float *loss;              // [1]
    int32_t *counts;          // [S, E]
    float *probs;             // [S, E]
    int32_t *num_tokens;      // [S + 1]
    void *ws_base;            // workspace
    BalanceWs ws;             // its parts (set by the launcher)
    int *err;
};

size_t balance_workspace_bytes(int T, int E, int S);
hipError_t launch_balance(const BalanceArgs &a, bool sigmoid, hipStream_t stream);

struct RouteBwdArgs {
    const float *logits;      // [T, E]
    const int64_t *topk_idx;  // [T, K]
    const float *dtopk_w;     // [T, K], or null
    const int32_t *counts;    // [S, E], or null
    const int32_t *num_tokens;  // [S + 1] with counts
    const float *dloss;       // [1] with counts
    const int32_t *seq_off;   // [S + 1], or null
    int T, E, K, S;
    float scale;
    float *dlogits;           // [T, E]
    int *err;
};

hipError_t launch_route_backward(const RouteBwdArgs &a, bool sigmoid, bool normalize,
                                 hipStream_t stream);

struct CombineBwdArgs {
    const uint16_t *dout;  // [T, h] bf16
    const uint16_t *y;     // [n_rows, h] bf16, or null without dtopk_w
    int64_t n_rows;
    int h, T, K;
    const float *topk_w;   // [T, K]
    const int32_t *pos;    // [T, K]
    uint16_t *dy;          // [n_rows, h] bf16, or null
    float *dtopk_w;        // [T, K], or null
    int *err;
};

hipError_t launch_combine_backward(const CombineBwdArgs &a, hipStream_t stream);

}  // namespace epx
