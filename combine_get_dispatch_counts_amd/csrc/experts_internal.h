// experts_internal.h -- launcher interface of the experts' arithmetic (weight
// quantiser, grouped products, whole layer for a few tokens). Arguments are
// checked in epx_api.hip; launchers assume valid shapes and return the HIP
// launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace epx {

struct QuantizeArgs {
    const uint16_t *w;  // [E, N, K] bf16
    int E, N, K;
    uint8_t *codes;     // [E, N, K]
    float *scales;      // [E, ceil(N/128), K/128]
};

hipError_t launch_quantize_weights(const QuantizeArgs &a, hipStream_t stream);

// The rows of L experts and their weights. Rows lie expert-major (off) or in
// low-latency regions (counts): region e * R_buf + s starts at row
// (e * R_buf + s) * cap and holds counts[e * R_buf + s] rows.
struct GroupedArgs {
    const void *x;        // [n_rows, K] bf16, or e4m3 codes
    const float *xs;      // FP8: [n_rows, scale_stride(K)]
    const void *w;        // [L, N, K], gated: [L, 2 N, K], gate rows then up rows
    const float *ws;      // FP8: [L, ceil(rows / 128), K / 128]
    int64_t n_rows;
    int K, N, L;          // N: output columns
    const int32_t *off;     // [L + 1], or null
    const int32_t *counts;  // [L * R_buf], or null
    int R_buf, cap;
    void *out;            // [n_rows, N] bf16; gated FP8: codes
    float *out_s;         // gated FP8: [n_rows, scale_stride(N)]
    int *err;
    int cus;              // compute units of the device
};

hipError_t launch_grouped(const GroupedArgs &a, bool fp8, bool gated, hipStream_t stream);

// The whole layer for T tokens: T <= kDecodeMaxTokens.
constexpr int kDecodeMaxTokens = 64;

struct DecodeArgs {
    const uint16_t *x;  // [T, h] bf16
    const int64_t *idx;  // [T, K]
    const float *topw;   // [T, K]
    const void *w13;     // [E, 2 f, h] bf16 or e4m3 codes
    const float *s13;    // FP8: [E, ceil(2f / 128), h / 128]
    const void *w2;      // [E, h, f]
    const float *s2;     // FP8: [E, ceil(h / 128), f / 128]
    int T, K, E, h, f;
    uint16_t *act;       // workspace [T, K, f] bf16
    uint16_t *out;       // [T, h] bf16
    int *err;
    int cus;
};

hipError_t launch_moe_decode(const DecodeArgs &a, bool fp8, hipStream_t stream);

}  // namespace epx
