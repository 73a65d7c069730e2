// Internal launchers of the feed-forward operators (C ABI: api_ffn.cpp): the router of a mixture of
// experts, the layer of its experts, and quantization and products in 8-bit floating point with a
// scale for each block of 128. Arguments are validated by api_ffn.cpp; a launcher only enqueues work
// on `stream` and returns hipGetLastError() of its launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace qaff {

int device_cu_count();

constexpr int kRouteMaxExperts = 1024, kRouteMaxChosen = 64;

struct RouteArgs {
    const void* logits;
    const float* bias;  // may be null
    float* weights;     // [tokens, top_k]
    int32_t* chosen;    // [tokens, top_k]
    int64_t tokens, row_stride;
    int experts, top_k, dtype;  // dtype code: 0 float32, 1 bf16, 2 float16
    bool sigmoid, renormalize;
    float scale;
};
hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream);

// One of an expert layer's three weights: codes, scales and biases of all experts, one after another.
struct ExpertWeight {
    const uint32_t* packed;
    const uint16_t* scales;
    const uint16_t* biases;
};

struct MoeArgs {
    const uint16_t* x;       // [tokens, width]
    const uint16_t* resid;   // [tokens, width] or null
    uint16_t* y;             // [tokens, width]
    const int32_t* chosen;   // [tokens, top_k]
    const float* weights;    // [tokens, top_k]
    ExpertWeight gate, up;   // [experts, hidden, width]
    ExpertWeight down;       // [experts, width, hidden]
    int64_t tokens;
    int width, hidden, top_k, experts, group, bits;
    void* workspace;
};
hipError_t launch_moe_ffn(const MoeArgs& a, bool f16, hipStream_t stream);
// Bytes of workspace for these sizes.
size_t moe_ffn_workspace(int64_t tokens, int64_t width, int64_t hidden, int64_t top_k, int64_t experts);

// Its kernels: few rows an expert (one translation unit a type), and many.
hipError_t launch_moe_few_bf16(const MoeArgs& a, hipStream_t stream);
hipError_t launch_moe_few_f16(const MoeArgs& a, hipStream_t stream);
hipError_t launch_moe_many(const MoeArgs& a, bool f16, hipStream_t stream);

constexpr int kBlock = 128;  // columns (and, for weights, rows) that share a scale

struct BlockQuantArgs {
    const void* x;   // [rows, cols], row_stride elements apart
    uint8_t* codes;  // [rows, cols] e4m3
    float* scales;   // [ceil(rows / block_rows), ceil(cols / 128)]
    int64_t rows, cols, row_stride;
    int dtype;       // 0 float32, 1 bf16, 2 float16
};
hipError_t launch_block_quantize(const BlockQuantArgs& a, bool by_row, hipStream_t stream);

struct BlockQmmArgs {
    const uint8_t *x, *w;             // e4m3 [m, k] and [n, k]
    const float *x_scales, *w_scales; // [m, kb] and [ceil(n / 128), kb], kb = ceil(k / 128)
    void* y;                          // [m, n]
    int64_t m, n, k;
    int dtype;                        // of y: 0 float32, 1 bf16, 2 float16
};
hipError_t launch_block_qmm(const BlockQmmArgs& a, hipStream_t stream);

}  // namespace qaff
