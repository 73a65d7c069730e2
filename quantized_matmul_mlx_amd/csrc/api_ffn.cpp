// The C ABI of the feed-forward operators (include/qaff.h): argument checks, all on the host before any
// launch, and dispatch. The chosen experts live on the device and cannot be checked here: the kernels pass
// over those that are not there.
#include "api_util.h"
#include "ffn.h"

#include <cmath>

namespace {

using qaff::after_launch;
using qaff::aligned;
using qaff::check_ptr;
using qaff::fail;

constexpr int64_t k2G = 1LL << 31;

bool any_dtype(qaff_dtype d) { return d == QAFF_F32 || d == QAFF_BF16 || d == QAFF_F16; }
uintptr_t esize(qaff_dtype d) { return d == QAFF_F32 ? 4 : 2; }

constexpr int64_t kMaxColumns = 32768;  // of an expert's weights: a row of x and its groups' sums fit a workgroup

constexpr int64_t kMaxBlockK = 1 << 18;  // a workgroup holds the scales of 16 rows of x

qaff_status check_moe_sizes(const char* op, int64_t tokens, int64_t width, int64_t hidden, int64_t top_k,
                            int64_t experts, int32_t group_size, int32_t bits) {
    if (bits < 1 || bits > 8 || bits == 7)
        return fail(QAFF_ERR_UNSUPPORTED, "%s: %d bits are not supported (1, 2, 3, 4, 5, 6 or 8)", op, bits);
    if (group_size != 32 && group_size != 64 && group_size != 128)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: group size %d is not supported (32, 64 or 128)", op, group_size);
    if (tokens < 0 || width < 0 || hidden < 0 || top_k < 0 || experts < 0)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: negative size", op);
    if (width % group_size != 0 || hidden % group_size != 0)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: width %lld and hidden %lld must be multiples of the group size %d", op,
                    (long long)width, (long long)hidden, group_size);
    if (width > kMaxColumns || hidden > kMaxColumns)
        return fail(QAFF_ERR_UNSUPPORTED, "%s: width or hidden above %lld", op, (long long)kMaxColumns);
    if (experts > 65535) return fail(QAFF_ERR_UNSUPPORTED, "%s: more than 65535 experts", op);
    if (top_k > 65535 || tokens >= k2G || tokens * top_k >= k2G)
        return fail(QAFF_ERR_UNSUPPORTED, "%s: 2^31 tokens or (token, expert) pairs or more", op);
    if (tokens * width >= 1LL << 34) return fail(QAFF_ERR_UNSUPPORTED, "%s: 2^34 outputs or more", op);
    return QAFF_OK;
}

qaff_status check_expert_weight(const char* op, const uint32_t* packed, const void* scales, const void* biases) {
    qaff_status st = check_ptr(op, "packed codes", packed, 4);
    if (st == QAFF_OK) st = check_ptr(op, "scales", scales, 2);
    if (st == QAFF_OK) st = check_ptr(op, "biases", biases, 2);
    return st;
}

}  // namespace

extern "C" {

qaff_status qaff_moe_route(const void* logits, qaff_dtype dtype, int64_t tokens, int64_t experts, int64_t row_stride,
                           const float* bias, int32_t sigmoid, int64_t top_k, int32_t renormalize, float scale,
                           float* weights, int32_t* chosen, hipStream_t stream) {
    const char* op = "qaff_moe_route";
    qaff::set_error("");
    if (!any_dtype(dtype)) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d", op, (int)dtype);
    if (tokens < 0 || experts < 0 || row_stride < 0) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: negative size", op);
    if (top_k < 0 || top_k > experts)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: %lld of %lld experts", op, (long long)top_k, (long long)experts);
    if (!std::isfinite(scale)) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: the factor is not finite", op);
    if (experts > qaff::kRouteMaxExperts || top_k > qaff::kRouteMaxChosen)
        return fail(QAFF_ERR_UNSUPPORTED, "%s: %lld of %lld experts (at most %d of %d)", op, (long long)top_k,
                    (long long)experts, qaff::kRouteMaxChosen, qaff::kRouteMaxExperts);
    if (tokens >= 1LL << 26) return fail(QAFF_ERR_UNSUPPORTED, "%s: 2^26 tokens or more", op);
    if (tokens == 0 || top_k == 0) return QAFF_OK;
    if (tokens > 1 && row_stride >= 1LL << 32) return fail(QAFF_ERR_UNSUPPORTED, "%s: rows 2^32 elements apart", op);
    qaff_status st = check_ptr(op, "logits", logits, esize(dtype));
    if (st == QAFF_OK) st = check_ptr(op, "weights", weights, 4);
    if (st == QAFF_OK) st = check_ptr(op, "chosen", chosen, 4);
    if (st != QAFF_OK) return st;
    if (bias && !aligned(bias, 4)) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: bias must be 4-byte aligned", op);
    qaff::RouteArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.weights = weights;
    a.chosen = chosen;
    a.tokens = tokens;
    a.row_stride = row_stride;
    a.experts = (int)experts;
    a.top_k = (int)top_k;
    a.dtype = (int)dtype;
    a.sigmoid = sigmoid != 0;
    a.renormalize = renormalize != 0;
    a.scale = scale;
    return after_launch(op, qaff::launch_moe_route(a, stream), stream);
}

size_t qaff_moe_ffn_workspace_size(int64_t tokens, int64_t width, int64_t hidden, int64_t top_k, int64_t experts,
                                   int32_t group_size, int32_t bits) {
    if (check_moe_sizes("qaff_moe_ffn_workspace_size", tokens, width, hidden, top_k, experts, group_size, bits) != QAFF_OK)
        return 0;
    if (tokens == 0 || width == 0 || hidden == 0 || top_k == 0 || experts == 0) return 0;
    return qaff::moe_ffn_workspace(tokens, width, hidden, top_k, experts);
}

qaff_status qaff_moe_ffn(const void* x, qaff_dtype dtype, int64_t tokens, int64_t width, int64_t hidden,
                         const int32_t* chosen, const float* weights, int64_t top_k, int64_t experts,
                         const uint32_t* gate_packed, const void* gate_scales, const void* gate_biases,
                         const uint32_t* up_packed, const void* up_scales, const void* up_biases,
                         const uint32_t* down_packed, const void* down_scales, const void* down_biases,
                         int32_t group_size, int32_t bits, const void* resid, void* workspace, size_t workspace_bytes,
                         void* y, hipStream_t stream) {
    const char* op = "qaff_moe_ffn";
    qaff::set_error("");
    if (dtype != QAFF_BF16 && dtype != QAFF_F16)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: dtype %d (bf16 or float16)", op, (int)dtype);
    qaff_status st = check_moe_sizes(op, tokens, width, hidden, top_k, experts, group_size, bits);
    if (st != QAFF_OK) return st;
    if (tokens == 0 || width == 0) return QAFF_OK;
    st = check_ptr(op, "y", y, 2);
    if (st != QAFF_OK) return st;
    if (resid && !aligned(resid, 2)) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: resid must be 2-byte aligned", op);
    const bool work = hidden > 0 && top_k > 0 && experts > 0;
    if (work) {
        st = check_ptr(op, "x", x, 2);
        if (st == QAFF_OK) st = check_ptr(op, "chosen", chosen, 4);
        if (st == QAFF_OK) st = check_ptr(op, "weights", weights, 4);
        if (st == QAFF_OK) st = check_expert_weight(op, gate_packed, gate_scales, gate_biases);
        if (st == QAFF_OK) st = check_expert_weight(op, up_packed, up_scales, up_biases);
        if (st == QAFF_OK) st = check_expert_weight(op, down_packed, down_scales, down_biases);
        if (st == QAFF_OK) st = check_ptr(op, "workspace", workspace, 16);
        if (st != QAFF_OK) return st;
        const size_t need = qaff::moe_ffn_workspace(tokens, width, hidden, top_k, experts);
        if (workspace_bytes < need)
            return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: a workspace of %zu bytes, %zu needed", op, workspace_bytes, need);
    }
    qaff::MoeArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.resid = static_cast<const uint16_t*>(resid);
    a.y = static_cast<uint16_t*>(y);
    a.chosen = chosen;
    a.weights = weights;
    a.gate = {gate_packed, static_cast<const uint16_t*>(gate_scales), static_cast<const uint16_t*>(gate_biases)};
    a.up = {up_packed, static_cast<const uint16_t*>(up_scales), static_cast<const uint16_t*>(up_biases)};
    a.down = {down_packed, static_cast<const uint16_t*>(down_scales), static_cast<const uint16_t*>(down_biases)};
    a.tokens = tokens;
    a.width = (int)width;
    a.hidden = (int)hidden;
    a.top_k = work ? (int)top_k : 0;
    a.experts = (int)experts;
    a.group = group_size;
    a.bits = bits;
    a.workspace = workspace;
    return after_launch(op, qaff::launch_moe_ffn(a, dtype == QAFF_F16, stream), stream);
}

qaff_status qaff_block_quantize(const void* x, qaff_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride,
                                int32_t block_rows, uint8_t* codes, float* scales, hipStream_t stream) {
    const char* op = "qaff_block_quantize";
    qaff::set_error("");
    if (!any_dtype(dtype)) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d", op, (int)dtype);
    if (block_rows != 1 && block_rows != qaff::kBlock)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: blocks of %d rows are not supported (1 or 128)", op, block_rows);
    if (rows < 0 || cols < 0 || row_stride < 0) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: negative size", op);
    if (rows > 1 && row_stride < cols)
        return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: rows %lld elements apart overlap", op, (long long)row_stride);
    if (rows == 0 || cols == 0) return QAFF_OK;
    if (rows >= 1LL << 32 || cols >= 1LL << 31 || row_stride >= 1LL << 31 ||
        rows * ((cols + qaff::kBlock - 1) / qaff::kBlock) >= 1LL << 28)
        return fail(QAFF_ERR_UNSUPPORTED, "%s: 2^28 blocks of a row or more", op);
    qaff_status st = check_ptr(op, "x", x, esize(dtype));
    if (st == QAFF_OK) st = check_ptr(op, "codes", codes, 1);
    if (st == QAFF_OK) st = check_ptr(op, "scales", scales, 4);
    if (st != QAFF_OK) return st;
    qaff::BlockQuantArgs a{};
    a.x = x;
    a.codes = codes;
    a.scales = scales;
    a.rows = rows;
    a.cols = cols;
    a.row_stride = row_stride;
    a.dtype = (int)dtype;
    return after_launch(op, qaff::launch_block_quantize(a, block_rows == 1, stream), stream);
}

qaff_status qaff_block_qmm(const uint8_t* x, const float* x_scales, int64_t m, const uint8_t* w, const float* w_scales,
                           int64_t n, int64_t k, void* y, qaff_dtype y_dtype, hipStream_t stream) {
    const char* op = "qaff_block_qmm";
    qaff::set_error("");
    if (!any_dtype(y_dtype)) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d", op, (int)y_dtype);
    if (m < 0 || n < 0 || k < 0) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: negative size", op);
    if (m >= k2G || n >= 1LL << 28 || k > kMaxBlockK)
        return fail(QAFF_ERR_UNSUPPORTED, "%s: 2^31 rows of x or 2^28 rows of w or more, or above %lld columns", op,
                    (long long)kMaxBlockK);
    if (m == 0 || n == 0) return QAFF_OK;
    qaff_status st = check_ptr(op, "y", y, esize(y_dtype));
    if (st == QAFF_OK && k > 0) {
        st = check_ptr(op, "x", x, 1);
        if (st == QAFF_OK) st = check_ptr(op, "x_scales", x_scales, 4);
        if (st == QAFF_OK) st = check_ptr(op, "w", w, 1);
        if (st == QAFF_OK) st = check_ptr(op, "w_scales", w_scales, 4);
    }
    if (st != QAFF_OK) return st;
    qaff::BlockQmmArgs a{};
    a.x = x;
    a.w = w;
    a.x_scales = x_scales;
    a.w_scales = w_scales;
    a.y = y;
    a.m = m;
    a.n = n;
    a.k = k;
    a.dtype = (int)y_dtype;
    return after_launch(op, qaff::launch_block_qmm(a, stream), stream);
}

}  // extern "C"
