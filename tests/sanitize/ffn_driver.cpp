// Runs the host code of the feed-forward entry points (api_ffn.cpp) with the launchers and the HIP runtime
// calls stubbed: refusals must launch nothing, accepted calls must launch once with what the caller passed.
// Built with AddressSanitizer and UndefinedBehaviorSanitizer.
#include "qaff.h"

#include "ffn.h"

#include <cmath>
#include <cstdio>
#include <limits>
#include <string>

static int launches = 0;
static std::string error;
static qaff::RouteArgs route;
static qaff::MoeArgs moe;
static qaff::BlockQuantArgs quant;
static qaff::BlockQmmArgs qmm;
static bool by_row, f16;
static hipError_t result = hipSuccess;

namespace qaff {
void set_error(const char* text) noexcept { error = text; }
int device_cu_count() { return 256; }
hipError_t launch_moe_route(const RouteArgs& a, hipStream_t) { return route = a, ++launches, result; }
hipError_t launch_moe_ffn(const MoeArgs& a, bool f, hipStream_t) { return moe = a, f16 = f, ++launches, result; }
size_t moe_ffn_workspace(int64_t tokens, int64_t, int64_t, int64_t, int64_t) { return (size_t)tokens * 64; }
hipError_t launch_block_quantize(const BlockQuantArgs& a, bool r, hipStream_t) {
    return quant = a, by_row = r, ++launches, result;
}
hipError_t launch_block_qmm(const BlockQmmArgs& a, hipStream_t) { return qmm = a, ++launches, result; }
}  // namespace qaff
hipError_t hipStreamSynchronize(hipStream_t) { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "stub"; }

#define CHECK(x)                                                     \
    do {                                                             \
        if (!(x)) {                                                  \
            std::printf("line %d: %s (%s)\n", __LINE__, #x, error.c_str()); \
            return 1;                                                \
        }                                                            \
    } while (0)

int main() {
    const int64_t big = std::numeric_limits<int64_t>::max(), low = std::numeric_limits<int64_t>::min();
    int32_t* i32 = reinterpret_cast<int32_t*>(0x10000);
    uint32_t* u32 = reinterpret_cast<uint32_t*>(0x10000);
    uint8_t* u8 = reinterpret_cast<uint8_t*>(0x10000);
    float* f32 = reinterpret_cast<float*>(0x10000);
    void* p = f32;
    int done = 0;

    auto choose = [&](int64_t tokens, int64_t experts, int64_t stride, int64_t top_k) {
        return qaff_moe_route(p, QAFF_F16, tokens, experts, stride, f32, 1, top_k, 1, 2.5f, f32, i32, nullptr);
    };
    CHECK(choose(3, 8, 10, 2) == QAFF_OK && launches == ++done);
    CHECK(route.tokens == 3 && route.experts == 8 && route.row_stride == 10 && route.top_k == 2 && route.dtype == 2 &&
          route.sigmoid && route.renormalize && route.scale == 2.5f);
    for (int64_t v : {big, low}) {
        CHECK(choose(v, 8, 8, 2) != QAFF_OK && choose(3, v, 8, 2) != QAFF_OK && choose(3, 8, v, 2) != QAFF_OK &&
              choose(3, 8, 8, v) != QAFF_OK);
    }
    CHECK(launches == done);

    auto layer = [&](int64_t tokens, int64_t width, int64_t hidden, int64_t top_k, int64_t experts, int32_t group, int32_t bits,
                     size_t bytes) {
        return qaff_moe_ffn(p, QAFF_F16, tokens, width, hidden, i32, f32, top_k, experts, u32, p, p, u32, p, p, u32, p, p, group,
                            bits, nullptr, p, bytes, p, nullptr);
    };
    CHECK(layer(3, 128, 64, 2, 4, 32, 4, 192) == QAFF_OK && launches == ++done);
    CHECK(f16 && moe.tokens == 3 && moe.width == 128 && moe.hidden == 64 && moe.top_k == 2 && moe.experts == 4 &&
          moe.group == 32 && moe.bits == 4 && moe.workspace == p);
    CHECK(layer(3, 128, 0, 2, 4, 32, 4, 0) == QAFF_OK && launches == ++done && moe.top_k == 0);  // y = resid
    CHECK(layer(3, 128, 64, 2, 4, 32, 4, 191) == QAFF_ERR_INVALID_ARGUMENT);
    for (int64_t v : {big, low, big - 31}) {
        CHECK(layer(v, 128, 64, 2, 4, 32, 4, 192) != QAFF_OK && layer(3, v, 64, 2, 4, 32, 4, 192) != QAFF_OK &&
              layer(3, 128, v, 2, 4, 32, 4, 192) != QAFF_OK && layer(3, 128, 64, v, 4, 32, 4, 192) != QAFF_OK &&
              layer(3, 128, 64, 2, v, 32, 4, 192) != QAFF_OK);
        CHECK(qaff_moe_ffn_workspace_size(v, v, v, v, v, 32, 4) == 0);
    }
    CHECK(layer(3, 128, 64, 2, 4, -2147483647 - 1, 4, 192) != QAFF_OK && layer(3, 128, 64, 2, 4, 32, 2147483647, 192) != QAFF_OK);
    CHECK(launches == done);

    auto quantize = [&](int64_t rows, int64_t cols, int64_t stride, int32_t block) {
        return qaff_block_quantize(p, QAFF_BF16, rows, cols, stride, block, u8, f32, nullptr);
    };
    CHECK(quantize(5, 200, 256, 1) == QAFF_OK && launches == ++done && by_row && quant.row_stride == 256 && quant.cols == 200);
    CHECK(quantize(5, 200, 200, 128) == QAFF_OK && launches == ++done && !by_row && quant.rows == 5);
    for (int64_t v : {big, low})
        CHECK(quantize(v, 200, 200, 1) != QAFF_OK && quantize(5, v, v, 1) != QAFF_OK && quantize(5, 200, v, 1) != QAFF_OK);
    CHECK(launches == done);

    auto product = [&](int64_t m, int64_t n, int64_t k) {
        return qaff_block_qmm(u8, f32, m, u8, f32, n, k, p, QAFF_F32, nullptr);
    };
    CHECK(product(3, 64, 256) == QAFF_OK && launches == ++done && qmm.m == 3 && qmm.n == 64 && qmm.k == 256 && qmm.y == p);
    CHECK(product(3, 64, 0) == QAFF_OK && launches == ++done && qmm.k == 0);
    for (int64_t v : {big, low})
        CHECK(product(v, 64, 256) != QAFF_OK && product(3, v, 256) != QAFF_OK && product(3, 64, v) != QAFF_OK);
    CHECK(launches == done);

    result = hipErrorLaunchFailure;
    CHECK(product(3, 64, 256) == QAFF_ERR_DEVICE && error.find("stub") != std::string::npos);
    result = hipErrorInvalidConfiguration;
    CHECK(quantize(5, 200, 256, 1) == QAFF_ERR_UNSUPPORTED);
    std::printf("all checks passed\n");
    return 0;
}
