// Runs the host code of the paged-cache entry points (api_paged.cpp) with the launchers and the HIP
// runtime calls stubbed: refusals must launch nothing, accepted calls must launch once with what the
// caller passed. Built with AddressSanitizer and UndefinedBehaviorSanitizer.
#include "qaff.h"

#include "paged.h"

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <limits>
#include <string>

static int launches = 0;
static std::string error;
static qaff::AttnArgs attn;
static qaff::RopeArgs rope;
static hipError_t result = hipSuccess;

namespace qaff {
void set_error(const char* text) noexcept { error = text; }
int device_cu_count() { return 256; }
hipError_t launch_paged_plan(const PlanArgs&, hipStream_t) { return ++launches, result; }
hipError_t launch_rope_append(const RopeArgs& a, bool, bool, hipStream_t) { return rope = a, ++launches, result; }
hipError_t launch_paged_attention(const AttnArgs& a, bool, int64_t, hipStream_t) { return attn = a, ++launches, result; }
size_t paged_attention_workspace(int64_t tokens, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) {
    return tokens > 100 ? 64 : 0;
}
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
    const int64_t big = std::numeric_limits<int64_t>::max();
    int32_t* i32 = reinterpret_cast<int32_t*>(0x10000);
    int64_t* i64 = reinterpret_cast<int64_t*>(0x10000);
    float* f32 = reinterpret_cast<float*>(0x10000);
    void* p = f32;
    auto plan = [&](int64_t requests, int64_t width, int64_t tokens, int32_t page) {
        return qaff_paged_plan(i32, i32, requests, i32, 4, i32, width, page, tokens, i32, i32, i32, i64, i32, nullptr);
    };
    CHECK(plan(2, 3, 5, 16) == QAFF_OK && launches == 1);
    CHECK(plan(big, 3, 5, 16) == QAFF_ERR_UNSUPPORTED && plan(2, 3, big, 16) == QAFF_ERR_UNSUPPORTED);
    CHECK(plan(2, -big - 1, 5, 16) == QAFF_ERR_INVALID_ARGUMENT && plan(2, 3, 5, -2147483647 - 1) == QAFF_ERR_UNSUPPORTED);
    CHECK(launches == 1);

    const int32_t sections[4] = {16, 8, 8, 0};
    const int32_t huge[4] = {2147483647, 2147483647, 2147483647, 2147483647};
    auto turn = [&](int64_t tokens, int64_t dim, int64_t pages, int64_t stride, int32_t axes, const int32_t* sec, int32_t inter) {
        return qaff_rope_append(p, p, p, QAFF_BF16, tokens, 4, 2, dim, 256, 64, 128, 64, 128, 64, i32, axes, sec, inter, 0, f32,
                                64, i64, p, p, pages, stride, 16, p, nullptr);
    };
    launches = 0;
    CHECK(turn(3, 64, 4, 2048, 1, nullptr, 0) == QAFF_OK && launches == 1 && rope.half == 32 && rope.sections[0] == 32);
    CHECK(rope.total_slots == 64 && rope.page_shift == 4);
    // interleaved, the 8 pairs of axis 1 are pairs 1, 5 .. 29 of 32; a ninth would be pair 33
    const int32_t too_many[4] = {8, 9, 8, 7};
    CHECK(turn(3, 64, 4, 2048, 4, sections, 1) == QAFF_OK && launches == 2 && rope.interleaved == 1);
    CHECK(turn(3, 64, 4, 2048, 4, too_many, 1) == QAFF_ERR_INVALID_ARGUMENT && launches == 2);
    CHECK(turn(3, 64, 4, 2048, 4, too_many, 0) == QAFF_OK && launches == 3);
    CHECK(turn(3, 64, 4, 2048, 4, huge, 1) == QAFF_ERR_INVALID_ARGUMENT && turn(3, 64, 4, 2048, 4, huge, 0) == QAFF_ERR_INVALID_ARGUMENT);
    CHECK(turn(big, 64, 4, 2048, 1, nullptr, 0) == QAFF_ERR_UNSUPPORTED && turn(3, big, 4, 2048, 1, nullptr, 0) == QAFF_ERR_UNSUPPORTED);
    CHECK(turn(3, 64, big, 2048, 1, nullptr, 0) == QAFF_ERR_UNSUPPORTED && turn(3, 64, 4, 2047, 1, nullptr, 0) == QAFF_ERR_INVALID_ARGUMENT);
    CHECK(launches == 3);

    auto attend = [&](int64_t tokens, int64_t heads, int64_t kv_heads, int64_t width, float scale, void* ws, size_t bytes) {
        return qaff_paged_attention(p, QAFF_F16, tokens, heads, 256, 64, p, p, 4, 4096, kv_heads, 64, 16, i32, width, i32, i32, 2,
                                    tokens, scale, 1, 0, ws, bytes, p, nullptr, nullptr);
    };
    launches = 0;
    CHECK(attend(3, 8, 2, 3, 0.125f, nullptr, 0) == QAFF_OK && launches == 1 && attn.group == 4 && attn.table_keys == 48);
    CHECK(attend(101, 8, 2, 3, 0.125f, p, 64) == QAFF_OK && launches == 2 && attn.partial == p);
    CHECK(attend(101, 8, 2, 3, 0.125f, p, 63) == QAFF_ERR_INVALID_ARGUMENT && attend(101, 8, 2, 3, 0.125f, nullptr, 64) == QAFF_ERR_INVALID_ARGUMENT);
    CHECK(attend(big, 8, 2, 3, 0.125f, p, 64) == QAFF_ERR_UNSUPPORTED && attend(3, big, 1, 3, 0.125f, p, 64) == QAFF_ERR_UNSUPPORTED);
    CHECK(attend(3, 8, 2, big, 0.125f, p, 64) == QAFF_ERR_UNSUPPORTED && attend(3, 8, 0, 3, 0.125f, p, 64) == QAFF_ERR_INVALID_ARGUMENT);
    CHECK(attend(3, 8, 2, 3, std::nanf(""), p, 64) == QAFF_ERR_INVALID_ARGUMENT && launches == 2);
    CHECK(qaff_paged_attention_workspace_size(big, 8, 2, 64, 16, big, big, big) == 0);
    result = hipErrorInvalidConfiguration;
    CHECK(attend(3, 8, 2, 3, 0.125f, nullptr, 0) == QAFF_ERR_UNSUPPORTED);
    result = hipErrorUnknown;
    CHECK(attend(3, 8, 2, 3, 0.125f, nullptr, 0) == QAFF_ERR_DEVICE && plan(2, 3, 5, 16) == QAFF_ERR_DEVICE);
    std::printf("all checks passed\n");
    return 0;
}
