// qaff_rope_append: rotary positions of the step's q and k and the write of k and v into the cache.
//
// Every value is read and written once, so the traffic bounds it. A token's angles serve all its
// heads: a workgroup takes one token, computes rot / 2 sines and cosines once into LDS and then
// walks the token's pairs.
#include "mfma16.h"
#include "paged.h"

namespace qaff {
namespace {

constexpr int kRopeThreads = 256;

// Sine and cosine of pos * f. The product is exact in float64 (31 + 24 bits fit only nearly: 53),
// and so is its reduction to a fraction of a turn, up to that rounding: at 2^20 positions a float32
// angle would already be off by 2^-4 rad. The remaining fraction, at most half a turn, needs no more
// than float32.
__device__ __forceinline__ float2 angle_of(int32_t pos, float f) {
    const double turns = (double)pos * (double)f * 0.15915494309189533577;  // 1 / (2 pi)
    const float r = (float)(turns - __builtin_rint(turns));
    float s, c;
    sincospif(2.0f * r, &s, &c);
    return make_float2(c, s);
}

__device__ __forceinline__ int axis_of(const RopeArgs& a, int i) {
    if (a.axes == 1) return 0;
    if (a.interleaved) {
        const int x = i % a.axes;
        return i / a.axes < a.sections[x] ? x : 0;
    }
    int x = 0, end = a.sections[0];
    while (i >= end && x + 1 < a.axes) end += a.sections[++x];
    return x;
}

// One value at a time: any strides and alignment, any head size.
template <bool F16>
__global__ __launch_bounds__(kRopeThreads) void rope_scalar_kernel(RopeArgs a, int traditional) {
    __shared__ float2 turn[256];
    const int64_t t = blockIdx.x;
    for (int i = threadIdx.x; i < a.half; i += kRopeThreads)
        turn[i] = angle_of(a.positions[axis_of(a, i) * a.tokens + t], a.inv_freq[i]);
    __syncthreads();
    const int64_t slot = a.kv_heads > 0 ? a.slots[t] : -1;
    const bool store = slot >= 0 && slot < a.total_slots;
    const int64_t page = slot >> a.page_shift, off = slot & ((1 << a.page_shift) - 1);
    const int units = a.dim - a.half;  // pairs, then the values that pass
    const int rows = a.heads + 2 * a.kv_heads;
    for (int u = threadIdx.x; u < rows * units; u += kRopeThreads) {
        const int row = u / units, i = u - row * units;
        const uint16_t* src;
        uint16_t* dst;
        if (row < a.heads) {
            src = a.q + t * a.q_ts + row * a.q_hs;
            dst = a.q_out + (t * a.heads + row) * a.dim;
        } else {
            if (!store) continue;
            const bool value = row >= a.heads + a.kv_heads;
            const int h = row - a.heads - (value ? a.kv_heads : 0);
            src = value ? a.v + t * a.v_ts + h * a.v_hs : a.k + t * a.k_ts + h * a.k_hs;
            dst = (value ? a.v_cache : a.k_cache) + page * a.page_stride + (((int64_t)h << a.page_shift) + off) * a.dim;
        }
        if (i >= a.half) {
            dst[i + a.half] = src[i + a.half];
            continue;
        }
        const int d0 = traditional ? 2 * i : i, d1 = traditional ? 2 * i + 1 : i + a.half;
        if (row >= a.heads + a.kv_heads) {
            dst[d0] = src[d0];
            dst[d1] = src[d1];
        } else {
            const float x = half_to_f32<F16>(src[d0]), y = half_to_f32<F16>(src[d1]);
            const float2 cs = turn[i];
            dst[d0] = f32_to_half_bits<F16>(x * cs.x - y * cs.y);
            dst[d1] = f32_to_half_bits<F16>(y * cs.x + x * cs.y);
        }
    }
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs& a, bool f16, bool traditional, hipStream_t stream) {
    const unsigned grid = (unsigned)a.tokens;
    if (f16) rope_scalar_kernel<true><<<grid, kRopeThreads, 0, stream>>>(a, traditional);
    else rope_scalar_kernel<false><<<grid, kRopeThreads, 0, stream>>>(a, traditional);
    return hipGetLastError();
}

}  // namespace qaff
