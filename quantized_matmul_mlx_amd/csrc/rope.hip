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

// Sine and cosine of pos * f. The product (up to 31 + 24 bits of 53) and its scaling to turns each round
// once in float64: together they are off by less than 2^-52 |turns| of a turn, which is nothing beside
// the fraction's float32 rounding up to about 2^24 turns and as large as that at 2^28. At 2^20 positions
// a float32 angle would already be off by 2^-4 rad. The remaining fraction, at most half a turn, needs no
// more than float32.
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

// 16 bytes at a time. A thread's unit is a piece of 8 values, or the two pieces whose values turn
// together (values i and i + half). The loads do not wait for the angles: every thread first asks for
// its units, then the workgroup computes the token's angles, then the units turn and go out. 8192 tokens
// of 32 + 8 + 8 heads of 128: 41.7 us, 4.83 TB/s (a large copy: 4.8 to 5.2); two units a thread keep
// enough loads on their way, one starts sooner where there are few (64 tokens: 3.5 us). A token of few heads
// leaves most of its workgroup idle: 8192 tokens of 1 + 1 + 1 heads of 64 take 10.8 us for their 6.4 MB.
template <bool F16, bool TRADITIONAL, int UNITS>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a, int blocks_per_token) {
    __shared__ float2 turn[256];
    const int64_t t = blockIdx.x / blocks_per_token;
    const int u0 = (blockIdx.x - (int)t * blocks_per_token) * (kRopeThreads * UNITS) + threadIdx.x;
    const int turning = TRADITIONAL ? a.half / 4 : a.half / 8;         // units of a row that turn
    const int per_row = turning + (a.dim - 2 * a.half) / 8;            // of q and k: those, and what passes
    const int turned_rows = (a.heads + a.kv_heads) * per_row;
    const int total = turned_rows + a.kv_heads * (a.dim / 8);
    const int64_t slot = a.kv_heads > 0 ? a.slots[t] : -1;
    const bool store = slot >= 0 && slot < a.total_slots;
    const int64_t cache_at = (slot >> a.page_shift) * a.page_stride + (slot & ((1 << a.page_shift) - 1)) * a.dim;

    u32x4a x[UNITS], y[UNITS];
    uint16_t* dst[UNITS];
    int piece[UNITS];
#pragma unroll
    for (int n = 0; n < UNITS; ++n) {
        const int u = u0 + n * kRopeThreads;
        dst[n] = nullptr;
        piece[n] = -1;  // passes
        if (u >= total) continue;
        const uint16_t* src;
        int row, i;
        if (u < turned_rows) {
            row = u / per_row;
            i = u - row * per_row;
            if (i < turning) piece[n] = i;
            else i += TRADITIONAL ? 0 : turning;  // behind both pieces of the pairs
        } else {
            const int w = u - turned_rows;
            row = w / (a.dim / 8);
            i = w - row * (a.dim / 8);
            row += a.heads + a.kv_heads;
        }
        if (row < a.heads) {
            src = a.q + t * a.q_ts + row * a.q_hs;
            dst[n] = a.q_out + (t * a.heads + row) * a.dim;
        } else {
            const bool value = row >= a.heads + a.kv_heads;
            const int h = row - a.heads - (value ? a.kv_heads : 0);
            src = value ? a.v + t * a.v_ts + h * a.v_hs : a.k + t * a.k_ts + h * a.k_hs;
            if (store) dst[n] = (value ? a.v_cache : a.k_cache) + cache_at + ((int64_t)h << a.page_shift) * a.dim;
        }
        if (!dst[n]) continue;
        dst[n] += 8 * i;
        x[n] = *reinterpret_cast<const u32x4a*>(src + 8 * i);
        if (!TRADITIONAL && piece[n] >= 0) y[n] = *reinterpret_cast<const u32x4a*>(src + 8 * i + a.half);
    }
    for (int i = threadIdx.x; i < a.half; i += kRopeThreads)
        turn[i] = angle_of(a.positions[axis_of(a, i) * a.tokens + t], a.inv_freq[i]);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < UNITS; ++n) {
        if (!dst[n]) continue;
        if (piece[n] >= 0 && TRADITIONAL) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 cs = turn[4 * piece[n] + e];
                const float p = half_to_f32<F16>(x[n][e] & 0xFFFFu), q = half_to_f32<F16>(x[n][e] >> 16);
                x[n][e] = pack_half2<F16>(p * cs.x - q * cs.y, q * cs.x + p * cs.y);
            }
        } else if (piece[n] >= 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 c0 = turn[8 * piece[n] + 2 * e], c1 = turn[8 * piece[n] + 2 * e + 1];
                const float p0 = half_to_f32<F16>(x[n][e] & 0xFFFFu), p1 = half_to_f32<F16>(x[n][e] >> 16);
                const float q0 = half_to_f32<F16>(y[n][e] & 0xFFFFu), q1 = half_to_f32<F16>(y[n][e] >> 16);
                x[n][e] = pack_half2<F16>(p0 * c0.x - q0 * c0.y, p1 * c1.x - q1 * c1.y);
                y[n][e] = pack_half2<F16>(q0 * c0.x + p0 * c0.y, q1 * c1.x + p1 * c1.y);
            }
            *reinterpret_cast<u32x4a*>(dst[n] + a.half) = y[n];
        }
        *reinterpret_cast<u32x4a*>(dst[n]) = x[n];
    }
}

template <bool F16, bool TRADITIONAL>
void launch_pieces(const RopeArgs& a, hipStream_t stream) {
    const int turning = TRADITIONAL ? a.half / 4 : a.half / 8;
    const int64_t units = (int64_t)(a.heads + a.kv_heads) * (turning + (a.dim - 2 * a.half) / 8) + a.kv_heads * (a.dim / 8);
    const int64_t blocks = (units + kRopeThreads - 1) / kRopeThreads;
    if (a.tokens * blocks <= 4096) {
        rope_kernel<F16, TRADITIONAL, 1><<<(unsigned)(a.tokens * blocks), kRopeThreads, 0, stream>>>(a, (int)blocks);
    } else {
        const int64_t wide = (blocks + 1) / 2;
        rope_kernel<F16, TRADITIONAL, 2><<<(unsigned)(a.tokens * wide), kRopeThreads, 0, stream>>>(a, (int)wide);
    }
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

hipError_t launch_rope_append(const RopeArgs& a, bool f16, bool traditional, hipStream_t stream) {
    const int64_t strides = a.q_ts | a.q_hs | a.k_ts | a.k_hs | a.v_ts | a.v_hs | a.page_stride;
    const bool pieces = a.dim % 8 == 0 && (traditional ? a.half % 4 == 0 : a.half % 8 == 0) && strides % 8 == 0 &&
                        aligned16(a.q) && aligned16(a.k) && aligned16(a.v) && aligned16(a.k_cache) &&
                        aligned16(a.v_cache) && aligned16(a.q_out);
    const int64_t units = (int64_t)(a.heads + 2 * a.kv_heads) * (a.dim / 8);
    if (pieces && grid_fits(a.tokens * (units / kRopeThreads + 1), kRopeThreads)) {
        if (f16) traditional ? launch_pieces<true, true>(a, stream) : launch_pieces<true, false>(a, stream);
        else traditional ? launch_pieces<false, true>(a, stream) : launch_pieces<false, false>(a, stream);
        return hipGetLastError();
    }
    if (!grid_fits(a.tokens, kRopeThreads)) return hipErrorInvalidConfiguration;
    const unsigned grid = (unsigned)a.tokens;
    if (f16) rope_scalar_kernel<true><<<grid, kRopeThreads, 0, stream>>>(a, traditional);
    else rope_scalar_kernel<false><<<grid, kRopeThreads, 0, stream>>>(a, traditional);
    return hipGetLastError();
}

}  // namespace qaff
