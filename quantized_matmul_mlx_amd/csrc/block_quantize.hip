// Quantization to 8-bit floating point (e4m3) with a float32 scale for each block: 128 columns of a row
// (activations), or 128 x 128 (weights).
//
//   scale = largest |x| of the block / 448, code = e4m3(x / scale), both quotients float32 rounded to
//   nearest even, the code the nearest e4m3 value of the quotient, of two the even one; a scale of 0
//   gives codes 0. A NaN or an infinity in a block makes all of the block's products NaN: its scale is NaN
//   or infinite.
//
// Bound by memory: one pass, 16 lanes of 8 values a block; [8192, 4096] bf16 by rows 20.4 us (101 MB, 4.95 TB/s), a weight
// of [4096, 14336] in blocks of 128 x 128 35.3 us (176 MB, 5.0 TB/s), a copy's rate.
#include "ffn.h"
#include "qaff_device.h"

namespace qaff {
namespace {

constexpr float kTop = 448.0f;  // the largest e4m3 value

typedef uint32_t u32x2w __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4w __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2b __attribute__((ext_vector_type(2), aligned(1)));

// The larger magnitude, NaN if either is one.
__device__ __forceinline__ float wider(float a, float b) {
    return (b != b || b > a) ? b : a;  // a NaN in a stays: no comparison with it is true
}

template <int CTRL> __device__ __forceinline__ float from_lane(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}

// Eight values from element i on, of which `n` are there (the others 0).
template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i, int n, float (&v)[8]) {
    if (n >= 8) {
        if constexpr (DT == 0) {
            const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + i);
            const u32x4 b = *reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + i + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = __uint_as_float(a[e]);
                v[4 + e] = __uint_as_float(b[e]);
            }
        } else {
            const u32x4w a = *reinterpret_cast<const u32x4w*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (DT == 1) {
                    v[2 * e] = __uint_as_float(a[e] << 16);
                    v[2 * e + 1] = __uint_as_float(a[e] & 0xffff0000u);
                } else {
                    v[2 * e] = (float)__builtin_bit_cast(f16x2, (uint32_t)a[e]).x;
                    v[2 * e + 1] = (float)__builtin_bit_cast(f16x2, (uint32_t)a[e]).y;
                }
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? load_as_f32(p, (size_t)(i + e), DT) : 0.f;
    }
}

// x / scale as float32 rounds it, from r = 1 / scale (rounded): q = v r is off by a step and a half at most, and two
// corrections q + (v - q scale) r, whose remainder a fused multiply-add forms exactly, first bring it within a step and
// then to the rounded quotient itself. Five instructions for about ten of the division, which is left to scales whose
// remainders could leave float32's range.
struct Scale {
    float s, r;
    bool plain;  // the corrections hold
};
__device__ __forceinline__ Scale make_scale(float s) {
    return Scale{s, 1.f / s, s >= 0x1p-90f && s <= 0x1p90f};
}

// e4m3 of v / scale, four at a time.
__device__ __forceinline__ uint32_t codes4(const float* v, const Scale& c) {
    float q[4];
    if (c.plain) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            q[e] = v[e] * c.r;
#pragma unroll
            for (int n = 0; n < 2; ++n) q[e] = __builtin_fmaf(__builtin_fmaf(-q[e], c.s, v[e]), c.r, q[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float d = v[e] / c.s;
            // a scale far below float32's smallest normal value is off by more than a rounding: no code past 448
            q[e] = c.s == 0.f ? 0.f : d != d ? d : fminf(fmaxf(d, -kTop), kTop);
        }
    }
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], r, true);
}

__device__ __forceinline__ void store8(uint8_t* p, int n, const float (&v)[8], const Scale& scale) {
    const uint32_t lo = codes4(v, scale), hi = codes4(v + 4, scale);
    if (n >= 8) {
        *reinterpret_cast<u32x2b*>(p) = u32x2b{lo, hi};
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = (uint8_t)((e < 4 ? lo : hi) >> (8 * (e & 3)));
    }
}

// A row's blocks: 16 lanes of 8 values a block, 16 blocks a workgroup, one after another over the rows.
template <int DT>
__global__ __launch_bounds__(256) void quantize_rows_kernel(BlockQuantArgs a, int64_t kb) {
    const int64_t b = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
    if (b >= a.rows * kb) return;  // 16 lanes leave together
    const int64_t row = b / kb, block = b % kb;
    const int64_t col = block * kBlock + threadIdx.x % 16 * 8;
    const int n = (int)min((int64_t)8, max((int64_t)0, a.cols - col));
    float v[8];
    load8<DT>(a.x, row * a.row_stride + col, n, v);
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = wider(top, fabsf(v[e]));
    top = wider(top, from_lane<0xB1>(top));   // lane ^ 1
    top = wider(top, from_lane<0x4E>(top));   // lane ^ 2
    top = wider(top, from_lane<0x141>(top));  // mirrored in 8 lanes
    top = wider(top, from_lane<0x140>(top));  // and in 16
    const float scale = top / kTop;
    if (n > 0) store8(a.codes + row * a.cols + col, n, v, make_scale(scale));
    if (threadIdx.x % 16 == 0) a.scales[b] = scale;
}

// A 128 x 128 block a workgroup: thread t has 8 columns of rows t / 16, + 16, ...
template <int DT>
__global__ __launch_bounds__(256) void quantize_tiles_kernel(BlockQuantArgs a, int64_t kb) {
    __shared__ float most[4];
    const int64_t row0 = (int64_t)blockIdx.y * kBlock + threadIdx.x / 16;
    const int64_t col = (int64_t)blockIdx.x * kBlock + threadIdx.x % 16 * 8;
    const int n = (int)min((int64_t)8, max((int64_t)0, a.cols - col));
    float v[8][8], top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = row0 + 16 * i;
        load8<DT>(a.x, row * a.row_stride + col, row < a.rows ? n : 0, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = wider(top, fabsf(v[i][e]));
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = wider(top, __shfl_xor(top, d, 64));
    if (threadIdx.x % 64 == 0) most[threadIdx.x / 64] = top;
    __syncthreads();
    const float scale = wider(wider(most[0], most[1]), wider(most[2], most[3])) / kTop;
    const Scale quotient = make_scale(scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = row0 + 16 * i;
        if (row < a.rows && n > 0) store8(a.codes + row * a.cols + col, n, v[i], quotient);
    }
    if (threadIdx.x == 0) a.scales[blockIdx.y * kb + blockIdx.x] = scale;
}

template <int DT>
hipError_t launch(const BlockQuantArgs& a, bool by_row, hipStream_t stream) {
    const int64_t kb = (a.cols + kBlock - 1) / kBlock;
    if (by_row) {
        const int64_t blocks = (a.rows * kb + 15) / 16;
        quantize_rows_kernel<DT><<<dim3((unsigned)blocks), dim3(256), 0, stream>>>(a, kb);
        return hipGetLastError();
    }
    const int64_t rb = (a.rows + kBlock - 1) / kBlock;
    for (int64_t r0 = 0; r0 < rb; r0 += 65535) {  // a grid's second axis holds 65535
        BlockQuantArgs p = a;
        const int64_t n = rb - r0 < 65535 ? rb - r0 : 65535, at = r0 * kBlock;
        p.x = static_cast<const char*>(a.x) + at * a.row_stride * (DT == 0 ? 4 : 2);
        p.codes += at * a.cols;
        p.scales += r0 * kb;
        p.rows -= at;
        quantize_tiles_kernel<DT><<<dim3((unsigned)kb, (unsigned)n), dim3(256), 0, stream>>>(p, kb);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_block_quantize(const BlockQuantArgs& a, bool by_row, hipStream_t stream) {
    if (a.dtype == 0) return launch<0>(a, by_row, stream);
    if (a.dtype == 1) return launch<1>(a, by_row, stream);
    return launch<2>(a, by_row, stream);
}

}  // namespace qaff
