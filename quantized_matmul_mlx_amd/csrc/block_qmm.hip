// Products of 8-bit floating point operands with a scale for each block of 128:
//
//   y[m, n] = sum_j xs[m, j] ws[n / 128, j] sum_{k in block j} x[m, k] w[n, k]
//
// Few rows of x: bound by the way of w from memory, so its values become float16 (exactly) for
// v_mfma_f32_16x16x32_f16, whose products and sums lose nothing that float32 holds; the 8-bit matrix
// instructions align each eight products to the largest of them and drop what lies 2^-13 below it (measured: off
// by 1.4e-5 of the sum for normal values, by 1.6e-4 of the sum of magnitudes at most for random codes).
#include "ffn.h"
#include "mfma16.h"

namespace qaff {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4b __attribute__((ext_vector_type(4), aligned(1)));

// Values 8 i .. 8 i + 7 of a lane's 32 as float16 (exact).
__device__ __forceinline__ f16x8 half8(i32x8 v, int i) {
    f16x8 o;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * i + e], 1.0f, false);
        const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 * i + e], 1.0f, true);
        o[4 * e] = lo.x;
        o[4 * e + 1] = lo.y;
        o[4 * e + 2] = hi.x;
        o[4 * e + 3] = hi.y;
    }
    return o;
}

// The sums of one block: 32 values a lane of a row of x and of a row of w, in any order of K.
__device__ __forceinline__ f32x4 block_sums(i32x8 x, i32x8 w) {
    f32x4 d = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) d = mfma16x16x32<true>(half8(x, i), half8(w, i), d);
    return d;
}

// 32 values from p on, of which n are there (the others 0).
__device__ __forceinline__ i32x8 load32(const uint8_t* p, int64_t n) {
    u32x4a lo = u32x4a{0u, 0u, 0u, 0u}, hi = lo;
    if (n >= 32) {
        const u32x4b a = *reinterpret_cast<const u32x4b*>(p), b = *reinterpret_cast<const u32x4b*>(p + 16);
        lo = u32x4a{a.x, a.y, a.z, a.w};
        hi = u32x4a{b.x, b.y, b.z, b.w};
    } else {
        for (int i = 0; i < 16; ++i) {
            if (i < n) lo[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
            if (16 + i < n) hi[i >> 2] |= (uint32_t)p[16 + i] << (8 * (i & 3));
        }
    }
    return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

constexpr int kWaves = 4;

// 16 x 16 outputs a workgroup, its waves taking the blocks of K in turn.
__global__ __launch_bounds__(64 * kWaves) void qmm_small_kernel(BlockQmmArgs a) {
    __shared__ f32x4 red[kWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * 16;
    const int64_t kb = (a.k + kBlock - 1) / kBlock;
    const uint8_t* xp = a.x + min(m0 + r, a.m - 1) * a.k + 32 * g;
    const uint8_t* wp = a.w + min(n0 + r, a.n - 1) * a.k + 32 * g;
    const float* ws = a.w_scales + n0 / kBlock * kb;
    const float* xs[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) xs[v] = a.x_scales + min(m0 + 4 * g + v, a.m - 1) * kb;
    f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int64_t j = wave; j < kb; j += kWaves) {
        const int64_t left = a.k - j * kBlock - 32 * g;
        const f32x4 d = block_sums(load32(xp + j * kBlock, left), load32(wp + j * kBlock, left));
        const float s = ws[j];
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[v] = __builtin_fmaf(xs[v][j] * s, d[v], acc[v]);
    }
    red[wave][lane] = acc;
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) acc += red[w][lane];
    if (n0 + r >= a.n) return;
#pragma unroll
    for (int v = 0; v < 4; ++v)
        if (m0 + 4 * g + v < a.m) store_from_f32(a.y, (size_t)((m0 + 4 * g + v) * a.n + n0 + r), a.dtype, acc[v]);
}

}  // namespace

size_t block_qmm_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_block_qmm(const BlockQmmArgs& a, hipStream_t stream) {
    const int64_t rows = 65535 * 16;  // a grid's second axis
    for (int64_t m0 = 0; m0 < a.m; m0 += rows) {
        BlockQmmArgs p = a;
        p.m = a.m - m0 < rows ? a.m - m0 : rows;
        p.x += m0 * a.k;
        p.x_scales += m0 * ((a.k + kBlock - 1) / kBlock);
        p.y = static_cast<char*>(a.y) + m0 * a.n * (a.dtype == 0 ? 4 : 2);
        qmm_small_kernel<<<dim3((unsigned)((a.n + 15) / 16), (unsigned)((p.m + 15) / 16)), dim3(64 * kWaves), 0, stream>>>(p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace qaff
