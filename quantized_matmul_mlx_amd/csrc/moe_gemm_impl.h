// The layer of a mixture of experts for many rows an expert: the same products as moe_few_impl.h as a GEMM
// over each expert's rows, on float16 matrix instructions.
//
//   1. moe_sort: the pairs of each expert in their order (a workgroup an expert looks through all pairs), and x
//      as float16 rows;
//   2. gate and up: h = silu(g) u of up to 192 rows x 64 columns a workgroup;
//   3. down: d of up to 192 rows x 128 columns;
//   4. moe_combine (moe_few_impl.h).
//
// Weights become float16 operands, rounded once to 11 bits, by two instructions for two codes: a code alone
// in a 16-bit half is the denormal c 2^-24, so an AND takes two 4-bit codes out of a word and a packed
// multiply-add forms s c + b. To stay inside float16's range every row of a weight has a power of two of its
// own, found when a workgroup takes its scales and biases into LDS, and so has every row of x (bf16 values
// keep their 8 bits) and every 16 columns of a row of h. Against float64, weights rounded to 8 bits instead
// would cost 1.5 times the rounding of y; these cost a hundredth.
//
// A workgroup of 4 waves has 128 rows of a weight, 32 a wave, dequantized once in registers by the wave that
// multiplies them, against up to 6 x 32 rows of x from LDS (only as many as there are). Two workgroups share a
// compute unit, so that one's products cover the other's loads. v_mfma_f32_32x32x16_f16: lane l supplies row
// l % 32 of x and of the weight, 8 values at k-slot l / 32; result v of lane l is D[8 (v / 4) + 4 (l / 32)
// + v % 4][l % 32].
#pragma once

#include "moe_few_impl.h"

#include <algorithm>

namespace qaff {
namespace {

constexpr int kMT = 6;                 // turns of 32 rows a workgroup takes at most
constexpr int kTileM = 32 * kMT;       // rows
constexpr int kGemmThreads = 256;
constexpr int kStep = 64;              // codes a stage of x
constexpr int kPitch = 2 * kStep;      // bytes of a row of a stage
constexpr int kPieceCount = kTileM * 8 / kGemmThreads;  // 16-byte pieces of a stage a thread

struct GemmArgs {
    const uint16_t* x;       // float16 rows of k values: [tokens] (DOWN false) or [sorted pairs]
    const float* x_scale;    // [tokens] what a row of x was divided by, or null
    const int8_t* h_exp;     // [sorted pairs, hidden / 16] exponents of h
    ExpertWeight w0, w1;
    const int32_t* order;    // [pairs]: sorted position -> pair
    const int32_t* offsets;  // [experts + 1]
    const float* weights;    // [pairs]
    uint16_t* h;             // [sorted pairs, n]
    int8_t* h_exp_out;
    float* d;                // [pairs, n]
    int k, n, top_k, experts, tiles_n, blocks;
};

// ---- the order of the pairs, and x as float16 -----------------------------------------------------

constexpr int kSortThreads = 1024;

// Workgroup e < experts: offsets[e] = pairs of lower experts, order[offsets[e] ..] = its pairs. The others: rows
// of x, a wave each, divided by a power of two that puts the largest value into [2^14, 2^15).
__global__ __launch_bounds__(kSortThreads) void moe_sort_kernel(const int32_t* chosen, int64_t pairs, int experts,
                                                                int32_t* order, int32_t* offsets, const uint16_t* x,
                                                                int64_t tokens, int width, uint16_t* xh, float* x_scale) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if ((int)blockIdx.x >= experts) {
        const int64_t t = (int64_t)(blockIdx.x - experts) * (kSortThreads / 64) + wave;
        if (t >= tokens) return;
        const uint16_t* src = x + t * width;
        float top = 0.f;
        for (int c = lane * 8; c < width; c += 512) {
            const u32x4h v = *reinterpret_cast<const u32x4h*>(src + c);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                top = fmaxf(top, fmaxf(fabsf(bf16_to_f32(v[q])), fabsf(__uint_as_float(v[q] & 0xffff0000u))));
        }
#pragma unroll
        for (int s = 32; s >= 1; s >>= 1) top = fmaxf(top, __shfl_xor(top, s, 64));
        const int ex = min((int)(__float_as_uint(top) >> 23), 254);     // infinities stay so
        const int up = min(14 + 127 - max(ex, 1), 120);                 // 2^up takes the largest to [2^14, 2^15)
        for (int c = lane * 8; c < width; c += 512) {
            const u32x4h v = *reinterpret_cast<const u32x4h*>(src + c);
            u32x4a o;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                o[q] = pack_half2<true>(ldexpf(bf16_to_f32(v[q]), up), ldexpf(__uint_as_float(v[q] & 0xffff0000u), up));
            *reinterpret_cast<u32x4a*>(xh + t * width + c) = o;
        }
        if (lane == 0) x_scale[t] = ldexpf(1.f, -up);
        return;
    }
    __shared__ int sums[2][kSortThreads / 64];
    const int e = blockIdx.x;
    // a thread's pairs lie side by side, so that its rank orders them
    const int64_t each = (pairs + kSortThreads - 1) / kSortThreads;
    const int64_t p0 = tid * each, p1 = min(pairs, p0 + each);
    int less = 0, mine = 0;
    for (int64_t p = p0; p < p1; ++p) {
        const int c = chosen[p];
        less += c >= 0 && c < e;
        mine += c == e;
    }
    const int before = wave_scan(mine);
    const int lower = wave_scan(less);
    if (lane == 63) {
        sums[0][wave] = before;
        sums[1][wave] = lower;
    }
    __syncthreads();
    int at = before - mine, base = 0, total = 0;
    for (int w = 0; w < kSortThreads / 64; ++w) {
        if (w < wave) at += sums[0][w];
        total += sums[0][w];
        base += sums[1][w];
    }
    for (int64_t p = p0; p < p1; ++p)
        if (chosen[p] == e) order[base + at++] = (int)p;
    if (tid == 0) {
        offsets[e] = base;
        if (e == experts - 1) offsets[experts] = base + total;
    }
}

// ---- weights as float16 operands ------------------------------------------------------------------

typedef f16x2 h2;

__device__ __forceinline__ uint32_t fma2(uint32_t c, h2 s, h2 b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(h2, c), s, b));
}

// Octet j of a block: codes times s + b. sb: the group's s 2^24 and b (float16 bits, low and high half).
// 4-bit codes come in the order c0 c4 c1 c5 c2 c6 c3 c7 (x is staged in it).
template <int BITS>
__device__ __forceinline__ f16x8 weight_operand(const uint32_t (&w)[BITS], int j, uint32_t sb) {
    const uint32_t lo = sb & 0xffffu, hi = sb >> 16;
    const h2 s = __builtin_bit_cast(h2, lo | lo << 16), b = __builtin_bit_cast(h2, hi | hi << 16);
    u32x4a o;
    if constexpr (BITS == 4) {
        const h2 s16 = s * (h2){(_Float16)0.0625f, (_Float16)0.0625f};
        const uint32_t v = w[j], v8 = v >> 8;
        o[0] = fma2(v & 0x000F000Fu, s, b);
        o[1] = fma2(v & 0x00F000F0u, s16, b);
        o[2] = fma2(v8 & 0x000F000Fu, s, b);
        o[3] = fma2(v8 & 0x00F000F0u, s16, b);
    } else if constexpr (BITS == 8) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            o[q] = fma2(__builtin_amdgcn_perm(0u, w[2 * j + (q >> 1)], q & 1 ? 0x0c030c02u : 0x0c010c00u), s, b);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            o[q] = fma2(code_at<BITS>(w, 8 * j + 2 * q) | code_at<BITS>(w, 8 * j + 2 * q + 1) << 16, s, b);
    }
    return __builtin_bit_cast(f16x8, o);
}

// ---- the GEMM -----------------------------------------------------------------------------------------

// LDS: two stages of x, then the scales and biases of the 128 weight rows.
inline int gemm_lds_bytes(int k, int group) { return 2 * kTileM * kPitch + 128 * (k / group + 1) * 4; }
constexpr int kGemmMaxLds = 158 * 1024;

template <int BITS, int GSHIFT, bool F16, bool DOWN>
__global__ __launch_bounds__(kGemmThreads, 2) void moe_gemm_kernel(GemmArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    __shared__ int src[kTileM];        // row of x
    __shared__ int pair[kTileM];       // DOWN: pair of the row
    __shared__ float row_scale[kTileM];
    __shared__ int where[3];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 31, h = lane >> 5;

    // Workgroups of one tile of rows follow each other on one XCD (workgroup i runs on XCD i % 8), whose L2 then
    // holds the rows.
    const int xcd = blockIdx.x % 8, seq = blockIdx.x / 8;
    const int tile = seq / a.tiles_n * 8 + xcd, tn = seq % a.tiles_n;
    if (wave == 0) {  // the expert and the rows of this tile
        int first = 0, found = -1;
        for (int base = 0; base < a.experts && found < 0; base += 64) {
            const int e = min(base + lane, a.experts - 1);
            const int n = base + lane < a.experts ? a.offsets[e + 1] - a.offsets[e] : 0;
            const int tiles = (n + kTileM - 1) / kTileM;
            const int upto = first + wave_scan(tiles);
            const uint64_t past = __builtin_amdgcn_ballot_w64(upto > tile);
            if (past) {
                found = base + __builtin_ctzll(past);
                const int l = __builtin_ctzll(past);
                first = __shfl(upto - tiles, l, 64);
            } else {
                first = __shfl(upto, 63, 64);
            }
        }
        if (lane == 0) {
            where[0] = found;
            if (found >= 0) {
                where[1] = a.offsets[found] + (tile - first) * kTileM;
                where[2] = a.offsets[found + 1];
            }
        }
    }
    __syncthreads();
    const int e = where[0];
    if (e < 0) return;
    const int row0 = where[1], rows = min(kTileM, where[2] - row0);
    const int turns = (rows + 31) / 32;
    const int kb = a.k / 32, gpr = kb >> GSHIFT, spitch = gpr + 1;
    uint8_t* xl = smem;
    uint32_t* sb = reinterpret_cast<uint32_t*>(smem + 2 * kTileM * kPitch);

    // this wave's weight rows: gate rows 64 tn + 16 wave + r and the up rows of the same columns, or 128 tn + ...
    const int wrow = DOWN ? 128 * tn + 32 * wave + r : 64 * tn + 16 * wave + (r & 15);
    const ExpertWeight& W = !DOWN && r >= 16 ? a.w1 : a.w0;
    const int64_t wr = (int64_t)e * a.n + min(wrow, a.n - 1);
    const uint32_t* pw = W.packed + wr * kb * BITS;

    // scales and biases to LDS, times the power of two of the row: the largest scale 2^24 lies in [2^14, 2^15)
    const uint16_t* sp = W.scales + wr * gpr;
    const uint16_t* bp = W.biases + wr * gpr;
    float top = 0.f;
    for (int g = h; g < gpr; g += 2)
        top = fmaxf(top, fmaxf(fabsf(half_to_f32<F16>(sp[g])), fabsf(half_to_f32<F16>(bp[g])) * 0x1p-20f));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const int up = min(14 + 127 - max(min((int)(__float_as_uint(top) >> 23), 254), 1), 120);
    uint32_t* sbw = sb + (32 * wave + r) * spitch;
    for (int g = h; g < gpr; g += 2)
        sbw[g] = pack_half2<true>(ldexpf(half_to_f32<F16>(sp[g]), up), ldexpf(half_to_f32<F16>(bp[g]), up - 24));
    const float col_scale = ldexpf(1.f, 24 - up);

    // rows of x: where they are and their power of two
    for (int i = tid; i < kTileM; i += kGemmThreads) {
        const int at = row0 + min(i, rows - 1);
        const int p = a.order[at];
        if constexpr (DOWN) {
            src[i] = at;
            pair[i] = p;
            int most = -128;
            for (int c = 0; c < a.k / 16; ++c) most = max(most, (int)a.h_exp[(int64_t)at * (a.k / 16) + c]);
            row_scale[i] = __int_as_float(most);  // the exponent, for now
        } else {
            src[i] = p / a.top_k;
            row_scale[i] = a.x_scale ? a.x_scale[p / a.top_k] : 1.f;
        }
    }
    __syncthreads();

    // this thread's pieces of a stage: row i * 32 + tid / 8, 16 bytes at slot tid % 8. Stage t = 2 u + s holds codes
    // 128 u + 32 s .. + 31 (k-slot 0) and 128 u + 64 + 32 s .. (k-slot 1).
    const int piece = tid & 7;
    const int col_in = (piece >> 2) * 64 + (piece & 3) * 8;
    const uint16_t* xp[kPieceCount];
    int most[kPieceCount];
#pragma unroll
    for (int i = 0; i < kPieceCount; ++i) {
        const int row = i * 32 + tid / 8;
        xp[i] = a.x + (int64_t)src[row] * a.k;
        if constexpr (DOWN) most[i] = __float_as_int(row_scale[row]);
    }
    if constexpr (DOWN) {
        __syncthreads();
        for (int i = tid; i < kTileM; i += kGemmThreads)
            row_scale[i] = a.weights[pair[i]] * ldexpf(1.f, __float_as_int(row_scale[i]));
    }
    u32x4a xr[kPieceCount];
    int xe[kPieceCount];
    auto load_x = [&](int t) {
        const int c = (t >> 1) * 128 + (t & 1) * 32 + col_in;
#pragma unroll
        for (int i = 0; i < kPieceCount; ++i) {
            xr[i] = u32x4a{0u, 0u, 0u, 0u};
            xe[i] = 0;
            if (i < turns && c < a.k) {
                const u32x4h v = *reinterpret_cast<const u32x4h*>(xp[i] + c);
                xr[i] = u32x4a{v.x, v.y, v.z, v.w};
                if constexpr (DOWN) xe[i] = a.h_exp[(int64_t)src[i * 32 + tid / 8] * (a.k / 16) + c / 16];
            }
        }
    };
    auto store_x = [&](int t) {
        uint8_t* to = xl + (t & 1) * (kTileM * kPitch);
#pragma unroll
        for (int i = 0; i < kPieceCount; ++i) {
            if (i >= turns) continue;
            const int row = i * 32 + tid / 8;
            u32x4a v = xr[i];
            if constexpr (DOWN) {  // to the power of two of the row
                const _Float16 f = (_Float16)ldexpf(1.f, max(xe[i] - most[i], -30));
                const h2 f2 = {f, f};
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, (uint32_t)v[q]) * f2);
            }
            if constexpr (BITS == 4)
                v = u32x4a{__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                           __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u)};
            *reinterpret_cast<u32x4a*>(to + row * kPitch + ((piece ^ (row >> 1)) & 7) * 16) = v;
        }
    };
    // A unit of 128 codes: this lane's blocks 2 h and 2 h + 1 of its four.
    const int units = (a.k + 127) / 128;
    uint32_t wq[2][2][BITS];
    auto load_w = [&](uint32_t (&w)[2][BITS], int u) {
#pragma unroll
        for (int s = 0; s < 2; ++s) load_block<BITS>(pw + min(4 * u + 2 * h + s, kb - 1) * BITS, w[s]);
    };

    f32x16 acc[kMT];
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][v] = 0.f;

    auto products = [&](const uint32_t (&w)[BITS], int t) {
        const uint8_t* from = xl + (t & 1) * (kTileM * kPitch) + r * kPitch;
        const int block = (t >> 1) * 4 + 2 * h + (t & 1);
        const uint32_t g = sbw[min(block >> GSHIFT, gpr - 1)];
        f16x8 o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = weight_operand<BITS>(w, q, g);
#pragma unroll
        for (int i = 0; i < kMT; ++i) {
            if (i >= turns) break;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f16x8 v = *reinterpret_cast<const f16x8*>(from + i * 32 * kPitch + ((4 * h + q) ^ (r >> 1 & 7)) * 16);
                acc[i] = mfma32x32x16<true>(v, o[q], acc[i]);
            }
        }
    };

    const int stages = 2 * units;
    load_x(0);
    load_w(wq[0], 0);
    store_x(0);
    load_x(1);
    for (int u = 0; u < units; u += 2) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int t = 2 * u + s;
            if (t >= stages) break;
            __syncthreads();  // stage t is there; nobody reads the other place any more
            if (s % 2 == 0) load_w(wq[(s / 2 + 1) & 1], min(u + s / 2 + 1, units - 1));
            if (t + 1 < stages) store_x(t + 1);
            if (t + 2 < stages) load_x(t + 2);
            products(wq[s / 2][s & 1], t);
        }
    }

#pragma unroll
    for (int i = 0; i < kMT; ++i) {
        if (i >= turns) break;
        if constexpr (DOWN) {
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int row = 32 * i + 8 * (v >> 2) + 4 * h + (v & 3);
                if (row < rows && wrow < a.n)
                    a.d[(int64_t)pair[row] * a.n + wrow] = acc[i][v] * (row_scale[row] * col_scale);
            }
        } else {
            // lanes r < 16 hold gate and r >= 16 up results: exchanged in pairs of rows, lanes with r < 16 keep row v
            // and the others row v + 1
            const float other = __shfl_xor(col_scale, 16, 64);
            const float gs = r < 16 ? col_scale : other, us = r < 16 ? other : col_scale;
#pragma unroll
            for (int v = 0; v < 16; v += 2) {
                uint32_t x0 = __float_as_uint(acc[i][v]), x1 = __float_as_uint(acc[i][v + 1]);
                swap16(x0, x1);
                const int vv = v + (r >> 4);
                const int row = 32 * i + 8 * (vv >> 2) + 4 * h + (vv & 3);
                const float xs = row_scale[row];
                const float hv = silu_f32(__uint_as_float(x0) * gs * xs) * (__uint_as_float(x1) * us * xs);
                // the 16 lanes of a row: their power of two
                float m = fabsf(hv);
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
                const int ex = min(max((int)(__float_as_uint(m) >> 23), 1), 254) - 127;
                if (row < rows && 64 * tn + 16 * wave < a.n) {
                    const int64_t at = row0 + row;
                    a.h[at * a.n + wrow] = f32_to_half_bits<true>(ldexpf(hv, -ex));
                    if ((r & 15) == 0) a.h_exp_out[at * (a.n / 16) + (64 * tn + 16 * wave) / 16] = (int8_t)ex;
                }
            }
        }
    }
}

// ---- launches -----------------------------------------------------------------------------------------

struct MoeSpace {  // byte offsets into the workspace
    int64_t xh, x_scale, order, offsets, h, h_exp, d, bytes;
};
inline MoeSpace moe_gemm_space(int64_t tokens, int64_t width, int64_t hidden, int64_t top_k, int64_t experts) {
    const int64_t pairs = tokens * top_k;
    MoeSpace s{};
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t was = at;
        at = round_up(at + bytes, 256);
        return was;
    };
    s.xh = take(tokens * width * 2);
    s.x_scale = take(tokens * 4);
    s.order = take(pairs * 4);
    s.offsets = take((experts + 1) * 4);
    s.h = take(pairs * hidden * 2);
    s.h_exp = take(pairs * (hidden / 16));
    s.d = take(pairs * width * 4);
    s.bytes = at;
    return s;
}

// Tiles of rows: whole ones, and at most one that is not whole an expert.
inline int64_t gemm_tiles(const MoeArgs& a) {
    const int64_t pairs = a.tokens * a.top_k;
    return round_up(pairs / kTileM + std::min(pairs, (int64_t)a.experts), 8);
}

template <int BITS, int GSHIFT, bool F16>
hipError_t launch_gemm_path(const MoeArgs& a, hipStream_t stream) {
    const int64_t pairs = a.tokens * a.top_k;
    const MoeSpace s = moe_gemm_space(a.tokens, a.width, a.hidden, a.top_k, a.experts);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    uint16_t* xh = reinterpret_cast<uint16_t*>(ws + s.xh);
    float* x_scale = reinterpret_cast<float*>(ws + s.x_scale);
    int32_t* order = reinterpret_cast<int32_t*>(ws + s.order);
    int32_t* offsets = reinterpret_cast<int32_t*>(ws + s.offsets);
    const int64_t convert = F16 ? 0 : (a.tokens + kSortThreads / 64 - 1) / (kSortThreads / 64);
    moe_sort_kernel<<<dim3((unsigned)(a.experts + convert)), dim3(kSortThreads), 0, stream>>>(
        a.chosen, pairs, a.experts, order, offsets, a.x, a.tokens, a.width, xh, x_scale);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    GemmArgs g{};
    g.order = order;
    g.offsets = offsets;
    g.weights = a.weights;
    g.top_k = a.top_k;
    g.experts = a.experts;
    const int64_t tiles = gemm_tiles(a);
    g.x = F16 ? a.x : xh;
    g.x_scale = F16 ? nullptr : x_scale;
    g.w0 = a.gate;
    g.w1 = a.up;
    g.h = reinterpret_cast<uint16_t*>(ws + s.h);
    g.h_exp_out = reinterpret_cast<int8_t*>(ws + s.h_exp);
    g.k = a.width;
    g.n = a.hidden;
    g.tiles_n = (a.hidden + 63) / 64;
    moe_gemm_kernel<BITS, GSHIFT, F16, false><<<dim3((unsigned)(tiles * g.tiles_n)), dim3(kGemmThreads),
                                               gemm_lds_bytes(a.width, a.group), stream>>>(g);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    g.x = g.h;
    g.x_scale = nullptr;
    g.h_exp = g.h_exp_out;
    g.w0 = g.w1 = a.down;
    g.d = reinterpret_cast<float*>(ws + s.d);
    g.k = a.hidden;
    g.n = a.width;
    g.tiles_n = (a.width + 127) / 128;
    moe_gemm_kernel<BITS, GSHIFT, F16, true><<<dim3((unsigned)(tiles * g.tiles_n)), dim3(kGemmThreads),
                                              gemm_lds_bytes(a.hidden, a.group), stream>>>(g);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    return launch_combine<F16>(a, g.d, stream);
}

// Whether the GEMM serves a call: from an average of 24 rows an expert on, where the scales of 128 weight rows fit
// LDS beside x and a launch holds the tiles (2^32 threads).
inline bool gemm_path(const MoeArgs& a) {
    const int64_t widest = std::max(a.hidden / 64, a.width / 128) + 1;
    return a.tokens * a.top_k >= (int64_t)24 * a.experts && gemm_tiles(a) * widest < (int64_t)1 << 24 && gemm_lds_bytes(a.width, a.group) <= kGemmMaxLds &&
           gemm_lds_bytes(a.hidden, a.group) <= kGemmMaxLds;
}

template <int BITS, bool F16>
hipError_t launch_moe_bits(const MoeArgs& a, hipStream_t stream) {
    if (!gemm_path(a)) return launch_few_bits<BITS, F16>(a, stream);
    if (a.group == 32) return launch_gemm_path<BITS, 0, F16>(a, stream);
    if (a.group == 64) return launch_gemm_path<BITS, 1, F16>(a, stream);
    return launch_gemm_path<BITS, 2, F16>(a, stream);
}

template <bool F16>
hipError_t launch_moe(const MoeArgs& a, hipStream_t stream) {
    if (a.top_k == 0 || a.experts == 0 || a.hidden == 0) return launch_combine<F16>(a, nullptr, stream);
    switch (a.bits) {
        case 1: return launch_moe_bits<1, F16>(a, stream);
        case 2: return launch_moe_bits<2, F16>(a, stream);
        case 3: return launch_moe_bits<3, F16>(a, stream);
        case 4: return launch_moe_bits<4, F16>(a, stream);
        case 5: return launch_moe_bits<5, F16>(a, stream);
        case 6: return launch_moe_bits<6, F16>(a, stream);
        case 8: return launch_moe_bits<8, F16>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace
}  // namespace qaff
