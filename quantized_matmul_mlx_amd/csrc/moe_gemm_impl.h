// The layer of a mixture of experts for many rows an expert: the same products as moe_few_impl.h as a GEMM
// over each expert's rows, on float16 matrix instructions.
//
//   1. moe_sort: the pairs of each expert in their order (a workgroup an expert looks through all pairs), and x
//      as float16 rows;
//   2. gate and up: h = silu(g) u of up to 160 rows x 64 columns a workgroup;
//   3. down: d of up to 160 rows x 128 columns;
//   4. moe_combine (moe_few_impl.h).
//
// Weights become float16 operands, rounded once to 11 bits, by two instructions for two codes: a code alone
// in a 16-bit half is the denormal c 2^-24, so an AND takes two 4-bit codes out of a word and a packed
// multiply-add forms s c + b. To stay inside float16's range every row of a weight has a power of two of its
// own, found when a workgroup takes its scales and biases into LDS, and so has every row of x (bf16 values
// keep their 8 bits) and every 16 columns of a row of h. Against float64, weights rounded to 8 bits instead
// would cost 1.5 times the rounding of y; these cost a hundredth. h has 11 bits and so loses no more.
//
// Measured (kernels alone): 2048 tokens through 8 of 128 x [768, 2048], 4 bits: sort 12.1 us, gate and up 165, down 129,
// combine 24, 155 GFLOP in all; 512 tokens through 2 of 8 x [14336, 4096]: 434 and 340 us, where the kernels for few
// rows take 3.8 ms. Bound by what surrounds the products of a tile: 143 of then 189 us stayed when all loads and
// dequantization were left out.
//
// A workgroup of 4 waves has 128 rows of a weight, 32 a wave, dequantized once in registers by the wave that
// multiplies them, against up to 5 x 32 rows of x from LDS (only as many as there are). Two workgroups share a
// compute unit, so that one's products cover the other's loads. v_mfma_f32_32x32x16_f16: lane l supplies row
// l % 32 of x and of the weight, 8 values at k-slot l / 32; result v of lane l is D[8 (v / 4) + 4 (l / 32)
// + v % 4][l % 32].
#pragma once

#include "moe_few_impl.h"

#include <algorithm>

namespace qaff {
namespace {

constexpr int kTileM = 160;            // rows a workgroup takes at most, in turns of 32
constexpr int kGemmThreads = 256;
constexpr int kStep = 64;              // codes a stage of x
constexpr int kPitch = 2 * kStep;      // bytes of a row of a stage
constexpr int kStages = 3;
constexpr int kStageBytes = kTileM * kPitch;

struct GemmArgs {
    const uint16_t* x;       // float16 rows of pad(k) values: [tokens] (DOWN false) or [sorted pairs]
    const float* x_scale;    // [tokens] what a row of x was divided by
    uint8_t* h_exp;          // [sorted pairs, hidden / 16] exponents of h, + 128
    ExpertWeight w0, w1;
    const int32_t* order;    // [pairs]: sorted position -> pair
    const int32_t* offsets;  // [experts + 1]
    const float* weights;    // [pairs]
    uint16_t* h;             // [sorted pairs, pad(n)]
    float* d;                // [pairs, n]
    int k, n, top_k, experts, tiles_n;
    int gshift;              // group size 32 << gshift
    int f16;                 // type of scales and biases
};

// Rows of x and h end with zeros up to a whole unit of 128 values. With 4-bit codes each 8 values lie in the order of
// their operands, 0 4 1 5 2 6 3 7.
__host__ __device__ constexpr int pad_unit(int k) { return (k + 127) / 128 * 128; }
__host__ __device__ constexpr int operand_place(int i) { return (i & ~7) | (i & 3) << 1 | (i >> 2 & 1); }

// ---- the order of the pairs, and x as float16 -----------------------------------------------------

constexpr int kSortThreads = 1024;

// Four pairs' experts from p on; -1 past the last pair.
__device__ __forceinline__ void sort_load(const int32_t* chosen, int64_t pairs, int64_t p, int (&c)[4]) {
    const int64_t at = min(p, max(pairs - 4, (int64_t)0));
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = chosen[min(at + i, pairs - 1)];
    if (p + 4 > pairs) {  // the loads above began early
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = p + i < pairs ? chosen[p + i] : -1;
    }
}
__device__ __forceinline__ int sort_less(const int32_t* chosen, int64_t pairs, int64_t p, int e) {
    int c[4], n = 0;
    sort_load(chosen, pairs, p, c);
#pragma unroll
    for (int i = 0; i < 4; ++i) n += c[i] >= 0 && c[i] < e;
    return n;
}

// Workgroup e < experts: offsets[e] = pairs of lower experts, order[offsets[e] ..] = its pairs. The others: rows
// of x in float16, a wave each, divided by a power of two that puts the largest value into [2^14, 2^15).
template <bool F16>
__global__ __launch_bounds__(kSortThreads) void moe_sort_kernel(const int32_t* chosen, int64_t pairs, int experts,
                                                                int32_t* order, int32_t* offsets, const uint16_t* x,
                                                                int64_t tokens, int width, uint16_t* xh, float* x_scale, int fours,
                                                                int hidden, uint16_t* h) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int pitch = pad_unit(width);
    if ((int)blockIdx.x >= experts) {
        const int64_t t = (int64_t)(blockIdx.x - experts) * (kSortThreads / 64) + wave;
        if (t >= tokens) return;
        const uint16_t* src = x + t * width;
        auto value = [&](uint32_t v) { return F16 ? half_to_f32<true>(v) : half_to_f32<false>(v); };
        float top = 0.f;
        for (int c = lane * 8; c < width; c += 512) {
            const u32x4h v = *reinterpret_cast<const u32x4h*>(src + c);
#pragma unroll
            for (int q = 0; q < 4; ++q) top = fmaxf(top, fmaxf(fabsf(value(v[q])), fabsf(value(v[q] >> 16))));
        }
#pragma unroll
        for (int s = 32; s >= 1; s >>= 1) top = fmaxf(top, __shfl_xor(top, s, 64));
        const int ex = min((int)(__float_as_uint(top) >> 23), 254);     // infinities stay so
        const int up = min(14 + 127 - max(ex, 1), 120);                 // 2^up takes the largest to [2^14, 2^15)
        for (int c = lane * 8; c < pitch; c += 512) {
            u32x4a o = u32x4a{0u, 0u, 0u, 0u};
            if (c < width) {
                const u32x4h v = *reinterpret_cast<const u32x4h*>(src + c);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    o[q] = pack_half2<true>(ldexpf(value(v[q]), up), ldexpf(value(v[q] >> 16), up));
                if (fours)
                    o = u32x4a{__builtin_amdgcn_perm(o.z, o.x, 0x05040100u), __builtin_amdgcn_perm(o.z, o.x, 0x07060302u),
                               __builtin_amdgcn_perm(o.w, o.y, 0x05040100u), __builtin_amdgcn_perm(o.w, o.y, 0x07060302u)};
            }
            *reinterpret_cast<u32x4a*>(xh + t * pitch + c) = o;
        }
        if (lane == 0) x_scale[t] = ldexpf(1.f, -up);
        return;
    }
    // Four runs of 4 pairs a thread at a time: run, thread and place order the pairs.
    constexpr int kWaves = kSortThreads / 64, kRuns = 4;
    __shared__ uint32_t sums[kRuns * kWaves];
    const int e = blockIdx.x;
    int base = 0;
    for (int64_t p0 = 0; p0 < pairs; p0 += 4 * kSortThreads) base += sort_less(chosen, pairs, p0 + 4 * tid, e);
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) base += __shfl_xor(base, s, 64);
    if (lane == 0) sums[wave] = (uint32_t)base;
    __syncthreads();
    base = 0;
    for (int w = 0; w < kWaves; ++w) base += (int)sums[w];
    __syncthreads();
    int total = 0;
    for (int64_t p0 = 0; p0 < pairs; p0 += 4 * kRuns * kSortThreads) {
        int c[kRuns][4];
        uint32_t before[kRuns];
#pragma unroll
        for (int q = 0; q < kRuns; ++q) sort_load(chosen, pairs, p0 + 4 * (q * kSortThreads + tid), c[q]);
#pragma unroll
        for (int q = 0; q < kRuns; ++q) {
            int mine = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) mine += c[q][i] == e;
            const int upto = wave_scan(mine);
            before[q] = upto - mine;
            if (lane == 63) sums[q * kWaves + wave] = upto;
        }
        __syncthreads();
        const int own = (int)sums[lane];  // kRuns * kWaves = 64 sums
        const int upto = wave_scan(own);
#pragma unroll
        for (int q = 0; q < kRuns; ++q) {
            int at = base + total + (int)before[q] + __shfl(upto - own, q * kWaves + wave, 64);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c[q][i] == e) order[at++] = (int)(p0 + 4 * (q * kSortThreads + tid) + i);
        }
        total += __shfl(upto, 63, 64);
        __syncthreads();
    }
    const int zeros = pad_unit(hidden) - hidden;  // of each of its rows of h
    for (int64_t i = tid; i < (int64_t)total * zeros; i += kSortThreads)
        h[(base + i / zeros) * pad_unit(hidden) + hidden + i % zeros] = 0;
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

// A group's scale and bias, both halves each: s 2^24, that / 16 (for 4-bit codes that stay in bits 4 .. 7) and b.
struct GroupOf {
    h2 s, s16, b;
};
__device__ __forceinline__ GroupOf group_of(uint32_t sb) {
    const uint32_t lo = sb & 0xffffu, hi = sb >> 16;
    const h2 s = __builtin_bit_cast(h2, lo | lo << 16);
    return GroupOf{s, s * (h2){(_Float16)0.0625f, (_Float16)0.0625f}, __builtin_bit_cast(h2, hi | hi << 16)};
}

// Word e of octet j of a block: two codes times s + b. 4-bit codes come in the order c0 c4 c1 c5 c2 c6 c3 c7 (x is
// staged in it).
template <int BITS>
__device__ __forceinline__ uint32_t weight_word(const uint32_t (&w)[BITS], int j, int e, const GroupOf& g) {
    if constexpr (BITS == 4) {
        const uint32_t v = e & 2 ? w[j] >> 8 : w[j];
        return e & 1 ? fma2(v & 0x00F000F0u, g.s16, g.b) : fma2(v & 0x000F000Fu, g.s, g.b);
    } else if constexpr (BITS == 8) {
        return fma2(__builtin_amdgcn_perm(0u, w[2 * j + (e >> 1)], e & 1 ? 0x0c030c02u : 0x0c010c00u), g.s, g.b);
    } else {
        return fma2(code_at<BITS>(w, 8 * j + 2 * e) | code_at<BITS>(w, 8 * j + 2 * e + 1) << 16, g.s, g.b);
    }
}

// ---- the GEMM -----------------------------------------------------------------------------------------

// LDS: three stages of x, then the scales and biases of the 128 weight rows.
// Scales and biases are there for a window of K: all of a row's up to 32 groups, and otherwise those of window_units
// units and of the unit behind them (whose first is read one step early), so that two workgroups fit a compute unit.
constexpr int kWindow = 32;
__host__ __device__ constexpr int window_units(int gshift) { return 3 * (((kWindow >> (2 - gshift)) - 1) / 3); }  // 6, 15, 30
__host__ __device__ constexpr int window_groups(int gpr, int gshift) {
    return gpr <= kWindow ? gpr : (4 * window_units(gshift) + 4) >> gshift;
}
inline int gemm_lds_bytes(int k, int gshift) {
    return kStages * kStageBytes + 128 * (window_groups(k >> (5 + gshift), gshift) + 1) * 4;
}

// The largest magnitude of the 16 lanes of a row.
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, __int_as_float(dpp<0xB1, 0xf>(__float_as_int(v))));   // lane ^ 1
    v = fmaxf(v, __int_as_float(dpp<0x4E, 0xf>(__float_as_int(v))));   // lane ^ 2
    v = fmaxf(v, __int_as_float(dpp<0x141, 0xf>(__float_as_int(v))));  // mirrored in 8
    return fmaxf(v, __int_as_float(dpp<0x140, 0xf>(__float_as_int(v))));  // and in 16
}

// The largest of n bytes.
__device__ __forceinline__ int most_of(const uint8_t* p, int n) {
    typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(1)));
    uint32_t m = 0;
    int i = 0;
    for (; i + 16 <= n; i += 16) {
        const u32x4u v = *reinterpret_cast<const u32x4u*>(p + i);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int b = 0; b < 4; ++b) m = max(m, (uint32_t)v[q] >> (8 * b) & 0xffu);
    }
    for (; i < n; ++i) m = max(m, (uint32_t)p[i]);
    return (int)m;
}

// A group's scale and bias as they lie in the window.
__device__ __forceinline__ uint32_t to_window(uint32_t s, uint32_t b, int up, bool f16) {
    auto value = [&](uint32_t v) { return f16 ? half_to_f32<true>(v) : half_to_f32<false>(v); };
    return pack_half2<true>(ldexpf(value(s), up), ldexpf(value(b), up - 24));
}

// What a workgroup finds before its loop.
struct GemmTile {
    const uint32_t* pw;      // this lane's weight row
    uint32_t* sb;            // the window of its scales and biases in LDS
    const uint16_t *sp, *bp; // and all of them
    int up;                  // scales are times 2^up there, biases 2^(up - 24)
    uint8_t* xl;
    const uint16_t* x;       // a.x, DOWN: from the tile's first row on
    const uint8_t* exps;     // DOWN: the exponents, from the tile's first row on
    const int *src, *pair;   // [kTileM] in LDS
    const float* row_scale;
    const int* most;         // DOWN: the largest exponent of the row, + 128
    float col_scale;
    int row0, rows, wrow, tn;
};

// T turns of 32 rows.
template <int BITS, bool DOWN, int T>
__device__ __forceinline__ void gemm_tile(const GemmArgs& a, const GemmTile& c, int tid) {
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 31, h = lane >> 5;
    const int kb = a.k / 32, gpr = kb >> a.gshift;

    // This thread's pieces of a stage: row i * 32 + tid / 8, 16 bytes at slot tid % 8. Stage t = 2 u + s holds codes
    // 128 u + 32 s .. + 31 (k-slot 0) and 128 u + 64 + 32 s .. (k-slot 1).
    const int piece = tid & 7, col_in = (piece >> 2) * 64 + (piece & 3) * 8;
    const int pitch = pad_unit(a.k);
    uint32_t xp[T], ep[T];  // bytes from c.x and c.exps on
    int most[T];
    uint8_t* to[T];
#pragma unroll
    for (int i = 0; i < T; ++i) {
        const int row = i * 32 + tid / 8;
        xp[i] = (uint32_t)(c.src[row] * pitch + col_in) * 2u;
        if constexpr (DOWN) {
            ep[i] = (uint32_t)(c.src[row] * (a.k / 16));
            most[i] = c.most[row];
        }
        to[i] = c.xl + row * kPitch + ((piece ^ (row >> 1)) & 7) * 16;
    }
    struct Ahead {
        u32x4a x[T];
        int e[T];
    };
    const int units = pitch / 128;
    auto load_x = [&](Ahead& s, int t, int i) {  // stages past the last one repeat it
        t = min(t, 2 * units - 1);
        const int col = (t >> 1) * 128 + (t & 1) * 32;
        s.x[i] = *reinterpret_cast<const u32x4a*>(reinterpret_cast<const uint8_t*>(c.x + col) + xp[i]);
        if constexpr (DOWN) s.e[i] = c.exps[ep[i] + (uint32_t)min((col + col_in) / 16, a.k / 16 - 1)];
    };
    auto store_x = [&](const Ahead& s, int stage, int i) {
        u32x4a v = s.x[i];
        if constexpr (DOWN) {  // to the power of two of the row: 2^(e - most), at least 2^-40 (0 in float16)
            const _Float16 f = (_Float16)__int_as_float((max(s.e[i] - most[i], -40) + 127) << 23);
            const h2 f2 = {f, f};
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, (uint32_t)v[q]) * f2);
        }
        *reinterpret_cast<u32x4a*>(to[i] + stage * kStageBytes) = v;
    };
    // A unit of 128 codes: this lane's blocks 2 h and 2 h + 1 of its four.
    auto load_w = [&](uint32_t (&w)[2][BITS], int u) {
#pragma unroll
        for (int s = 0; s < 2; ++s) load_block<BITS>(c.pw + min(4 * min(u, units - 1) + 2 * h + s, kb - 1) * BITS, w[s]);
    };
    int base = 0;  // the window's first group
    auto group_at = [&](int t) {
        return group_of(c.sb[min(((t >> 1) * 4 + 2 * h + (t & 1)) >> a.gshift, gpr - 1) - base]);
    };
    f32x16 acc[T];
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][v] = 0.f;

    // The products of a stage are 4 T, n = q T + i for octet q and turn i. The x operand of each is read kDepth products
    // ahead (a read takes longer than a product), over the border of two stages too, and the weight operand of the next
    // octet is formed word by word beside them; so are the stores and loads of x.
    constexpr int kDepth = T == 5 ? 5 : 8, kCount = 4 * T;
    static_assert(kCount % kDepth == 0, "the operands' places turn with the stages");
    f16x8 f[kDepth];
    auto read = [&](int stage, int n) {
        return *reinterpret_cast<const f16x8*>(c.xl + stage * kStageBytes + (n % T * 32 + r) * kPitch +
                                               ((4 * h + n / T) ^ (r >> 1 & 7)) * 16);
    };
    u32x4a o;  // the weight operand of the next octet
    auto step = [&](int t, int stage, const uint32_t (&w)[BITS], const uint32_t (&follow)[BITS], GroupOf& g, Ahead& x) {
        uint32_t own[BITS], next[BITS];
#pragma unroll
        for (int i = 0; i < BITS; ++i) {
            own[i] = w[i];
            next[i] = follow[i];
            // here, not where the loads are issued, which would wait for them
            asm volatile("" : "+v"(own[i]), "+v"(next[i]));
        }
        const GroupOf gn = group_at(t + 1);
        // After this barrier nobody reads stage t - 1 any more, whose place stage t + 2 takes; stage t + 1, stored one
        // step ago, is there.
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const f16x8 now = __builtin_bit_cast(f16x8, o);
#pragma unroll
            for (int i = 0; i < T; ++i) {
                const int n = q * T + i;
                acc[i] = mfma32x32x16<true>(f[n % kDepth], now, acc[i]);
                f[n % kDepth] = n + kDepth < kCount ? read(stage, n + kDepth) : read((stage + 1) % kStages, n + kDepth - kCount);
                if (n < T) store_x(x, (stage + 2) % kStages, n);
                else if (n < 2 * T) load_x(x, t + 4, n - T);
#pragma unroll
                for (int e = 4 * i / T; e < 4 * (i + 1) / T; ++e)
                    o[e] = q < 3 ? weight_word<BITS>(own, q + 1, e, g) : weight_word<BITS>(next, 0, e, gn);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        g = gn;
    };

    Ahead xa, xb;
    uint32_t w0[2][BITS], w1[2][BITS], w2[2][BITS];
#pragma unroll
    for (int i = 0; i < T; ++i) load_x(xa, 0, i);
    load_w(w0, 0);
#pragma unroll
    for (int i = 0; i < T; ++i) load_x(xb, 1, i);
    load_w(w1, 1);
#pragma unroll
    for (int i = 0; i < T; ++i) {
        store_x(xa, 0, i);
        load_x(xa, 2, i);
    }
#pragma unroll
    for (int i = 0; i < T; ++i) {
        store_x(xb, 1, i);
        load_x(xb, 3, i);
    }
    GroupOf g = group_at(0);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = weight_word<BITS>(w0[0], 0, e, g);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kDepth; ++n) f[n] = read(0, n);
    auto unit = [&](int u, int stage, const uint32_t (&w)[2][BITS], const uint32_t (&follow)[2][BITS],
                    uint32_t (&free)[2][BITS]) {
        load_w(free, u + 2);
        step(2 * u, stage, w[0], w[1], g, xa);
        step(2 * u + 1, (stage + 1) % kStages, w[1], follow[0], g, xb);
    };
    int move = gpr > kWindow ? window_units(a.gshift) : units;  // the unit from which on the next window is read
    for (int u = 0;; u += 3) {  // six steps: the stages and the weights' registers turn
        if (u == move) {
            base = (4 * u) >> a.gshift;
            move += window_units(a.gshift);
            const int there = min(window_groups(gpr, a.gshift), gpr - base);
            for (int i = h; i < there; i += 2) c.sb[i] = to_window(c.sp[base + i], c.bp[base + i], c.up, a.f16);
            __builtin_amdgcn_wave_barrier();  // the row's other lanes read it
        }
        unit(u, 0, w0, w1, w2);
        if (u + 1 >= units) break;
        unit(u + 1, 2, w1, w2, w0);
        if (u + 2 >= units) break;
        unit(u + 2, 1, w2, w0, w1);
        if (u + 3 >= units) break;
    }

#pragma unroll
    for (int i = 0; i < T; ++i) {
        if constexpr (DOWN) {
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int row = 32 * i + 8 * (v >> 2) + 4 * h + (v & 3);
                if (row < c.rows && c.wrow < a.n)
                    a.d[(int64_t)c.pair[row] * a.n + c.wrow] = acc[i][v] * (c.row_scale[row] * c.col_scale);
            }
        } else {
            // lanes r < 16 hold gate and r >= 16 up results: exchanged in pairs of rows, lanes with r < 16 keep row v
            // and the others row v + 1
            const float other = __shfl_xor(c.col_scale, 16, 64);
            const float gs = r < 16 ? c.col_scale : other, us = r < 16 ? other : c.col_scale;
#pragma unroll
            for (int v = 0; v < 16; v += 2) {
                uint32_t x0 = __float_as_uint(acc[i][v]), x1 = __float_as_uint(acc[i][v + 1]);
                swap16(x0, x1);
                const int vv = v + (r >> 4);
                const int row = 32 * i + 8 * (vv >> 2) + 4 * h + (vv & 3);
                const float xs = c.row_scale[row];
                const float hv = silu_f32(__uint_as_float(x0) * gs * xs) * (__uint_as_float(x1) * us * xs);
                // the power of two of the row's 16 columns
                const int ex = min(max((int)(__float_as_uint(row_max(fabsf(hv))) >> 23), 1), 254) - 127;
                if (row < c.rows && 64 * c.tn + 16 * wave < a.n) {
                    const int64_t at = c.row0 + row;
                    a.h[at * pad_unit(a.n) + (BITS == 4 ? operand_place(c.wrow) : c.wrow)] =
                        f32_to_half_bits<true>(ldexpf(hv, -ex));
                    if ((r & 15) == 0) {
                        a.h_exp[at * (a.n / 16) + (64 * c.tn + 16 * wave) / 16] = (uint8_t)(ex + 128);
                    }
                }
            }
        }
    }
}

template <int BITS, bool DOWN>
__global__ __launch_bounds__(kGemmThreads, 2) void moe_gemm_kernel(GemmArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    __shared__ int src[kTileM];        // row of x
    __shared__ int pair[kTileM];       // DOWN: pair of the row
    __shared__ int most[kTileM];
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
        int first = 0, found = -1, at = 0, end = 0;
        for (int base = 0; base < a.experts && found < 0; base += 256) {  // four experts a lane
            int off[5], tiles = 0, mine = 0;
#pragma unroll
            for (int j = 0; j < 5; ++j) off[j] = a.offsets[min(base + 4 * lane + j, a.experts)];
#pragma unroll
            for (int j = 0; j < 4; ++j) tiles += (off[j + 1] - off[j] + kTileM - 1) / kTileM;
            const int upto = first + wave_scan(tiles);
            const uint64_t past = __builtin_amdgcn_ballot_w64(upto > tile);
            if (past) {
                const int l = __builtin_ctzll(past);
                int below = upto - tiles, e = 0, e_first = 0;  // of lane l: which of its experts
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = (off[j + 1] - off[j] + kTileM - 1) / kTileM;
                    if (tile >= below && tile < below + n) {
                        e = base + 4 * lane + j;
                        e_first = below;
                        at = off[j];
                        mine = off[j + 1];
                    }
                    below += n;
                }
                found = __shfl(e, l, 64);
                first = __shfl(e_first, l, 64);
                at = __shfl(at, l, 64);
                end = __shfl(mine, l, 64);
            } else {
                first = __shfl(upto, 63, 64);
            }
        }
        if (lane == 0) {
            where[0] = found;
            where[1] = at + (tile - first) * kTileM;
            where[2] = end;
        }
    }
    __syncthreads();
    const int e = where[0];
    if (e < 0) return;
    GemmTile c;
    c.row0 = where[1];
    c.rows = min(kTileM, where[2] - c.row0);
    c.tn = tn;
    const int kb = a.k / 32, gpr = kb >> a.gshift, window = window_groups(gpr, a.gshift);

    // rows of x: where they are and their power of two
    for (int i = tid; i < kTileM; i += kGemmThreads) {
        const int at = c.row0 + min(i, c.rows - 1);
        const int p = a.order[at];
        if constexpr (DOWN) {
            const int m = most_of(a.h_exp + (int64_t)at * (a.k / 16), a.k / 16);
            src[i] = at - c.row0;
            pair[i] = p;
            most[i] = m;
            row_scale[i] = a.weights[p] * ldexpf(1.f, m - 128);
        } else {
            src[i] = p / a.top_k;
            row_scale[i] = a.x_scale[p / a.top_k];
        }
    }

    // this wave's weight rows: gate rows 64 tn + 16 wave + r and the up rows of the same columns, or 128 tn + ...
    c.wrow = DOWN ? 128 * tn + 32 * wave + r : 64 * tn + 16 * wave + (r & 15);
    const ExpertWeight& W = !DOWN && r >= 16 ? a.w1 : a.w0;
    const int64_t wr = (int64_t)e * a.n + min(c.wrow, a.n - 1);
    c.pw = W.packed + wr * kb * BITS;

    // Scales and biases to LDS, times the power of two of the row: the largest scale 2^24 lies in [2^14, 2^15). First as
    // they are, eight groups a load (the lanes of a row take eights in turn), then changed where they lie.
    c.sp = W.scales + wr * gpr;
    c.bp = W.biases + wr * gpr;
    c.sb = reinterpret_cast<uint32_t*>(smem + kStages * kStageBytes) + (32 * wave + r) * (window + 1);
    auto value = [&](uint32_t v) { return a.f16 ? half_to_f32<true>(v) : half_to_f32<false>(v); };
    float top = 0.f;
    auto see = [&](uint32_t v) { top = fmaxf(top, fmaxf(fabsf(value(v)), fabsf(value(v >> 16)) * 0x1p-20f)); };
    auto both = [](uint32_t s, uint32_t b) { return (s & 0xffffu) | b << 16; };
    for (int g = 8 * h; g < window; g += 16) {
        if (g + 8 <= window) {
            const u32x4h sv = *reinterpret_cast<const u32x4h*>(c.sp + g), bv = *reinterpret_cast<const u32x4h*>(c.bp + g);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                c.sb[g + 2 * q] = __builtin_amdgcn_perm(bv[q], sv[q], 0x05040100u);
                c.sb[g + 2 * q + 1] = __builtin_amdgcn_perm(bv[q], sv[q], 0x07060302u);
            }
        } else {
            for (int q = g; q < window; ++q) c.sb[q] = both(c.sp[q], c.bp[q]);
        }
    }
    for (int g0 = 8 * h; g0 < window; g0 += 16)
#pragma unroll
        for (int q = 0; q < 8; ++q) see(c.sb[min(g0 + q, window - 1)]);
    for (int g = window + 8 * h; g < gpr; g += 16) {  // those past the window count, too
        if (g + 8 <= gpr) {
            const u32x4h sv = *reinterpret_cast<const u32x4h*>(c.sp + g), bv = *reinterpret_cast<const u32x4h*>(c.bp + g);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                see(both(sv[q], bv[q]));
                see(both(sv[q] >> 16, bv[q] >> 16));
            }
        } else {
            for (int q = g; q < gpr; ++q) see(both(c.sp[q], c.bp[q]));
        }
    }
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const int up = min(14 + 127 - max(min((int)(__float_as_uint(top) >> 23), 254), 1), 120);
    for (int g0 = 8 * h; g0 < window; g0 += 16)
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (g0 + q < window) {
                const uint32_t v = c.sb[g0 + q];
                c.sb[g0 + q] = to_window(v, v >> 16, up, a.f16);
            }
    c.up = up;
    c.col_scale = ldexpf(1.f, 24 - up);
    c.xl = smem;
    c.x = DOWN ? a.x + (int64_t)c.row0 * pad_unit(a.k) : a.x;
    c.exps = a.h_exp + (DOWN ? (int64_t)c.row0 * (a.k / 16) : 0);
    c.src = src;
    c.pair = pair;
    c.most = most;
    c.row_scale = row_scale;
    __syncthreads();
    // as many turns as the rows need: 64, 128 or 160 rows (of an expert with 128 rows on average nearly all fit)
    if (c.rows <= 64) gemm_tile<BITS, DOWN, 2>(a, c, tid);
    else if (c.rows <= 128) gemm_tile<BITS, DOWN, 4>(a, c, tid);
    else gemm_tile<BITS, DOWN, 5>(a, c, tid);
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
    s.xh = take(tokens * pad_unit((int)width) * 2);
    s.x_scale = take(tokens * 4);
    s.order = take(pairs * 4);
    s.offsets = take((experts + 1) * 4);
    s.h = take(pairs * pad_unit((int)hidden) * 2);
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

template <int BITS>
hipError_t launch_gemm_path(const MoeArgs& a, bool f16, hipStream_t stream) {
    const int64_t pairs = a.tokens * a.top_k;
    const MoeSpace s = moe_gemm_space(a.tokens, a.width, a.hidden, a.top_k, a.experts);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    uint16_t* xh = reinterpret_cast<uint16_t*>(ws + s.xh);
    float* x_scale = reinterpret_cast<float*>(ws + s.x_scale);
    int32_t* order = reinterpret_cast<int32_t*>(ws + s.order);
    int32_t* offsets = reinterpret_cast<int32_t*>(ws + s.offsets);
    GemmArgs g{};
    g.h = reinterpret_cast<uint16_t*>(ws + s.h);
    const dim3 sort((unsigned)(a.experts + (a.tokens + kSortThreads / 64 - 1) / (kSortThreads / 64)));
    if (f16)
        moe_sort_kernel<true><<<sort, dim3(kSortThreads), 0, stream>>>(a.chosen, pairs, a.experts, order, offsets, a.x, a.tokens,
                                                                       a.width, xh, x_scale, BITS == 4, a.hidden, g.h);
    else
        moe_sort_kernel<false><<<sort, dim3(kSortThreads), 0, stream>>>(a.chosen, pairs, a.experts, order, offsets, a.x, a.tokens,
                                                                        a.width, xh, x_scale, BITS == 4, a.hidden, g.h);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    g.order = order;
    g.offsets = offsets;
    g.weights = a.weights;
    g.top_k = a.top_k;
    g.experts = a.experts;
    g.gshift = a.group == 32 ? 0 : a.group == 64 ? 1 : 2;
    g.f16 = f16;
    const int64_t tiles = gemm_tiles(a);
    g.x = xh;
    g.x_scale = x_scale;
    g.w0 = a.gate;
    g.w1 = a.up;
    g.h_exp = ws + s.h_exp;
    g.k = a.width;
    g.n = a.hidden;
    g.tiles_n = (a.hidden + 63) / 64;
    moe_gemm_kernel<BITS, false><<<dim3((unsigned)(tiles * g.tiles_n)), dim3(kGemmThreads),
                                   gemm_lds_bytes(a.width, g.gshift), stream>>>(g);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    g.x = g.h;
    g.w0 = g.w1 = a.down;
    g.d = reinterpret_cast<float*>(ws + s.d);
    g.k = a.hidden;
    g.n = a.width;
    g.tiles_n = (a.width + 127) / 128;
    moe_gemm_kernel<BITS, true><<<dim3((unsigned)(tiles * g.tiles_n)), dim3(kGemmThreads),
                                  gemm_lds_bytes(a.hidden, g.gshift), stream>>>(g);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    return f16 ? launch_combine<true>(a, g.d, stream) : launch_combine<false>(a, g.d, stream);
}

// Whether the GEMM serves a call: from an average of 20 rows an expert on (128 x [768, 2048] in 4 bits, 8 experts a token:
// 376 tokens, 23.5 rows, take 171 us with it and 218 with the kernels for few rows; at 256 tokens, 16 rows, one pass
// of those, they take 162), or of two of their passes where rows are so long that LDS holds fewer than 10 (8 x [8192, 8192]:
// 80 tokens of 2 experts, 20 rows, 405 us with it, 64 tokens, 16 rows, 697 with the others in two passes;
// 8 x [14336, 4096], four rows a pass: 64 tokens 387 against 685), as long as a launch holds the tiles (2^32 threads) and
// x is addressed in 32 bits.
inline bool gemm_path(const MoeArgs& a) {
    const int64_t widest = std::max(a.hidden / 64, a.width / 128) + 1, pairs = a.tokens * a.top_k;
    const int64_t row = 2 * (int64_t)std::max(a.hidden, a.width) + 16;
    int64_t pass = kTileRows;  // rows that LDS holds for the other kernels
    while (pass > 1 && pass * row > 140 * 1024) pass /= 2;
    return pairs >= std::min((int64_t)20, 2 * pass) * a.experts && a.tokens * pad_unit(a.width) < (int64_t)1 << 31 &&
           gemm_tiles(a) * widest < (int64_t)1 << 24;
}

}  // namespace
}  // namespace qaff
