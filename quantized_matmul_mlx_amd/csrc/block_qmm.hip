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
#include "wave.h"

#include <algorithm>

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

// A lane's 32 values of the block at p, of which `left` bytes are there: the pieces of 16 at 16 g and 64 + 16 g (four
// lanes of a row read 64 bytes side by side). What is not there is 0.
__device__ __forceinline__ i32x8 load_block32(const uint8_t* p, int g, int64_t left) {
    u32x4a lo = u32x4a{0u, 0u, 0u, 0u}, hi = lo;
    if (left >= kBlock) {
        const u32x4b a = *reinterpret_cast<const u32x4b*>(p + 16 * g), b = *reinterpret_cast<const u32x4b*>(p + 64 + 16 * g);
        lo = u32x4a{a.x, a.y, a.z, a.w};
        hi = u32x4a{b.x, b.y, b.z, b.w};
    } else {
        for (int i = 0; i < 16; ++i) {
            if (16 * g + i < left) lo[i >> 2] |= (uint32_t)p[16 * g + i] << (8 * (i & 3));
            if (64 + 16 * g + i < left) hi[i >> 2] |= (uint32_t)p[64 + 16 * g + i] << (8 * (i & 3));
        }
    }
    return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// ---- few rows ---------------------------------------------------------------------------------------
//
// 16 MT x 16 NT outputs a workgroup, whose waves take the blocks of K in turn, each straight from memory (x from L2)
// into operands, two blocks ahead; no wave waits for another before their sums meet in LDS. The scales of x are
// in LDS from the start. With TAIL the last block of K is not whole.

constexpr int kFewWaves = 8;

inline int few_lds(int mt, int nt, int64_t kb) {
    return (int)std::max((int64_t)mt * 16 * 4 * kb, (int64_t)kFewWaves * mt * nt * 64 * 16);
}
constexpr int kFewMaxLds = 152 * 1024;

template <int MT, int NT, bool TAIL>
__global__ __launch_bounds__(64 * kFewWaves) void qmm_few_kernel(BlockQmmArgs a) {
    extern __shared__ __attribute__((aligned(16))) float lds[];  // scales [kb][16 MT], then sums [wave][tile][lane][4]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NT), m0 = (int64_t)blockIdx.y * (16 * MT);
    const int kb = (int)((a.k + kBlock - 1) / kBlock), whole = (int)(a.k / kBlock);
    const uint8_t *xp[MT], *wp[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i) xp[i] = a.x + min(m0 + 16 * i + r16, a.m - 1) * a.k;
#pragma unroll
    for (int j = 0; j < NT; ++j) wp[j] = a.w + min(n0 + 16 * j + r16, a.n - 1) * a.k;
    const float* ws = a.w_scales + n0 / kBlock * kb;  // NT tiles lie in one block of 128 columns

    struct Ahead {
        i32x8 x[MT], w[NT];
        float s;
    };
    // Each workgroup begins at another block of K: rows 4 KB apart share a channel of L2 block by block, and with all
    // workgroups at the same one loads take longer ([1, 4096] x [4096, 4096]: 5.5 us against
    // 6.6, [61, 4096] x [14336, 4096]: 30.5 against 35.5).
    const int first = whole > 0 ? (int)((uint32_t)blockIdx.x * 5u % (uint32_t)whole) : 0;
    auto block_of = [&](int b) {
        const int at = wave + b * kFewWaves + first;
        return at < whole ? at : at - whole;
    };
    auto load = [&](Ahead& s, int, int b) {
        const int64_t at = (int64_t)block_of(b) * kBlock;
#pragma unroll
        for (int j = 0; j < NT; ++j) s.w[j] = load_block32(wp[j] + at, g, kBlock);
#pragma unroll
        for (int i = 0; i < MT; ++i) s.x[i] = load_block32(xp[i] + at, g, kBlock);
        s.s = ws[block_of(b)];
    };
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto products = [&](const Ahead& s, int block) {
        f16x8 w[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) w[j][q] = half8(s.w[j], q);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            f32x4 d[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f16x8 x = half8(s.x[i], q);
#pragma unroll
                for (int j = 0; j < NT; ++j) d[j] = mfma16x16x32<true>(x, w[j][q], d[j]);
            }
            f32x4 scale = *reinterpret_cast<const f32x4*>(lds + block * (16 * MT) + 16 * i + 4 * g);
#pragma unroll
            for (int v = 0; v < 4; ++v) scale[v] *= s.s;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][j][v] = __builtin_fmaf(scale[v], d[j][v], acc[i][j][v]);
        }
    };
    const int items = (whole - wave + kFewWaves - 1) / kFewWaves;
    Ahead A, B;
    if (items > 0) {
        load(A, 0, 0);
        load(B, 0, min(1, items - 1));
    }
    for (int i = tid; i < 16 * MT * kb; i += 64 * kFewWaves) {  // rows follow each other: whole rows are read
        const int row = i / kb, b = i % kb;
        lds[b * (16 * MT) + row] = a.x_scales[min(m0 + row, a.m - 1) * kb + b];
    }
    __syncthreads();
    if (items > 0)
        pipeline(items, items, A, B, load, [&](const Ahead& s, int, int b) { products(s, block_of(b)); });
    if constexpr (TAIL) {
        if (whole % kFewWaves == wave) {
#pragma unroll
            for (int j = 0; j < NT; ++j) A.w[j] = load_block32(wp[j] + (int64_t)whole * kBlock, g, a.k % kBlock);
#pragma unroll
            for (int i = 0; i < MT; ++i) A.x[i] = load_block32(xp[i] + (int64_t)whole * kBlock, g, a.k % kBlock);
            A.s = ws[whole];
            products(A, whole);
        }
    }
    __syncthreads();  // nobody reads scales any more
    f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) red[((wave * MT + i) * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int t = wave; t < MT * NT; t += kFewWaves) {
        f32x4 sum = red[t * 64 + lane];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) sum += red[(w * MT * NT + t) * 64 + lane];
        const int64_t n = n0 + t % NT * 16 + r16;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int64_t m = m0 + t / NT * 16 + 4 * g + v;
            if (m < a.m && n < a.n) store_from_f32(a.y, (size_t)(m * a.n + n), a.dtype, sum[v]);
        }
    }
}

template <int MT, int NT>
hipError_t launch_few(const BlockQmmArgs& a, hipStream_t stream) {
    const int64_t kb = (a.k + kBlock - 1) / kBlock, rows = (int64_t)65535 * 16 * MT;  // a grid's second axis
    for (int64_t m0 = 0; m0 < a.m; m0 += rows) {
        BlockQmmArgs p = a;
        p.m = std::min(rows, a.m - m0);
        p.x += m0 * a.k;
        p.x_scales += m0 * kb;
        p.y = static_cast<char*>(a.y) + m0 * a.n * (a.dtype == 0 ? 4 : 2);
        const dim3 grid((unsigned)((a.n + 16 * NT - 1) / (16 * NT)), (unsigned)((p.m + 16 * MT - 1) / (16 * MT)));
        if (a.k % kBlock) qmm_few_kernel<MT, NT, true><<<grid, dim3(64 * kFewWaves), few_lds(MT, NT, kb), stream>>>(p);
        else qmm_few_kernel<MT, NT, false><<<grid, dim3(64 * kFewWaves), few_lds(MT, NT, kb), stream>>>(p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Columns a workgroup: 64, 32 or 16, the most that still give every compute unit one.
template <int MT>
hipError_t launch_few_rows(const BlockQmmArgs& a, hipStream_t stream) {
    const int64_t tiles = ((a.m + 16 * MT - 1) / (16 * MT)) * ((a.n + 15) / 16), cus = device_cu_count();
    if (tiles >= 4 * cus) return launch_few<MT, 4>(a, stream);
    if (tiles >= 2 * cus) return launch_few<MT, 2>(a, stream);
    return launch_few<MT, 1>(a, stream);
}

// ---- tiles -----------------------------------------------------------------------------------------
//
// More rows: a workgroup has 16 MT x 16 WAVES NT outputs, wave w the columns 16 NT w of them and all rows. With SPLIT
// it has that many sets of waves, each for a part of K with stages of its own; their sums meet in LDS in the end.
//  * w goes straight from memory into the products' operands, three blocks of K ahead in registers: no
//    wave shares its rows, and LDS, which the rows of x already fill, carries it not.
//  * x goes through LDS, three blocks of it there at a time (16-byte pieces, swapped within a row by half the row's
//    number so that 16 rows at one offset fall on distinct banks), with the products of its and w's scales beside it.
//  * One v_mfma_f32_16x16x128_f8f6f4 is a block of K for 16 x 16 outputs (32 cycles); its four results a
//    lane enter the totals with the scales by four multiply-adds (16 cycles), those of the previous 16 rows
//    while the products of these run.
//  * EXACT: products of float16 operands instead, for float32 outputs (the others have 16 bits).
// A lane's 32 values of a block are the pieces lane / 16 and 4 + lane / 16, of x and w alike.
// Measured: [2048, 14336] x [4096, 14336] 156 to 163 us, 1.5 PFLOP/s (its products and scaling alone would allow 3.5), bound by
// LDS reads of x (40 us of it), vector memory instructions (35) and misses of L2 (24); [61, 4096] x [14336, 4096], K in two
// parts, 16.4 us, 3.7 TB/s.

__device__ __forceinline__ f32x4 mfma_f8(i32x8 a, i32x8 b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

template <int T> struct Type { static constexpr int value = T; };

// TAIL: k is not a multiple of 128 (but of 16): the last block's pieces past the end are 0 in w.
template <int WAVES, int MT, int NT, int SPLIT, bool EXACT, bool TAIL>
__global__ __launch_bounds__(64 * WAVES * SPLIT) void qmm_tile_kernel(BlockQmmArgs a, int tiles_m, int tiles_n) {
    constexpr int kThreads = 64 * WAVES, kRows = 16 * MT, kCols = 16 * WAVES * NT;
    constexpr int kPieces = kRows * 8 / kThreads;  // pieces of x a thread and block
    constexpr int kScales = (kCols + kBlock - 1) / kBlock;  // blocks of 128 columns
    constexpr int kPanel = kThreads / kRows;       // blocks of K whose scales are loaded together
    constexpr int kStages = 3;
    __shared__ __attribute__((aligned(16))) uint8_t x_all[SPLIT][kStages][kRows * kBlock];
    __shared__ __attribute__((aligned(16))) float s_all[SPLIT][2][kPanel][kScales][kRows];
    const int part = SPLIT > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads) : 0;
    auto& xl = x_all[part];
    auto& sl = s_all[part];
    const int tid = threadIdx.x % kThreads, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int tm = blockIdx.x % tiles_m, tn = blockIdx.x / tiles_m;
    const int64_t m0 = (int64_t)tm * kRows, n0 = (int64_t)tn * kCols;
    const int kb = (int)((a.k + kBlock - 1) / kBlock);
    // This part's blocks: `own` from b0 on (at least one; `turns` count), in the order at(0), at(1), ...; past them it
    // repeats others, whose scales are stored as 0.
    const int turns = (kb + SPLIT - 1) / SPLIT, b0 = min(part * turns, kb - 1), count = min(turns, kb - part * turns);
    const int own = max(count, 1), first = SPLIT > 1 ? (int)((uint32_t)tn * 5u % (uint32_t)own) : 0;
    auto at = [&](int b) {
        const int i = b + first;
        return b0 + min(i < own ? i : i - own, own - 1);
    };

    // this thread's pieces of x: row and place in LDS; its scales: row tid % kRows, block tid / kRows of a panel
    const uint8_t* xp[kPieces];
    int slot[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int row = (i * kThreads + tid) / 8;
        xp[i] = a.x + min(m0 + row, a.m - 1) * a.k;
        slot[i] = row * kBlock + ((tid & 7) ^ (row >> 1 & 7)) * 16;
    }
    const int scale_row = tid % kRows, scale_block = tid / kRows;
    const float* xsp = a.x_scales + min(m0 + scale_row, a.m - 1) * kb;
    const uint8_t* wp[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) wp[j] = a.w + min(n0 + wave * 16 * NT + 16 * j + r16, a.n - 1) * a.k;

    struct Ahead {
        u32x4a x[kPieces];
        u32x4a lo[NT], hi[NT];
    };
    struct Scales {
        float x, w[kScales];
    };
    auto load_x = [&](Ahead& s, int b) {
        b = at(b);
        const int left = TAIL ? (int)min(a.k - (int64_t)b * kBlock, (int64_t)kBlock) : kBlock;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)  // a piece past the row's end repeats the last one: w is 0 there
            s.x[i] = *reinterpret_cast<const u32x4a*>(xp[i] + (int64_t)b * kBlock + min(16 * (tid & 7), left - 16));
    };
    auto load_w = [&](Ahead& s, int b) {
        b = at(b);
        const int left = TAIL ? (int)min(a.k - (int64_t)b * kBlock, (int64_t)kBlock) : kBlock;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            s.lo[j] = *reinterpret_cast<const u32x4a*>(wp[j] + (int64_t)b * kBlock + min(16 * g, left - 16));
            s.hi[j] = *reinterpret_cast<const u32x4a*>(wp[j] + (int64_t)b * kBlock + min(64 + 16 * g, left - 16));
        }
    };
    auto load_scales = [&](Scales& s, int panel) {
        const int b = at(panel * kPanel + scale_block);
        s.x = xsp[b];
#pragma unroll
        for (int i = 0; i < kScales; ++i) s.w[i] = a.w_scales[min(n0 / kBlock + i, (a.n - 1) / kBlock) * kb + b];
    };
    auto store_scales = [&](const Scales& s, int panel) {
#pragma unroll
        for (int i = 0; i < kScales; ++i)
            sl[panel & 1][scale_block][i][scale_row] = panel * kPanel + scale_block < count ? s.x * s.w[i] : 0.f;
    };
    auto operand = [&](const Ahead& s, int j, int b) {
        u32x4a lo = s.lo[j], hi = s.hi[j];
        if constexpr (TAIL) {
            const int64_t left = a.k - (int64_t)at(b) * kBlock;
            if (16 * g >= left) lo = u32x4a{0u, 0u, 0u, 0u};
            if (64 + 16 * g >= left) hi = u32x4a{0u, 0u, 0u, 0u};
        }
        return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
    auto store_x = [&](const Ahead& s, int stage) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) *reinterpret_cast<u32x4a*>(&xl[stage][slot[i]]) = s.x[i];
    };

    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // x operand and scales of 16 rows. Read one turn ahead, over the border of two blocks too.
    const int p0 = r16 * kBlock + (g ^ (r16 >> 1)) * 16, p1 = r16 * kBlock + ((4 + g) ^ (r16 >> 1)) * 16;
    const int sw = wave * 16 * NT / kBlock;
    i32x8 x[2];
    f32x4 scale[3], d[2][NT];
    auto read = [&](int stage, int b, int i) {
        const u32x4a lo = *reinterpret_cast<const u32x4a*>(&xl[stage][16 * i * kBlock + p0]);
        const u32x4a hi = *reinterpret_cast<const u32x4a*>(&xl[stage][16 * i * kBlock + p1]);
        x[i & 1] = i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
    auto read_scale = [&](int b, int i, int to) {
        scale[to] = *reinterpret_cast<const f32x4*>(&sl[b / kPanel & 1][b % kPanel][sw][16 * i + 4 * g]);
    };
    static_assert(MT % 2 == 0, "a block's first turn follows an odd one");
    auto products = [&](const Ahead& s, int b, int stage) {
        i32x8 w[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) w[j] = operand(s, j, b);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if (i + 1 < MT) read(stage, b, i + 1);
            else read((stage + 1) % kStages, b + 1, 0);
            // each product is followed by the scaling of the same columns one turn before (16 rows above, or the
            // last rows of the block before); the compiler would put the scaling first, where its operands are
            // not there yet
            f32x4 now = scale[0];
            read_scale(i + 1 < MT ? b : b + 1, (i + 1) % MT, 0);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                d[i & 1][j] = EXACT ? block_sums(x[i & 1], w[j]) : mfma_f8(x[i & 1], w[j]);
                __builtin_amdgcn_sched_barrier(0);
                f32x4& sum = acc[(i + MT - 1) % MT][j];
#pragma unroll
                for (int v = 0; v < 4; ++v) sum[v] = __builtin_fmaf(scale[1][v], d[(i + 1) & 1][j][v], sum[v]);
                asm volatile("" : "+v"(sum));  // here, not sunk past the branches below, with its operands kept alive
                __builtin_amdgcn_sched_barrier(0);
            }
            scale[1] = now;
        }
    };

    Ahead s[3];
    Scales sc;
    load_scales(sc, 0);
    load_x(s[0], 0);
    load_x(s[1], 1);
    load_w(s[0], 0);
    store_scales(sc, 0);
    load_scales(sc, 1);
    store_x(s[0], 0);
    store_x(s[1], 1);
    load_x(s[2], 2);
    load_w(s[1], 1);
    load_x(s[0], 3);
    load_w(s[2], 2);
    load_x(s[1], 4);
#pragma unroll
    for (int j = 0; j < NT; ++j) d[1][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    scale[1] = f32x4{0.f, 0.f, 0.f, 0.f};
    __syncthreads();
    read(0, 0, 0);
    read_scale(0, 0, 0);
    for (int b = 0; b < turns; b += 3) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            // After this barrier nobody reads block b + i - 1 any more, whose place block b + i + 2 takes; block
            // b + i + 1, stored one turn ago, is there.
            __syncthreads();
            store_x(s[(i + 2) % 3], (i + 2) % 3);
            load_x(s[(i + 2) % 3], b + i + 5);
            if ((b + i) % kPanel == 0) {  // the panel of the blocks b + i + kPanel ..
                store_scales(sc, (b + i) / kPanel + 1);
                load_scales(sc, (b + i) / kPanel + 2);
            }
            products(s[i], b + i, i);
            load_w(s[i], b + i + 3);
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[MT - 1][j][v] = __builtin_fmaf(scale[1][v], d[1][j][v], acc[MT - 1][j][v]);
    if constexpr (SPLIT > 1) {  // the parts' sums, in order
        static_assert(sizeof(x_all) >= (SPLIT - 1) * WAVES * MT * NT * 1024, "");
        f32x4* red = reinterpret_cast<f32x4*>(&x_all[0][0][0]);
        auto place = [&](int p, int i, int j) { return (((p - 1) * WAVES + wave) * MT * NT + i * NT + j) * 64 + lane; };
        __syncthreads();  // nobody reads x any more
        if (part > 0)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) red[place(part, i, j)] = acc[i][j];
        __syncthreads();
        if (part > 0) return;
#pragma unroll
        for (int p = 1; p < SPLIT; ++p)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[i][j] += red[place(p, i, j)];
    }
    auto store = [&](auto type) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int64_t m = m0 + 16 * i + 4 * g + v;
                if (m >= a.m) continue;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int64_t n = n0 + wave * 16 * NT + 16 * j + r16;
                    if (n < a.n) store_from_f32(a.y, (size_t)(m * a.n + n), type.value, acc[i][j][v]);
                }
            }
    };
    if (EXACT) store(Type<0>());
    else if (a.dtype == 1) store(Type<1>());
    else store(Type<2>());
}

template <int WAVES, int MT, int NT, int SPLIT>
hipError_t launch_tiles(const BlockQmmArgs& a, hipStream_t stream) {
    const int tiles_m = (int)((a.m + 16 * MT - 1) / (16 * MT));
    const int tiles_n = (int)((a.n + 16 * WAVES * NT - 1) / (16 * WAVES * NT));
    const dim3 grid((unsigned)tiles_m * (unsigned)tiles_n), block(64 * WAVES * SPLIT);
    if (a.k % kBlock) {
        if (a.dtype == 0) qmm_tile_kernel<WAVES, MT, NT, SPLIT, true, true><<<grid, block, 0, stream>>>(a, tiles_m, tiles_n);
        else qmm_tile_kernel<WAVES, MT, NT, SPLIT, false, true><<<grid, block, 0, stream>>>(a, tiles_m, tiles_n);
    } else {
        if (a.dtype == 0) qmm_tile_kernel<WAVES, MT, NT, SPLIT, true, false><<<grid, block, 0, stream>>>(a, tiles_m, tiles_n);
        else qmm_tile_kernel<WAVES, MT, NT, SPLIT, false, false><<<grid, block, 0, stream>>>(a, tiles_m, tiles_n);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_qmm(const BlockQmmArgs& a, hipStream_t stream) {
    const bool aligned = a.k > 0 && a.k % 16 == 0 && (uintptr_t)a.x % 16 == 0 && (uintptr_t)a.w % 16 == 0;
    const int64_t cus = device_cu_count();
    auto tiles = [&](int rows, int cols) { return ((a.m + rows - 1) / rows) * ((a.n + cols - 1) / cols); };
    // Tiles of 128 x 256 where half the compute units get one ([1280, 4096] x [4096, 4096], 160 of them: 48 us against 66
    // with 64 x 128; [512, 4096], 64 of them, would leave most units idle: 25 with 64 x 128). Below that 64 x 64 with K
    // split where each unit gets one at most, and 64 x 128 otherwise ([256, 4096] x [4096, 4096], 256 tiles of 64 x 64:
    // 18.6 against 22; [512, 4096], 512 of them: 31 against 25). From 17 rows of x on where half the units get a tile of
    // 64 x 64: [61, 4096] x [14336, 4096] 17 against 29.7 us with the kernel for few rows, [64, 8192] x [8192, 8192]
    // 25.9 against 28, but [64, 4096] x [4096, 4096] 15.9 against 13.8; from 65 rows on always, since that kernel
    // would read w more than once.
    if (aligned && a.m > 16 && a.m * a.n < (int64_t)1 << 40) {
        if (a.m > 64 && tiles(128, 256) >= cus / 2) return launch_tiles<8, 8, 2, 1>(a, stream);
        if (tiles(64, 64) > cus) return launch_tiles<4, 4, 2, 1>(a, stream);
        if (a.m > 64 || tiles(64, 64) >= cus / 2) return launch_tiles<4, 4, 1, 2>(a, stream);
    }
    const int64_t kb = (a.k + kBlock - 1) / kBlock;
    if (a.m > 32 && few_lds(4, 4, kb) <= kFewMaxLds) return launch_few_rows<4>(a, stream);
    if (a.m > 16 && few_lds(2, 4, kb) <= kFewMaxLds) return launch_few_rows<2>(a, stream);
    return launch_few_rows<1>(a, stream);
}

}  // namespace qaff
