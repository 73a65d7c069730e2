// The layer of a mixture of experts for few rows an expert (moe.hip: fewer than 20 on average): products of gathered
// rows with each expert's weights, read once for up to 16 rows.
//
//   h[p] = silu(gate[e] x[t]) * (up[e] x[t]),  d[p] = weight[p] down[e] h[p],  p = (t, j), e = chosen[p]
//   y[t] = resid[t] + sum_j d[t, j]
//
// Bound by the weights' way from memory: at 4 bits a row of 16 x 16 products takes 8 bytes of codes and
// 512 multiply-adds of the matrix cores, which wait most of the time.
//  * Codes enter the products exactly, as B + c (an AND and an OR put codes into the mantissas of B), and
//    each group's scale and bias are applied to the group's sums:
//      sum x (s c + b) = s sum x (B + c) + (b - B s) sum x.
//    No weight is rounded, and the sums of x come from LDS, where they are formed once a workgroup.
//    Measured (kernels alone): 64 tokens through 8 of 128 x [768, 2048], 4 bits: gate and up 58 us, down 34, combine 6.7,
//    340 MB in all, 3.5 TB/s; one token, each pair alone: 7.9 and 7.4 us.
//  * h = silu(g) u is rounded to the type of x: the matrix instructions take 16-bit operands of one type, and x and
//    the code operands B + c have that one. d, its sum over a token and both products' sums are float32.
//  * v_mfma_f32_16x16x32: a lane loads a whole block of 32 codes (16 bytes at 4 bits) of weight row
//    lane % 16, block lane / 16 of a chunk of 128. A product may only cover one group, so for groups of
//    64 and 32 the lanes exchange halves and quarters of their blocks (v_permlane32_swap, v_permlane16_swap)
//    and read x in the order that results.
#pragma once

#include "ffn.h"
#include "mfma16.h"
#include "wave.h"

#include <hip/hip_runtime.h>

#include <algorithm>

namespace qaff {
namespace {

typedef uint32_t u32x4h __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2h __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32h __attribute__((aligned(2)));

constexpr int kTileRows = 16;  // rows of x a pass
// Chunks of 128 codes that are loaded together: two units of two weights are in registers at a time.
template <int BITS> constexpr int kUnit = BITS <= 4 ? 2 : 1;
constexpr int kFewWaves = 4;
constexpr int kFewBlocks = 3;  // workgroups a compute unit (168 registers a lane)
constexpr int kFewThreads = 64 * kFewWaves;

struct FewArgs {
    const uint16_t* x;           // rows of k values
    ExpertWeight w0, w1;         // of n rows of k codes each (w1: the up weight)
    const int32_t* chosen;       // [pairs]
    const float* weights;        // [pairs]
    void* out;                   // [pairs, n]
    int64_t pairs;
    int k, kpad, n, top_k, experts;
    int rows;                    // rows of x in LDS (1 to 16)
    int ksplit;                  // waves that share a tile's K
};

// ---- codes as operands ----------------------------------------------------------------------------

// B of the exact operands: 128 + c has 8 bits for codes of up to 6 bits; 8-bit codes are bf16 values
// themselves. float16 holds 1024 + c.
template <bool F16, int BITS> constexpr float kCodeBase = F16 ? 1024.f : BITS == 8 ? 0.f : 128.f;

// The mask of two 4-bit codes in a scalar and B (both halves) in a vector register, for one v_and_or_b32 for two codes.
struct CodeConsts {
    uint32_t mask, base;
};
template <bool F16> __device__ __forceinline__ CodeConsts make_code_consts() {
    uint32_t base = F16 ? 0x64006400u : 0x43004300u;
    asm volatile("" : "+v"(base));
    return CodeConsts{(uint32_t)__builtin_amdgcn_readfirstlane(0x000F000F), base};
}

template <bool F16, int BITS>
__device__ __forceinline__ u32x4a code_operand(const uint32_t (&w)[BITS], int j, const CodeConsts& cc) {
    const uint32_t base = cc.base;
    u32x4a o;
    if constexpr (BITS == 4) {  // pairs (c0, c4), (c1, c5), (c2, c6), (c3, c7): x is staged in that order
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = ((w[j] >> (4 * e)) & cc.mask) | base;
    } else if constexpr (BITS == 8 && F16) {  // bytes of the word between bytes of the base
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = __builtin_amdgcn_perm(0x64646464u, w[2 * j + (e >> 1)], e & 1 ? 0x04030402u : 0x04010400u);
    } else if constexpr (BITS == 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t v = w[2 * j + (e >> 1)] >> (e & 1 ? 16 : 0);
            o[e] = pack_bf16x2((float)(v & 0xffu), (float)((v >> 8) & 0xffu));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = code_at<BITS>(w, 8 * j + 2 * e) | code_at<BITS>(w, 8 * j + 2 * e + 1) << 16 | base;
    }
    return o;
}

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// Four registers of lane group g (lane / 16), register j holding octet j of block g of a chunk, into
// registers that hold one group each: groups of 64: registers 2 p and 2 p + 1 hold group p; of 32: register
// i holds block i. x_offset is the code that the lane's octet of register i then starts with.
template <int GSHIFT>
__device__ __forceinline__ void regroup(uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    if constexpr (GSHIFT < 2) {
        swap32(r0, r2);  // r0: octets 0 (lower half), 2 (upper) of blocks 0, 1; r2: of blocks 2, 3
        swap32(r1, r3);
    }
    if constexpr (GSHIFT == 0) {
        swap16(r0, r1);  // r0: octets 0 .. 3 of block 0; r1: of block 1
        swap16(r2, r3);
    }
}
template <int GSHIFT> __device__ __forceinline__ int x_lane_offset(int g) {
    return GSHIFT == 2 ? 32 * g : GSHIFT == 1 ? 32 * (g & 1) + 16 * (g >> 1) : 8 * g;
}
template <int GSHIFT> constexpr int x_step_offset(int i) {
    return GSHIFT == 2 ? 8 * i : GSHIFT == 1 ? 64 * (i >> 1) + 8 * (i & 1) : 32 * i;
}

// The operands of one chunk, register i of lane group g as x_lane_offset + x_step_offset say.
template <bool F16, int BITS, int GSHIFT>
__device__ __forceinline__ void chunk_operands(const uint32_t (&w)[BITS], const CodeConsts& cc, op8<F16> (&o)[4]) {
    if constexpr (BITS == 4) {  // an octet is a word: exchanged before it is spread
        uint32_t v[4] = {w[0], w[1], w[2], w[3]};
        regroup<GSHIFT>(v[0], v[1], v[2], v[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = __builtin_bit_cast(op8<F16>, code_operand<F16, 4>(v, j, cc));
    } else {
        u32x4a v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = code_operand<F16, BITS>(w, j, cc);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t r0 = v[0][e], r1 = v[1][e], r2 = v[2][e], r3 = v[3][e];
            regroup<GSHIFT>(r0, r1, r2, r3);
            v[0][e] = r0; v[1][e] = r1; v[2][e] = r2; v[3][e] = r3;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = __builtin_bit_cast(op8<F16>, v[j]);
    }
}

// ---- loads ------------------------------------------------------------------------------------------

// A unit's codes, scales and biases of one weight row: kUnit blocks of this lane, and the unit's groups, as many as
// a whole unit has. `over`: groups that the window had to start early to stay inside the tensor.
template <int BITS, int GSHIFT> struct UnitLoads {
    static constexpr int kGroups = kUnit<BITS> * 4 >> GSHIFT;
    static constexpr int kWords = (kGroups + 1) / 2;
    uint32_t w[kUnit<BITS>][BITS];
    uint32_t s[kWords], b[kWords];
    int over;
};

template <int WORDS> __device__ __forceinline__ void load_halves(const uint16_t* p, uint32_t (&o)[WORDS]) {
    if constexpr (WORDS == 4) {
        const u32x4h v = *reinterpret_cast<const u32x4h*>(p);
        o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
    } else if constexpr (WORDS == 2) {
        const u32x2h v = *reinterpret_cast<const u32x2h*>(p);
        o[0] = v.x; o[1] = v.y;
    } else {
        o[0] = *reinterpret_cast<const u32h*>(p);
    }
}

// One expert's part of a weight: rows of kb blocks, and how many halves of scales lie from its first on to the end of
// the tensor (at most 2^31 - 1 of them matter).
struct ExpertRows {
    const uint32_t* packed;
    const uint16_t *scales, *biases;
    int kb, halves;
};
template <int BITS, int GSHIFT>
__device__ __forceinline__ ExpertRows expert_rows(const ExpertWeight& W, int e, int experts, int n, int kb) {
    const int64_t gpr = kb >> GSHIFT, row = (int64_t)e * n;
    const int64_t halves = ((int64_t)experts * n - row) * gpr;
    return ExpertRows{W.packed + row * kb * BITS, W.scales + row * gpr, W.biases + row * gpr, kb,
                      (int)(halves < 0x7fffffff ? halves : 0x7fffffff)};
}

// Unit u of row `row` (an expert's codes and groups are counted in 32 bits: 2^15 rows of 2^15 codes at most). The blocks
// past the row's end repeat its last one (x is 0 there); the groups past it are the next row's, and are masked where
// they are used.
template <int BITS, int GSHIFT>
__device__ __forceinline__ void load_unit(UnitLoads<BITS, GSHIFT>& L, const ExpertRows& W, int row, int u, int g) {
    typedef UnitLoads<BITS, GSHIFT> U;
    const int want = row * (W.kb >> GSHIFT) + u * U::kGroups;
    const int at = min(want, W.halves - 2 * U::kWords);  // a tensor has 32 rows at least
    L.over = want - at;
    load_halves(W.scales + (uint32_t)at, L.s);
    load_halves(W.biases + (uint32_t)at, L.b);
#pragma unroll
    for (int c = 0; c < kUnit<BITS>; ++c) {
        const uint32_t block = (uint32_t)(row * W.kb + min(4 * (u * kUnit<BITS> + c) + g, W.kb - 1));
        load_block<BITS>(W.packed + block * BITS, L.w[c]);
    }
}

// The window of a row's last unit, which `there` groups of it fill, moved to its place and masked.
template <int WORDS> __device__ __forceinline__ void mend_window(uint32_t (&w)[WORDS], int over, int there) {
#pragma unroll
    for (int by = 1; by < WORDS; by *= 2)
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = over & 2 * by ? (i + by < WORDS ? w[i + by] : 0u) : w[i];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
        w[i] = over & 1 ? __builtin_amdgcn_alignbit(i + 1 < WORDS ? w[i + 1] : 0u, w[i], 16) : w[i];
        w[i] &= there >= 2 * i + 2 ? ~0u : there == 2 * i + 1 ? 0xffffu : 0u;
    }
}

// ---- products ---------------------------------------------------------------------------------------

// acc += x . (unit of a weight)^T. xa: the lane's row of x in LDS at the unit's first code, xs: the sums of x of the
// unit's groups ([group][16 rows], at the lane's four result rows), there: groups of the row from the unit on.
// SUMS: sums of x a group (16 rows', or 1 where all rows are the same).
template <int BITS, int GSHIFT, bool F16, int SUMS = kTileRows>
__device__ __forceinline__ void unit_product(const UnitLoads<BITS, GSHIFT>& L, const uint8_t* xa, const float* xs, int there,
                                             const CodeConsts& cc, f32x4& acc) {
    constexpr int kEach = 1 << GSHIFT;  // products a group
    // copies: were the loaded registers written here, the compiler would copy each load and wait for it there
    constexpr int kWords = UnitLoads<BITS, GSHIFT>::kWords;
    uint32_t sw[kWords], bw[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        sw[i] = L.s[i];
        bw[i] = L.b[i];
    }
    if (there < 2 * kWords) {
        mend_window(sw, L.over, there);
        mend_window(bw, L.over, there);
    }
#pragma unroll
    for (int c = 0; c < kUnit<BITS>; ++c) {
        op8<F16> o[4];
        uint32_t w[BITS];
#pragma unroll
        for (int i = 0; i < BITS; ++i) {
            w[i] = L.w[c][i];
            asm volatile("" : "+v"(w[i]));  // here, not where the loads are issued, which would wait for them
        }
        chunk_operands<F16, BITS, GSHIFT>(w, cc, o);
#pragma unroll
        for (int p = 0; p < (4 >> GSHIFT); ++p) {
            f32x4 d = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int step = p * kEach + i;
                d = mfma16x16x32<F16>(*reinterpret_cast<const op8<F16>*>(xa + 256 * c + 2 * x_step_offset<GSHIFT>(step)),
                                      o[step], d);
            }
            const int grp = (4 * c >> GSHIFT) + p;
            f32x4 sum;
            if constexpr (SUMS == 1) sum = f32x4{xs[grp], xs[grp], xs[grp], xs[grp]};
            else sum = *reinterpret_cast<const f32x4*>(xs + grp * SUMS);
            const float s = half_to_f32<F16>(sw[grp >> 1] >> (16 * (grp & 1)));
            const float b = half_to_f32<F16>(bw[grp >> 1] >> (16 * (grp & 1)));
            const float beta = __builtin_fmaf(-kCodeBase<F16, BITS>, s, b);
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[v] = __builtin_fmaf(s, d[v], __builtin_fmaf(beta, sum[v], acc[v]));
        }
    }
}

// Octet o of a row of x (0 where it is not there) into LDS: the values at xl, in the order of 4-bit operands, and the
// sum of its group at xs, SUMS apart; the lanes of a group come together.
template <int BITS, int GSHIFT, bool F16, int SUMS>
__device__ __forceinline__ void stage_octet(u32x4h h, bool there, int o, uint8_t* xl, float* xs) {
    constexpr int kOct = 4 << GSHIFT;  // octets of a group
    u32x4a v = there ? u32x4a{h.x, h.y, h.z, h.w} : u32x4a{0u, 0u, 0u, 0u};
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) sum += half_to_f32<F16>(v[q]) + half_to_f32<F16>(v[q] >> 16);
#pragma unroll
    for (int d = 1; d < kOct; d <<= 1) sum += __shfl_xor(sum, d, 64);
    if (o % kOct == 0) xs[o / kOct * SUMS] = sum;
    if constexpr (BITS == 4)
        v = u32x4a{__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                   __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u)};
    *reinterpret_cast<u32x4a*>(xl + 16 * o) = v;
}

// Pairs of expert e whose rank lies in [first, first + count) into rows[0 ..), by the whole workgroup; returns how
// many the expert has, up to that point or more. Eight pairs a thread at a time, all of them loaded together;
// counts: LDS for the hits of each 64 of them.
__device__ __forceinline__ int list_rows(const int32_t* chosen, int64_t pairs, int e, int first, int count, int tid,
                                         int* counts, int* rows) {
    const int lane = tid & 63, wave = tid >> 6;
    int rank = 0;
    for (int64_t base = 0; base < pairs && rank <= first + count; base += 8 * kFewThreads) {
        bool mine[8];
        uint64_t hits[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t p = base + i * kFewThreads + tid;
            mine[i] = chosen[min(p, pairs - 1)] == e;  // no branch around the load: the eight go out together
            mine[i] &= p < pairs;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            hits[i] = __builtin_amdgcn_ballot_w64(mine[i]);
            if (lane == 0) counts[i * kFewWaves + wave] = __builtin_popcountll(hits[i]);
        }
        __syncthreads();
        const int own = lane < 8 * kFewWaves ? counts[lane] : 0;
        const int upto = wave_scan(own);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int before = rank - first + __shfl(upto - own, i * kFewWaves + wave, 64);
            const int at = before + __builtin_popcountll(hits[i] & ((1ull << lane) - 1));
            if (mine[i] && at >= 0 && at < count) rows[at] = (int)(base + i * kFewThreads + tid);
        }
        rank += __shfl(upto, 63, 64);
        __syncthreads();  // rows are there; counts are written again
    }
    return rank;
}

// DOWN = false: gate and up, h out (16-bit). DOWN = true: two neighbouring tiles of the down weight, rows
// of d out (float32, times the pair's weight).
//
// A workgroup has x of up to 16 rows of one expert in LDS. Its waves walk 16-row tiles of the two weights, each
// wave a tile of its own, or ksplit waves the parts of K of one tile where there are few tiles (their sums meet in
// LDS). A wave's units of 256 codes, over all its tiles, are one sequence with the next two always on their way,
// also while the workgroup looks for its rows and loads x.
template <int BITS, int GSHIFT, bool F16, bool DOWN>
__global__ __launch_bounds__(kFewThreads, kFewBlocks) void moe_few_kernel(FewArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    __shared__ int rows[kTileRows];
    __shared__ float weight_of[kTileRows];
    __shared__ int counts[8 * kFewWaves];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int e = blockIdx.y;
    const int pitch = 2 * a.kpad + 16;  // 16 rows at one offset fall on distinct banks
    uint8_t* xl = smem;
    float* xs = reinterpret_cast<float*>(smem + (size_t)a.rows * pitch);
    float* red = xs + (a.kpad >> (5 + GSHIFT)) * kTileRows;
    const int kb = a.k / 32, octets = a.kpad / 8;
    constexpr int kTileN = DOWN ? 32 : 16;
    const int tiles = (a.n + kTileN - 1) / kTileN;
    const int side = kFewWaves / a.ksplit;  // tiles at a time
    const int ks = wave % a.ksplit;
    const int units = a.kpad / (128 * kUnit<BITS>), each = (units + a.ksplit - 1) / a.ksplit;
    const int u0 = ks * each;                                // this wave's units of a tile: u0 .. u0 + each - 1
    const int t0 = blockIdx.x * side + wave / a.ksplit;      // and tiles: t0, t0 + step, ...
    const int step = gridDim.x * side;
    const int turns = (tiles - (int)blockIdx.x * side + step - 1) / step;  // the same for all waves

    typedef UnitLoads<BITS, GSHIFT> Unit;
    const ExpertRows w0 = expert_rows<BITS, GSHIFT>(a.w0, e, a.experts, a.n, kb);
    const ExpertRows w1 = expert_rows<BITS, GSHIFT>(a.w1, e, a.experts, a.n, kb);
    // Item (turn, i): unit u0 + i of tile t0 + turn step. Items past the row's end or the last tile repeat others.
    auto load = [&](Unit (&L)[2], int turn, int i) {
        const int n0 = min(t0 + turn * step, tiles - 1) * kTileN + r16;
        const int u = min(u0 + i, units - 1);
        load_unit(L[0], w0, min(n0, a.n - 1), u, g);
        load_unit(L[1], DOWN ? w0 : w1, min(DOWN ? n0 + 16 : n0, a.n - 1), u, g);
    };
    Unit A[2], B[2];
    const CodeConsts cc = make_code_consts<F16>();

    for (int first = 0;; first += a.rows) {
        load(A, 0, 0);
        load(B, each > 1 ? 0 : min(1, turns - 1), each > 1 ? 1 : 0);
        const int total = list_rows(a.chosen, a.pairs, e, first, a.rows, tid, counts, rows);
        if (first >= total) return;
        const int nr = min(a.rows, total - first);
        if constexpr (DOWN)
            if (tid < nr) weight_of[tid] = a.weights[rows[tid]];
        // x of the tile's rows, and its groups' sums
        for (int i0 = tid; i0 < nr * octets; i0 += 4 * kFewThreads) {
            u32x4h h[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // four pieces a thread on their way together
                const int i = min(i0 + q * kFewThreads, nr * octets - 1), r = i / octets, o = min(i % octets, a.k / 8 - 1);
                const int64_t src = DOWN ? rows[r] : rows[r] / a.top_k;
                h[q] = *reinterpret_cast<const u32x4h*>(a.x + src * a.k + 8 * o);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = i0 + q * kFewThreads, r = i / octets, o = i % octets;
                if (i < nr * octets)  // whole groups of lanes
                    stage_octet<BITS, GSHIFT, F16, kTileRows>(h[q], 8 * o < a.k, o, xl + (size_t)r * pitch, xs + r);
            }
        }
        __syncthreads();
        const uint8_t* xa = xl + (size_t)min(r16, a.rows - 1) * pitch + 2 * x_lane_offset<GSHIFT>(g);
        f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
        auto finish = [&](int turn) {  // the tile's sums are complete
            if (a.ksplit > 1) {        // over its waves, in order
#pragma unroll
                for (int m = 0; m < 2; ++m) *reinterpret_cast<f32x4*>(red + ((wave * 2 + m) * 64 + lane) * 4) = acc[m];
                __syncthreads();
                if (ks == 0)
#pragma unroll 1
                    for (int w = 1; w < a.ksplit; ++w)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
                            acc[m] += *reinterpret_cast<const f32x4*>(red + (((wave + w) * 2 + m) * 64 + lane) * 4);
                __syncthreads();  // red is written again
            }
            if (ks == 0) {
                const int n0 = (t0 + turn * step) * kTileN + r16;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int r = 4 * g + v;
                    if (r >= nr) continue;
                    const int64_t p = rows[r];
                    if constexpr (DOWN) {
                        const float w = weight_of[r];
                        float* d = static_cast<float*>(a.out) + p * a.n;
                        if (n0 < a.n) d[n0] = w * acc[0][v];
                        if (n0 + 16 < a.n) d[n0 + 16] = w * acc[1][v];
                    } else if (n0 < a.n) {
                        static_cast<uint16_t*>(a.out)[p * a.n + n0] =
                            f32_to_half_bits<F16>(silu_f32(acc[0][v]) * acc[1][v]);
                    }
                }
            }
            acc[0] = acc[1] = f32x4{0.f, 0.f, 0.f, 0.f};
        };
        auto take = [&](const Unit (&L)[2], int turn, int i) {
            const int u = u0 + i;
            if (u < units) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    unit_product<BITS, GSHIFT, F16>(L[m], xa + (size_t)u * (256 * kUnit<BITS>),
                                                    xs + u * Unit::kGroups * kTileRows + 4 * g,
                                                    (kb >> GSHIFT) - u * Unit::kGroups, cc, acc[m]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (i == each - 1) finish(turn);
        };
        const int items = turns * each;
        pipeline(items, each, A, B, load, take);
        __syncthreads();  // rows and x are written again
    }
}

// ---- few pairs --------------------------------------------------------------------------------------
//
// Where the pairs are few beside the experts, hardly any two name the same one: each pair works alone, without a
// search for the rows of its expert, and the waves of a workgroup take the pairs of a token in the second product, so
// that their sum needs no launch of its own. What counts is how many loads depend on each other: the pair's expert, then
// its weights and x together.

// One row of k values as operands: in LDS at xl (all 16 operand rows read it), its groups' sums at xs.
template <int BITS, int GSHIFT, bool F16>
__device__ __forceinline__ void stage_row(const uint16_t* x, int k, int kpad, uint8_t* xl, float* xs, int from, int by) {
    for (int o0 = from; o0 < kpad / 8; o0 += 2 * by) {
        u32x4h h[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) h[q] = *reinterpret_cast<const u32x4h*>(x + 8 * min(o0 + q * by, k / 8 - 1));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int o = o0 + q * by;
            if (o < kpad / 8) stage_octet<BITS, GSHIFT, F16, 1>(h[q], 8 * o < k, o, xl, xs);
        }
    }
}

// h of pair blockIdx.y, 16 columns a workgroup, whose waves share K.
template <int BITS, int GSHIFT, bool F16>
__global__ __launch_bounds__(kFewThreads, kFewBlocks) void moe_pair_kernel(FewArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    __shared__ f32x2 red[kFewWaves][16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t p = blockIdx.y;
    const int e = __builtin_amdgcn_readfirstlane(a.chosen[p]);
    if ((uint32_t)e >= (uint32_t)a.experts) return;
    uint8_t* xl = smem;
    float* xs = reinterpret_cast<float*>(smem + 2 * a.kpad);
    const int kb = a.k / 32, units = a.kpad / (128 * kUnit<BITS>), each = (units + kFewWaves - 1) / kFewWaves;
    const int u0 = wave * each;
    typedef UnitLoads<BITS, GSHIFT> Unit;
    const int n0 = blockIdx.x * 16 + r16, row = min(n0, a.n - 1);
    const ExpertRows w0 = expert_rows<BITS, GSHIFT>(a.w0, e, a.experts, a.n, kb);
    const ExpertRows w1 = expert_rows<BITS, GSHIFT>(a.w1, e, a.experts, a.n, kb);
    auto load = [&](Unit (&L)[2], int, int i) {
        const int u = min(u0 + i, units - 1);
        load_unit(L[0], w0, row, u, g);
        load_unit(L[1], w1, row, u, g);
    };
    Unit A[2], B[2];
    const CodeConsts cc = make_code_consts<F16>();
    load(A, 0, 0);
    if (each > 1) load(B, 0, 1);
    stage_row<BITS, GSHIFT, F16>(a.x + p / a.top_k * a.k, a.k, a.kpad, xl, xs, tid, kFewThreads);
    __syncthreads();
    f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
    const uint8_t* xa = xl + 2 * x_lane_offset<GSHIFT>(g);
    pipeline(each, each, A, B, load, [&](const Unit (&L)[2], int, int i) {
        const int u = u0 + i;
        if (u >= units) return;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            unit_product<BITS, GSHIFT, F16, 1>(L[m], xa + (size_t)u * (256 * kUnit<BITS>), xs + u * Unit::kGroups,
                                               (kb >> GSHIFT) - u * Unit::kGroups, cc, acc[m]);
            __builtin_amdgcn_sched_barrier(0);
        }
    });
    if (g == 0) red[wave][r16] = f32x2{acc[0][0], acc[1][0]};  // all result rows are the same
    __syncthreads();
    if (tid < 16 && n0 < a.n) {
        f32x2 sum = red[0][tid];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) sum += red[w][tid];
        static_cast<uint16_t*>(a.out)[p * a.n + n0] = f32_to_half_bits<F16>(silu_f32(sum.x) * sum.y);
    }
}

constexpr int kPairWaves = 16;

// y of token blockIdx.y, 16 columns a workgroup: pairs of waves take the token's pairs in turn, each wave half of K.
template <int BITS, int GSHIFT, bool F16>
__global__ __launch_bounds__(64 * kPairWaves) void moe_pair_down_kernel(FewArgs a, const uint16_t* resid) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t t = blockIdx.y;
    const int kb = a.k / 32, units = a.kpad / (128 * kUnit<BITS>), each = (units + 1) / 2;
    const int region = 2 * a.kpad + (a.kpad >> (5 + GSHIFT)) * 4;
    uint8_t* xl = smem + (wave >> 1) * region;  // h of the pair, staged by both of its waves
    float* xs = reinterpret_cast<float*>(xl + 2 * a.kpad);
    float* red = reinterpret_cast<float*>(smem + kPairWaves / 2 * region);  // [top_k][2][16]
    typedef UnitLoads<BITS, GSHIFT> Unit;
    const int n0 = blockIdx.x * 16 + r16;
    const CodeConsts cc = make_code_consts<F16>();
    const int rounds = (a.top_k + kPairWaves / 2 - 1) / (kPairWaves / 2);
    for (int q = 0; q < rounds; ++q) {
        const int j = q * (kPairWaves / 2) + (wave >> 1);
        const int64_t p = t * a.top_k + min(j, a.top_k - 1);
        const int e = __builtin_amdgcn_readfirstlane(a.chosen[p]);
        const bool there = j < a.top_k && (uint32_t)e < (uint32_t)a.experts;
        const ExpertRows w0 = expert_rows<BITS, GSHIFT>(a.w0, there ? e : 0, a.experts, a.n, kb);
        const int u0 = (wave & 1) * each, mine = there ? min(each, units - u0) : 0;
        auto load = [&](Unit& L, int, int i) { load_unit(L, w0, min(n0, a.n - 1), min(u0 + i, units - 1), g); };
        Unit A, B;
        if (mine > 0) load(A, 0, 0);
        if (mine > 1) load(B, 0, 1);
        if (there) stage_row<BITS, GSHIFT, F16>(a.x + p * a.k, a.k, a.kpad, xl, xs, (wave & 1) * 64 + lane, 128);
        __syncthreads();
        if (mine > 0) {
            f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
            const uint8_t* xa = xl + 2 * x_lane_offset<GSHIFT>(g);
            pipeline(mine, mine, A, B, load, [&](const Unit& L, int, int i) {
                const int u = u0 + i;
                unit_product<BITS, GSHIFT, F16, 1>(L, xa + (size_t)u * (256 * kUnit<BITS>), xs + u * Unit::kGroups,
                                                   (kb >> GSHIFT) - u * Unit::kGroups, cc, acc);
            });
            if (g == 0) red[(j * 2 + (wave & 1)) * 16 + r16] = acc[0];  // all result rows are the same
        } else if (there && g == 0) {
            red[(j * 2 + (wave & 1)) * 16 + r16] = 0.f;
        }
        __syncthreads();  // red is there; h is staged again
    }
    const int col = blockIdx.x * 16 + tid;
    if (tid < 16 && col < a.n) {
        const int64_t at = t * a.n + col;
        float sum = resid ? half_to_f32<F16>(resid[at]) : 0.f;
        for (int j = 0; j < a.top_k; ++j) {
            const int64_t p = t * a.top_k + j;
            if ((uint32_t)a.chosen[p] < (uint32_t)a.experts)
                sum = __builtin_fmaf(a.weights[p], red[j * 32 + tid] + red[j * 32 + 16 + tid], sum);
        }
        static_cast<uint16_t*>(a.out)[at] = f32_to_half_bits<F16>(sum);
    }
}

// y[t] = resid[t] + sum_j d[t, j] over the pairs whose expert is here, eight columns a thread.
template <bool F16>
__global__ __launch_bounds__(256) void moe_combine_kernel(const float* d, const int32_t* chosen, const uint16_t* resid,
                                                          uint16_t* y, int64_t tokens, int width, int top_k, int experts) {
    const int cols = width / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= tokens * cols) return;
    const int64_t t = i / cols;
    const int64_t at = t * width + (i % cols) * 8;
    float sum[8];
    if (resid) {
        const u32x4h r = *reinterpret_cast<const u32x4h*>(resid + at);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            sum[2 * q] = half_to_f32<F16>(r[q]);
            sum[2 * q + 1] = half_to_f32<F16>(r[q] >> 16);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[q] = 0.f;
    }
    for (int j = 0; j < top_k; ++j) {
        const int64_t p = t * top_k + j;
        if ((uint32_t)chosen[p] >= (uint32_t)experts) continue;
        const f32x4* src = reinterpret_cast<const f32x4*>(d + p * width + (i % cols) * 8);
        const f32x4 lo = src[0], hi = src[1];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            sum[q] += lo[q];
            sum[4 + q] += hi[q];
        }
    }
    u32x4h o;
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = pack_half2<F16>(sum[2 * q], sum[2 * q + 1]);
    *reinterpret_cast<u32x4h*>(y + at) = o;
}

// ---- launches ---------------------------------------------------------------------------------------

inline int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

template <int BITS, int GSHIFT, bool F16, bool DOWN>
hipError_t launch_few_kernel(FewArgs a, hipStream_t stream) {
    a.kpad = (int)round_up(a.k, 128 * kUnit<BITS>);
    const int pitch = 2 * a.kpad + 16;
    const int sums = (a.kpad >> (5 + GSHIFT)) * kTileRows * 4;
    constexpr int kRed = kFewWaves * 2 * 64 * 16;
    // Rows of x a pass: 8 up to an average of 2 rows an expert, 16 above (a smaller x lets more workgroups share a compute
    // unit, 16 rows of 2048 values two, 8 rows three; but an expert of more rows is read twice: 64 tokens through 8 of
    // 128 experts, 4 rows on average, take 110 us with 8 rows a pass and 95 with 16).
    const int64_t used = std::min(a.pairs, (int64_t)a.experts);
    a.rows = (int)std::min(a.pairs, a.pairs <= 2 * used ? (int64_t)8 : (int64_t)kTileRows);
    while (a.rows > 1 && a.rows * pitch + sums + kRed > 150 * 1024) a.rows = (a.rows + 1) / 2;
    const int lds = a.rows * pitch + sums + kRed;
    const int tiles = (a.n + (DOWN ? 31 : 15)) / (DOWN ? 32 : 16);
    const int64_t slots = used;  // experts that have work, at most
    // Waves that share a tile: as many as it takes to give all of them work. Workgroups of
    // an expert: as many as run at once, each over several tiles, so that x is loaded few times.
    const int64_t room = (int64_t)device_cu_count() * std::min((int64_t)kFewBlocks, (int64_t)(160 * 1024 / (lds + 512)));
    a.ksplit = 1;
    while (a.ksplit < kFewWaves && slots * tiles * a.ksplit < room * kFewWaves) a.ksplit *= 2;
    const int side = kFewWaves / a.ksplit;
    const int64_t most = (tiles + side - 1) / side;
    const int64_t gx = std::max((int64_t)1, std::min(most, room / slots));
    moe_few_kernel<BITS, GSHIFT, F16, DOWN><<<dim3((unsigned)gx, (unsigned)a.experts), dim3(kFewThreads), lds, stream>>>(a);
    return hipGetLastError();
}

template <bool F16>
hipError_t launch_combine(const MoeArgs& a, const float* d, hipStream_t stream) {
    const int64_t threads = a.tokens * (a.width / 8);
    moe_combine_kernel<F16><<<dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream>>>(
        d, a.chosen, a.resid, a.y, a.tokens, a.width, d ? a.top_k : 0, a.experts);
    return hipGetLastError();
}

// Whether each pair works alone: the pairs are no more than the experts, and their rows fit LDS. 4-bit 128 x [768, 2048],
// 8 experts a token: 8 tokens (64 pairs) take 46 us so and 79 with rows gathered by expert, 16 tokens (128 pairs) 85
// against 87.
inline bool pair_path(const MoeArgs& a) {
    return a.tokens * a.top_k <= a.experts && a.hidden <= 4096 && a.top_k <= 64;
}

template <int BITS, int GSHIFT, bool F16>
hipError_t launch_pairs(const MoeArgs& a, FewArgs f, hipStream_t stream) {
    f.kpad = (int)round_up(f.k, 128 * kUnit<BITS>);
    moe_pair_kernel<BITS, GSHIFT, F16><<<dim3((unsigned)((f.n + 15) / 16), (unsigned)f.pairs), dim3(kFewThreads),
                                         2 * f.kpad + (f.kpad >> (5 + GSHIFT)) * 4, stream>>>(f);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    f.x = static_cast<const uint16_t*>(f.out);
    f.w0 = a.down;
    f.out = a.y;
    f.k = a.hidden;
    f.n = a.width;
    f.kpad = (int)round_up(f.k, 128 * kUnit<BITS>);
    const int lds = kPairWaves / 2 * (2 * f.kpad + (f.kpad >> (5 + GSHIFT)) * 4) + a.top_k * 32 * 4;
    moe_pair_down_kernel<BITS, GSHIFT, F16><<<dim3((unsigned)((f.n + 15) / 16), (unsigned)a.tokens), dim3(64 * kPairWaves),
                                              lds, stream>>>(f, a.resid);
    return hipGetLastError();
}

template <int BITS, int GSHIFT, bool F16>
hipError_t launch_few(const MoeArgs& a, hipStream_t stream) {
    const int64_t pairs = a.tokens * a.top_k;
    uint16_t* h = static_cast<uint16_t*>(a.workspace);
    float* d = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + round_up(pairs * a.hidden * 2, 256));
    FewArgs f{};
    f.chosen = a.chosen;
    f.weights = a.weights;
    f.pairs = pairs;
    f.top_k = a.top_k;
    f.experts = a.experts;
    f.x = a.x;
    f.w0 = a.gate;
    f.w1 = a.up;
    f.out = h;
    f.k = a.width;
    f.n = a.hidden;
    if (pair_path(a)) return launch_pairs<BITS, GSHIFT, F16>(a, f, stream);
    hipError_t e = launch_few_kernel<BITS, GSHIFT, F16, false>(f, stream);
    if (e != hipSuccess) return e;
    f.x = h;
    f.w0 = f.w1 = a.down;
    f.out = d;
    f.k = a.hidden;
    f.n = a.width;
    e = launch_few_kernel<BITS, GSHIFT, F16, true>(f, stream);
    if (e != hipSuccess) return e;
    return launch_combine<F16>(a, d, stream);
}

template <int BITS, bool F16>
hipError_t launch_few_bits(const MoeArgs& a, hipStream_t stream) {
    if (a.group == 32) return launch_few<BITS, 0, F16>(a, stream);
    if (a.group == 64) return launch_few<BITS, 1, F16>(a, stream);
    return launch_few<BITS, 2, F16>(a, stream);
}

template <bool F16>
hipError_t launch_few_any(const MoeArgs& a, hipStream_t stream) {
    switch (a.bits) {
        case 1: return launch_few_bits<1, F16>(a, stream);
        case 2: return launch_few_bits<2, F16>(a, stream);
        case 3: return launch_few_bits<3, F16>(a, stream);
        case 4: return launch_few_bits<4, F16>(a, stream);
        case 5: return launch_few_bits<5, F16>(a, stream);
        case 6: return launch_few_bits<6, F16>(a, stream);
        case 8: return launch_few_bits<8, F16>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace
}  // namespace qaff
