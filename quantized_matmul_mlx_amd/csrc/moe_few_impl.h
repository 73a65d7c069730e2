// The layer of a mixture of experts for few rows an expert: products of gathered rows with each
// expert's weights, read once for up to 16 rows.
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
//  * v_mfma_f32_16x16x32: a lane loads a whole block of 32 codes (16 bytes at 4 bits) of weight row
//    lane % 16, block lane / 16 of a chunk of 128. A product may only cover one group, so for groups of
//    64 and 32 the lanes exchange halves and quarters of their blocks (v_permlane32_swap, v_permlane16_swap)
//    and read x in the order that results.
#pragma once

#include "ffn.h"
#include "mfma16.h"
#include "wave.h"

#include <hip/hip_runtime.h>

namespace qaff {
namespace {

typedef uint32_t u32x4h __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2h __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32h __attribute__((aligned(2)));

constexpr int kTileRows = 16;  // rows of x a pass
constexpr int kUnit = 2;       // chunks of 128 codes that are loaded together
constexpr int kFewWaves = 4;

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
    int by_pair;                 // grid y walks pairs (the first of each expert works) instead of experts
};

// ---- codes as operands ----------------------------------------------------------------------------

// B of the exact operands: 128 + c has 8 bits for codes of up to 6 bits; 8-bit codes are bf16 values
// themselves. float16 holds 1024 + c.
template <bool F16, int BITS> constexpr float kCodeBase = F16 ? 1024.f : BITS == 8 ? 0.f : 128.f;

template <bool F16, int BITS>
__device__ __forceinline__ u32x4a code_operand(const uint32_t (&w)[BITS], int j) {
    constexpr uint32_t base = F16 ? 0x64006400u : 0x43004300u;
    u32x4a o;
    if constexpr (BITS == 4) {  // pairs (c0, c4), (c1, c5), (c2, c6), (c3, c7): x is staged in that order
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = ((w[j] >> (4 * e)) & 0x000F000Fu) | base;
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
__device__ __forceinline__ void chunk_operands(const uint32_t (&w)[BITS], op8<F16> (&o)[4]) {
    if constexpr (BITS == 4) {  // an octet is a word: exchanged before it is spread
        uint32_t v[4] = {w[0], w[1], w[2], w[3]};
        regroup<GSHIFT>(v[0], v[1], v[2], v[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = __builtin_bit_cast(op8<F16>, code_operand<F16, 4>(v, j));
    } else {
        u32x4a v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = code_operand<F16, BITS>(w, j);
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

// A unit's codes, scales and biases of one weight row: kUnit blocks of this lane, and the unit's groups.
template <int BITS, int GSHIFT> struct UnitLoads {
    static constexpr int kGroups = kUnit * 4 >> GSHIFT;
    static constexpr int kWords = (kGroups + 1) / 2;
    uint32_t w[kUnit][BITS];
    uint32_t s[kWords], b[kWords];
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

// Unit u of weight row `row` (counted over all experts). Blocks past the row's end repeat its last one:
// x is 0 there. Groups likewise.
template <int BITS, int GSHIFT>
__device__ __forceinline__ void load_unit(UnitLoads<BITS, GSHIFT>& L, const ExpertWeight& W, int64_t row, int u, int kb,
                                          int g) {
    typedef UnitLoads<BITS, GSHIFT> U;
    const int gpr = kb >> GSHIFT;
    const uint16_t* sp = W.scales + row * gpr;
    const uint16_t* bp = W.biases + row * gpr;
    if ((u + 1) * (4 * kUnit) <= kb) {
        load_halves(sp + u * U::kGroups, L.s);
        load_halves(bp + u * U::kGroups, L.b);
    } else {
#pragma unroll
        for (int i = 0; i < U::kWords; ++i) {
            const int g0 = min(u * U::kGroups + 2 * i, gpr - 1), g1 = min(u * U::kGroups + 2 * i + 1, gpr - 1);
            L.s[i] = (uint32_t)sp[g0] | (uint32_t)sp[g1] << 16;
            L.b[i] = (uint32_t)bp[g0] | (uint32_t)bp[g1] << 16;
        }
    }
    const uint32_t* pw = W.packed + row * kb * BITS;
#pragma unroll
    for (int c = 0; c < kUnit; ++c) load_block<BITS>(pw + min(4 * (u * kUnit + c) + g, kb - 1) * BITS, L.w[c]);
}

// ---- products ---------------------------------------------------------------------------------------

// acc[m] += x . (unit of weight m)^T for both weights. xa: the lane's row of x in LDS at the unit's first
// code, xs: the sums of x of the unit's groups ([group][16 rows], at the lane's four result rows).
template <int BITS, int GSHIFT, bool F16>
__device__ __forceinline__ void unit_product(const UnitLoads<BITS, GSHIFT> (&L)[2], const uint8_t* xa, const float* xs,
                                             f32x4 (&acc)[2]) {
    constexpr int kEach = 1 << GSHIFT;  // products a group
#pragma unroll
    for (int c = 0; c < kUnit; ++c) {
        op8<F16> o[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) chunk_operands<F16, BITS, GSHIFT>(L[m].w[c], o[m]);
#pragma unroll
        for (int p = 0; p < (4 >> GSHIFT); ++p) {
            f32x4 d[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int step = p * kEach + i;
                const op8<F16> a = *reinterpret_cast<const op8<F16>*>(xa + 256 * c + 2 * x_step_offset<GSHIFT>(step));
#pragma unroll
                for (int m = 0; m < 2; ++m) d[m] = mfma16x16x32<F16>(a, o[m][step], d[m]);
            }
            const int grp = (4 * c >> GSHIFT) + p;
            const f32x4 sum = *reinterpret_cast<const f32x4*>(xs + grp * kTileRows);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float s = half_to_f32<F16>(L[m].s[grp >> 1] >> (16 * (grp & 1)));
                const float b = half_to_f32<F16>(L[m].b[grp >> 1] >> (16 * (grp & 1)));
                const float beta = __builtin_fmaf(-kCodeBase<F16, BITS>, s, b);
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[m][v] = __builtin_fmaf(s, d[m][v], __builtin_fmaf(beta, sum[v], acc[m][v]));
            }
        }
    }
}

// Pairs of the expert e whose rank lies in [first, first + count) into rows[0 ..), by one wave; returns
// the expert's pairs up to that point or more.
__device__ __forceinline__ int list_rows(const int32_t* chosen, int64_t pairs, int e, int first, int count, int lane,
                                         int* rows) {
    int rank = 0;
    for (int64_t base = 0; base < pairs && rank <= first + count; base += 256) {
        bool mine[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t p = base + 64 * i + lane;
            mine[i] = p < pairs && chosen[p < pairs ? p : 0] == e;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t hits = __builtin_amdgcn_ballot_w64(mine[i]);
            const int at = rank + __builtin_popcountll(hits & ((1ull << lane) - 1)) - first;
            if (mine[i] && at >= 0 && at < count) rows[at] = (int)(base + 64 * i + lane);
            rank += __builtin_popcountll(hits);
        }
    }
    return rank;
}

// DOWN = false: gate and up, h out (16-bit). DOWN = true: two neighbouring tiles of the down weight, rows
// of d out (float32, times the pair's weight).
template <int BITS, int GSHIFT, bool F16, bool DOWN>
__global__ __launch_bounds__(64 * kFewWaves) void moe_few_kernel(FewArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    __shared__ int rows[kTileRows];
    __shared__ int found;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    constexpr int kOct = 4 << GSHIFT;  // octets of x a group
    int e = blockIdx.y;
    if (a.by_pair) {
        e = a.chosen[blockIdx.y];
        if ((uint32_t)e >= (uint32_t)a.experts) return;
        bool before = false;  // the first pair of an expert works for all of them
        for (int base = 0; base < (int)blockIdx.y; base += 64)
            before |= base + lane < (int)blockIdx.y && a.chosen[min(base + lane, (int)blockIdx.y)] == e;
        if (__builtin_amdgcn_ballot_w64(before)) return;
    }
    const int pitch = 2 * a.kpad + 16;  // 16 rows at one offset fall on distinct banks
    uint8_t* xl = smem;
    float* xs = reinterpret_cast<float*>(smem + (size_t)a.rows * pitch);
    float* red = xs + (a.kpad >> (5 + GSHIFT)) * kTileRows;
    const int kb = a.k / 32, octets = a.kpad / 8;
    const int tile_n = DOWN ? 32 : 16;
    const int tiles = (a.n + tile_n - 1) / tile_n;
    const int side = kFewWaves / a.ksplit;  // tiles at a time
    const int ks = wave % a.ksplit;
    const int units = a.kpad / (128 * kUnit), each = (units + a.ksplit - 1) / a.ksplit;

    for (int first = 0;; first += a.rows) {
        if (wave == 0) {
            const int n = list_rows(a.chosen, a.pairs, e, first, a.rows, lane, rows);
            if (lane == 0) found = n;
        }
        __syncthreads();
        const int total = found;
        if (first >= total) return;
        const int nr = min(a.rows, total - first);
        // x of the tile's rows, and its groups' sums
        for (int i = tid; i < nr * octets; i += 64 * kFewWaves) {
            const int r = i / octets, o = i % octets;
            const int64_t src = DOWN ? rows[r] : rows[r] / a.top_k;
            u32x4a v = u32x4a{0u, 0u, 0u, 0u};
            if (8 * o < a.k) {
                const u32x4h h = *reinterpret_cast<const u32x4h*>(a.x + src * a.k + 8 * o);
                v = u32x4a{h.x, h.y, h.z, h.w};
            }
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) sum += half_to_f32<F16>(v[q]) + half_to_f32<F16>(v[q] >> 16);
#pragma unroll
            for (int d = 1; d < kOct; d <<= 1) sum += __shfl_xor(sum, d, 64);
            if (o % kOct == 0) xs[o / kOct * kTileRows + r] = sum;
            if constexpr (BITS == 4)
                v = u32x4a{__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                           __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u)};
            *reinterpret_cast<u32x4a*>(xl + (size_t)r * pitch + 16 * o) = v;
        }
        __syncthreads();
        const uint8_t* xa = xl + (size_t)min(r16, a.rows - 1) * pitch + 2 * x_lane_offset<GSHIFT>(g);
        for (int t0 = blockIdx.x * side; t0 < tiles; t0 += gridDim.x * side) {
            const int tile = t0 + wave / a.ksplit;
            f32x4 acc[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
            const int n0 = tile * tile_n + r16;
            const int64_t row0 = (int64_t)e * a.n + min(n0, a.n - 1);
            const int64_t row1 = DOWN ? (int64_t)e * a.n + min(n0 + 16, a.n - 1) : row0;
            for (int u = ks * each; u < min(units, (ks + 1) * each); ++u) {
                UnitLoads<BITS, GSHIFT> L[2];
                load_unit(L[0], a.w0, row0, u, kb, g);
                load_unit(L[1], DOWN ? a.w0 : a.w1, row1, u, kb, g);
                unit_product<BITS, GSHIFT, F16>(L, xa + (size_t)u * (256 * kUnit),
                                                xs + u * UnitLoads<BITS, GSHIFT>::kGroups * kTileRows + 4 * g, acc);
            }
            if (a.ksplit > 1) {  // sums over the waves of the tile, in order
                __syncthreads();
#pragma unroll
                for (int m = 0; m < 2; ++m) *reinterpret_cast<f32x4*>(red + ((wave * 2 + m) * 64 + lane) * 4) = acc[m];
                __syncthreads();
                if (ks == 0)
                    for (int w = 1; w < a.ksplit; ++w)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
                            acc[m] += *reinterpret_cast<const f32x4*>(red + (((wave + w) * 2 + m) * 64 + lane) * 4);
            }
            if (ks == 0) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int r = 4 * g + v;
                    if (r >= nr) continue;
                    const int64_t p = rows[r];
                    if constexpr (DOWN) {
                        const float w = a.weights[p];
                        float* d = static_cast<float*>(a.out) + p * a.n;
                        if (n0 < a.n) d[n0] = w * acc[0][v];
                        if (n0 + 16 < a.n) d[n0 + 16] = w * acc[1][v];
                    } else if (n0 < a.n) {
                        static_cast<uint16_t*>(a.out)[p * a.n + n0] =
                            f32_to_half_bits<F16>(silu_f32(acc[0][v]) * acc[1][v]);
                    }
                }
            }
        }
        __syncthreads();  // rows, x and red are written again
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
hipError_t launch_few_kernel(FewArgs a, int64_t tokens, hipStream_t stream) {
    a.kpad = (int)round_up(a.k, 128 * kUnit);
    const int pitch = 2 * a.kpad + 16;
    const int sums = (a.kpad >> (5 + GSHIFT)) * kTileRows * 4;
    constexpr int kRed = kFewWaves * 2 * 64 * 16;
    a.rows = (int)(a.pairs < kTileRows ? a.pairs : kTileRows);
    while (a.rows > 1 && a.rows * pitch + sums + kRed > 150 * 1024) a.rows = (a.rows + 1) / 2;
    const int lds = a.rows * pitch + sums + kRed;
    const int tiles = (a.n + (DOWN ? 31 : 15)) / (DOWN ? 32 : 16);
    a.by_pair = a.pairs < a.experts;
    const int slots = (int)(a.by_pair ? a.pairs : a.experts);
    a.ksplit = kFewWaves;
    const int side = kFewWaves / a.ksplit;
    const int gx = (tiles + side - 1) / side;
    moe_few_kernel<BITS, GSHIFT, F16, DOWN><<<dim3(gx, slots), dim3(64 * kFewWaves), lds, stream>>>(a);
    return hipGetLastError();
}

template <bool F16>
hipError_t launch_combine(const MoeArgs& a, const float* d, hipStream_t stream) {
    const int64_t threads = a.tokens * (a.width / 8);
    moe_combine_kernel<F16><<<dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream>>>(
        d, a.chosen, a.resid, a.y, a.tokens, a.width, d ? a.top_k : 0, a.experts);
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
    hipError_t e = launch_few_kernel<BITS, GSHIFT, F16, false>(f, a.tokens, stream);
    if (e != hipSuccess) return e;
    f.x = h;
    f.w0 = f.w1 = a.down;
    f.out = d;
    f.k = a.hidden;
    f.n = a.width;
    e = launch_few_kernel<BITS, GSHIFT, F16, true>(f, a.tokens, stream);
    if (e != hipSuccess) return e;
    return launch_combine<F16>(a, d, stream);
}

template <int BITS, bool F16>
hipError_t launch_few_bits(const MoeArgs& a, hipStream_t stream) {
    if (a.group == 32) return launch_few<BITS, 0, F16>(a, stream);
    if (a.group == 64) return launch_few<BITS, 1, F16>(a, stream);
    return launch_few<BITS, 2, F16>(a, stream);
}

}  // namespace
}  // namespace qaff
