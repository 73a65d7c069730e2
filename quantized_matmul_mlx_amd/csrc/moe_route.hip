// The router of a mixture of experts: for each token the top_k experts of the largest keys (ties to
// the lowest index) and their weights.
//
//   key[e] = logit[e], or score[e] + bias[e] with a bias; score = softmax(logits) or 1 / (1 + exp(-logit))
//   weight = score of the chosen expert (over the sum of the chosen ones' scores), times a factor
//
// Both scores grow with the logit, so without a bias the choice needs no score and is exact. With one,
// the scores are float64: two sums that differ in the seventh digit still come in their order.
//
// A token takes 2^n lanes (16 lanes of 8 logits for 128 experts, a wave at most), so that a step of
// the search for the largest key serves several tokens: in each lane over its own logits, then over the
// lanes. The chosen key is struck out and the search repeats, top_k times. Bound by that chain of exchanges:
// 16384 tokens of 128 experts, 8 chosen, take 8.7 us (kernel alone; 9.4 MB, 1.1 TB/s), 64 tokens 6.6.
#include "ffn.h"
#include "qaff_device.h"

namespace qaff {
namespace {

// Lanes that hold one token's logits: lane i of the group has experts i, i + LANES, ... The exchanges below stay in
// registers: a read from another lane through LDS takes as long as the rest of a round.
template <int CTRL, typename T> __device__ __forceinline__ T from_lane(T v) {
    if constexpr (sizeof(T) == 8) {
        const int64_t b = __builtin_bit_cast(int64_t, v);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xf, 0xf, false);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, 0xf, 0xf, false);
        return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
    } else {
        return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
    }
}
// The value 16 (32) lanes on or before.
template <bool WIDE> __device__ __forceinline__ uint32_t other_half(uint32_t v) {
    const bool upper = threadIdx.x & (WIDE ? 32 : 16);
    const auto r = WIDE ? __builtin_amdgcn_permlane32_swap(v, v, false, false) : __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return upper ? r[0] : r[1];
}
template <bool WIDE, typename T> __device__ __forceinline__ T from_half(T v) {
    if constexpr (sizeof(T) == 8) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        return __builtin_bit_cast(T, (uint64_t)other_half<WIDE>((uint32_t)(b >> 32)) << 32 | other_half<WIDE>((uint32_t)b));
    } else {
        return __builtin_bit_cast(T, other_half<WIDE>(__builtin_bit_cast(uint32_t, v)));
    }
}
template <int LANES, typename T, typename Op>
__device__ __forceinline__ T group_reduce(T v, Op op) {
    static_assert(LANES >= 16, "a row of 16 lanes at least");
    v = op(v, from_lane<0xB1>(v));   // lane ^ 1
    v = op(v, from_lane<0x4E>(v));   // lane ^ 2
    v = op(v, from_lane<0x141>(v));  // mirrored in 8 lanes
    v = op(v, from_lane<0x140>(v));  // and in 16
    if constexpr (LANES >= 32) v = op(v, from_half<false>(v));
    if constexpr (LANES >= 64) v = op(v, from_half<true>(v));
    return v;
}
template <int LANES, typename T> __device__ __forceinline__ T group_max(T v) {
    return group_reduce<LANES>(v, [](T a, T b) { return b > a ? b : a; });
}
template <int LANES> __device__ __forceinline__ int group_min(int v) {
    return group_reduce<LANES>(v, [](int a, int b) { return min(a, b); });
}
template <int LANES, typename T> __device__ __forceinline__ T group_sum(T v) {
    return group_reduce<LANES>(v, [](T a, T b) { return a + b; });
}

template <typename K> struct Math;
template <> struct Math<float> {
    static __device__ __forceinline__ float exp(float v) { return ::expf(v); }
};
template <> struct Math<double> {
    static __device__ __forceinline__ double exp(double v) { return ::exp(v); }
};

// K: the type of keys and scores (double where a bias takes part in the choice).
template <int LANES, int EACH, typename K>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
    constexpr int kTokens = 256 / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t token = (int64_t)blockIdx.x * kTokens + threadIdx.x / LANES;
    // a group past the last token repeats it: all lanes stay in the exchanges below
    const int64_t t = token < a.tokens ? token : a.tokens - 1;
    const K none = -__builtin_inf();
    K x[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int e = lane + i * LANES;
        x[i] = e < a.experts ? (K)load_as_f32(a.logits, (size_t)(t * a.row_stride + e), a.dtype) : none;
        if (!(x[i] == x[i])) x[i] = none;  // a NaN is never better than a number
    }
    // softmax: the largest logit and the sum of exp(logit - largest); no expert left: sum 0
    K top = none, sum = 0;
    const bool softmax = !a.sigmoid;
    if (softmax) {
#pragma unroll
        for (int i = 0; i < EACH; ++i) top = x[i] > top ? x[i] : top;
        top = group_max<LANES>(top);
    }
    auto score = [&](K v) -> K {  // softmax: before the division by the sum
        if (v == none) return 0;
        if (a.sigmoid) return 1 / (1 + Math<K>::exp(-v));
        return v == top ? (K)1 : Math<K>::exp(v - top);
    };
    if (softmax && (a.bias || !a.renormalize)) {
#pragma unroll
        for (int i = 0; i < EACH; ++i) sum += score(x[i]);
        sum = group_sum<LANES>(sum);
    }
    K key[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        key[i] = x[i];
        const int e = lane + i * LANES;
        if (a.bias && x[i] != none) {
            const K s = score(x[i]);
            const K k = (softmax ? s / sum : s) + (K)a.bias[e];
            key[i] = k == k ? k : none;
        }
    }
    // top_k rounds; lane r of the group keeps the r-th chosen expert (r, r + LANES, ... where top_k is larger)
    constexpr int kKeep = (kRouteMaxChosen + LANES - 1) / LANES;
    int mine[kKeep];
    K mine_x[kKeep];
    uint32_t taken = 0;  // bit i: this lane's logit i is chosen already
    K total = 0;
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        mine[j] = 0;
        mine_x[j] = none;
        for (int r = 0; r < LANES && j * LANES + r < a.top_k; ++r) {
            K best = none;
            int at = 1 << 30;
            K at_x = none;
#pragma unroll
            for (int i = EACH - 1; i >= 0; --i) {  // from the back: of equal keys the lowest index stays
                const int e = lane + i * LANES;
                if (!(taken >> i & 1) && e < a.experts && key[i] >= best) {
                    best = key[i];
                    at = e;
                    at_x = x[i];
                }
            }
            const K most = group_max<LANES>(best);
            const int who = group_min<LANES>(best == most ? at : 1 << 30);
            if (who == at) taken |= 1u << (at / LANES);
            if (a.bias) at_x = __shfl(at_x, who % LANES, LANES);
            else at_x = most;  // the key is the logit
            if (lane == r) {
                mine[j] = who;
                mine_x[j] = at_x;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        mine_x[j] = j * LANES + lane < a.top_k ? score(mine_x[j]) : (K)0;
        total += mine_x[j];
    }
    total = a.renormalize ? group_sum<LANES>(total) : softmax ? sum : (K)1;
    if (token >= a.tokens) return;
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
        const int r = j * LANES + lane;
        if (r >= a.top_k) continue;
        const K w = total > 0 ? mine_x[j] / total : (K)0;
        a.chosen[token * a.top_k + r] = mine[j];
        a.weights[token * a.top_k + r] = (float)(w * (K)a.scale);
    }
}

template <int LANES, int EACH>
hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
    constexpr int kTokens = 256 / LANES;
    const unsigned blocks = (unsigned)((a.tokens + kTokens - 1) / kTokens);
    if (a.bias) route_kernel<LANES, EACH, double><<<dim3(blocks), dim3(256), 0, stream>>>(a);
    else route_kernel<LANES, EACH, float><<<dim3(blocks), dim3(256), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream) {
    if (a.experts <= 64) return launch_route<16, 4>(a, stream);
    if (a.experts <= 128) return launch_route<16, 8>(a, stream);
    if (a.experts <= 256) return launch_route<32, 8>(a, stream);
    if (a.experts <= 512) return launch_route<64, 8>(a, stream);
    return launch_route<64, 16>(a, stream);
}

}  // namespace qaff
