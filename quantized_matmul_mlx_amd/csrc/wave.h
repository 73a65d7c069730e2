// Sums over a wave's 64 lanes in registers (DPP), without LDS round trips, and a stream of loads that stays ahead of
// their use.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qaff {

// v of the lane that the DPP control names, 0 where that lane is not there.
template <int CTRL, int ROWS> __device__ __forceinline__ int dpp(int v) {
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS> __device__ __forceinline__ int64_t dpp(int64_t v) {
    const uint32_t lo = (uint32_t)dpp<CTRL, ROWS>((int)(uint32_t)v);
    return (int64_t)((uint64_t)(uint32_t)dpp<CTRL, ROWS>((int)(v >> 32)) << 32 | lo);
}

// Inclusive sums over the wave's lanes: within rows of 16 lanes (row_shr 1, 2, 4, 8), then the last
// lane of a row to the next rows (row_bcast 15 and 31).
template <typename T> __device__ __forceinline__ T wave_scan(T v) {
    v += dpp<0x111, 0xf>(v);
    v += dpp<0x112, 0xf>(v);
    v += dpp<0x114, 0xf>(v);
    v += dpp<0x118, 0xf>(v);
    v += dpp<0x142, 0xa>(v);
    v += dpp<0x143, 0xc>(v);
    return v;
}

// Lane `lane`'s value (the same lane for the whole wave), in a scalar register.
__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// Walks items (turn, i), 0 <= i < each, in order, with the next two in the registers A and B (which hold the first two
// at the start). The loads in the loop have no conditions: the compiler counts those on their way to wait for the ones
// it needs, and with a branch around some would wait for all. So the last one may repeat an item that is there.
template <typename Units, typename Load, typename Take>
__device__ __forceinline__ void pipeline(int items, int each, Units& A, Units& B, Load load, Take take) {
    int t0 = 0, i0 = 0, t1 = 0, i1 = 0;  // the items in A and B
    auto advance = [&](int& t, int& i) {
        if (++i >= each) {
            i = 0;
            ++t;
        }
    };
    advance(t1, i1);
    int n = 0;
    for (; n + 2 < items; n += 2) {
        int t = t1, i = i1;
        advance(t, i);
        take(A, t0, i0);
        load(A, t, i);
        t0 = t;
        i0 = i;
        if (n + 3 < items) advance(t, i);
        take(B, t1, i1);
        load(B, t, i);
        t1 = t;
        i1 = i;
    }
    take(A, t0, i0);
    if (n + 1 < items) take(B, t1, i1);
}

}  // namespace qaff
