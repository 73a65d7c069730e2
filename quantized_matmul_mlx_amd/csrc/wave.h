// Sums over a wave's 64 lanes in registers (DPP), without LDS round trips.
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

}  // namespace qaff
