// ep_wave.h -- sums and maxima over a wave by lane-to-lane moves inside the
// vector unit (DPP), without a trip through LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_device.h"

namespace ep {

// Workgroups of a launch with one row or token to a wave or workgroup; longer batches
// take more launches (a grid has fewer than 2^32 threads).
constexpr int64_t kLaunchGroups = 1 << 21;

// v of the lane that CTRL names in this row of 16 lanes.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
constexpr int kDppSwap1 = 0xB1;   // quad_perm 1 0 3 2
constexpr int kDppSwap2 = 0x4E;   // quad_perm 2 3 0 1
constexpr int kDppMirror8 = 0x141;
constexpr int kDppMirror16 = 0x140;

__device__ __forceinline__ double readlane_f(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sum, largest value over each row of 16 lanes, in every lane of the row.
template <class V>
__device__ __forceinline__ V row_sum(V v) {
    v += dpp<kDppSwap1>(v);
    v += dpp<kDppSwap2>(v);
    v += dpp<kDppMirror8>(v);
    v += dpp<kDppMirror16>(v);
    return v;
}
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, dpp<kDppSwap1>(v));
    v = fmaxf(v, dpp<kDppSwap2>(v));
    v = fmaxf(v, dpp<kDppMirror8>(v));
    v = fmaxf(v, dpp<kDppMirror16>(v));
    return v;
}
// The same over the wave's 64 lanes.
template <class V>
__device__ __forceinline__ V wave_sum(V v) {
    v = row_sum(v);
    return (readlane_f(v, 0) + readlane_f(v, 16)) + (readlane_f(v, 32) + readlane_f(v, 48));
}
__device__ __forceinline__ float wave_max(float v) {
    v = row_max(v);
    return fmaxf(fmaxf(readlane_f(v, 0), readlane_f(v, 16)), fmaxf(readlane_f(v, 32), readlane_f(v, 48)));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
// In a scalar register.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, dpp<kDppSwap1>(v));
    v = max(v, dpp<kDppSwap2>(v));
    v = max(v, dpp<kDppMirror8>(v));
    v = max(v, dpp<kDppMirror16>(v));
    return max(max((uint32_t)readlane((int)v, 0), (uint32_t)readlane((int)v, 16)),
               max((uint32_t)readlane((int)v, 32), (uint32_t)readlane((int)v, 48)));
}

}  // namespace ep
