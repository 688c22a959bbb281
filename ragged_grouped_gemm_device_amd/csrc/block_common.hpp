// Device-side helpers of the operators around a MoE block.
#pragma once

#include "block_launch.hpp"
#include "common.hpp"

namespace moe {

__device__ __forceinline__ void unpack8(uint4 w, float* v) {
    unpack_bf16x4(make_uint2(w.x, w.y), v);
    unpack_bf16x4(make_uint2(w.z, w.w), v + 4);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

// Reductions over the G = 16 or 64 neighbouring lanes of a group, the result in all of them: lane
// exchanges inside a row of 16 by DPP, then across rows.
template <int CTRL>
__device__ __forceinline__ float lane_dpp(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}
template <int G, class Op>
__device__ __forceinline__ float lanes_reduce(float v, Op op) {
    static_assert(G == 16 || G == 64, "group of lanes");
    v = op(v, lane_dpp<0xB1>(v));   // lane ^ 1
    v = op(v, lane_dpp<0x4E>(v));   // lane ^ 2
    v = op(v, lane_dpp<0x141>(v));  // the other quad of 8 lanes
    v = op(v, lane_dpp<0x140>(v));  // the other half of 16 lanes
    if constexpr (G == 64) {
        v = op(v, __shfl_xor(v, 16, 64));
        v = op(v, __shfl_xor(v, 32, 64));
    }
    return v;
}
template <int G>
__device__ __forceinline__ float lanes_max(float v) {
    return lanes_reduce<G>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
    return lanes_reduce<G>(v, [](float a, float b) { return a + b; });
}

}  // namespace moe
