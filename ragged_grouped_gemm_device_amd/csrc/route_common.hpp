// Device-side pieces of the ragged layout that both routers share.
#pragma once

#include "common.hpp"

namespace moe {

// Lanes of this wavefront whose value of e (0 <= e < 2^nbits) equals ours.
__device__ __forceinline__ uint64_t match_lanes(int e, bool valid, int nbits) {
    uint64_t m = __ballot(valid);
    for (int b = 0; b < nbits; ++b) {
        const bool bit = (e >> b) & 1;
        const uint64_t bb = __ballot(bit);
        m &= bit ? bb : ~bb;
    }
    return valid ? m : 0ull;
}

// In-order ranks of the pairs [q0, q1) by one wavefront, 64 at a time: pair p
// with expert e gets row cnt[e] + (earlier lanes with the same e), and the
// group's first lane advances cnt[e] (cnt: the wavefront's own LDS row).
__device__ __forceinline__ void rank_pairs(const int32_t* __restrict__ topk_idx, int64_t q0, int64_t q1,
                                           int nbits, int32_t* cnt, int32_t* __restrict__ row_of,
                                           int32_t* __restrict__ src_of) {
    const int lane = lane_id();
    const uint64_t lt = (lane == 0) ? 0ull : (~0ull >> (64 - lane));
    for (int64_t sb = q0; sb < q1; sb += 64) {
        const int64_t p = sb + lane;
        const bool valid = p < q1;
        const int e = valid ? topk_idx[p] : 0;
        const uint64_t m = match_lanes(e, valid, nbits);
        int32_t row = 0;
        if (valid) row = cnt[e] + __popcll(m & lt);
        wave_lds_sync();
        if (valid && (m & lt) == 0ull) cnt[e] = row + __popcll(m);  // group leader advances
        wave_lds_sync();
        if (valid) {
            row_of[p] = row;
            src_of[row] = (int32_t)p;
        }
    }
}

}  // namespace moe
