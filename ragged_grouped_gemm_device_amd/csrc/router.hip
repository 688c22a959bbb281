// The router with scores, a balance bias, groups of experts and renormalised weights, and its
// gradient (gfx950).
//
//   s = sigmoid(l) or softmax(l); c = s + b (b a bias that takes part in the choice alone);
//   a group of E / G neighbouring experts is worth its best c, or the sum of its two best;
//   the k best c within the best groups, ties to the lower index; w_j = scale s_j (/ sum_i s_i).
//
// The choice is that of 64-bit arithmetic at fp32 cost: scores are formed in fp32, whose error is
// bounded; a token with two values nearer than that bound where their order matters (about one in
// a thousand) is chosen again with 64-bit scores. Without a bias the logits themselves are
// compared, which is exact.
//
// Choosing k of E: L = 16 lanes hold a token (four tokens a wavefront; 64 lanes beyond 256 experts
// or 16 choices). k rounds of a maximum over the lanes' own maxima give a value that at least k
// experts reach and, the lanes being as random samples, few others (about k + 4 of 256 for k = 8);
// those are gathered in LDS and each counts the ones ahead of it. A round costs four DPP steps, not
// a pass over all E.
#include <algorithm>

#include "block_common.hpp"
#include "launch.hpp"

namespace moe {

constexpr int kScoresThreads = 256;
constexpr float kUnavailable = -INFINITY;

struct RouteArgs {
    const float* logits;
    const float* bias;  // nullable
    int T, E, k;
    int sigmoid, groups, kept, top, renorm;
    float scale;
    uint32_t group_mul;  // e / (E / groups) = e * group_mul >> 22
    int32_t* topk_idx;
    float* topk_w;
    int32_t* err_word;  // nullable
    int CT;             // tokens a workgroup
    int32_t* hist;      // [workgroups, E], or nullptr: no counts
    int32_t* src_of;    // filled with -1 beside the counts
    int64_t M_cap;
};

// LDS of a wavefront: candidates (or, for a 64-bit choice, all scores), the groups' values, and the
// chosen experts of its tokens.
template <int L, int PER>
struct RouteLds {
    static constexpr int kTokens = 64 / L, kRow = L * PER;
    union {
        uint2 cand[kTokens][kRow];  // key, expert
        float key[kTokens][kRow];
        double exact[64 * PER];
    };
    double gexact[kRouteMaxGroups];
    float gval[kTokens][kRouteMaxGroups];
    uint16_t sel[kTokens][kRouteMaxTopk];
    uint8_t gkept[kTokens][kRouteMaxGroups];
};

__device__ __forceinline__ float logistic(float x) { return 1.f / (1.f + __expf(-x)); }

// exp(a - b) with the rounding of the difference made good: it would be an error of up to 2^-24 |a - b| of
// the result.
__device__ __forceinline__ float exp_of_difference(float a, float b) {
    const float d = a - b, bb = d - a;
    const float e = (a - (d - bb)) - (b + bb);
    return expf(d) * (1.f + e);
}

// A chosen expert's score from its logit. Renormalised weights take it over exp(shift), shift the best chosen
// logit (the sigmoid's: where that is negative), so that they keep their precision where all scores underflow.
struct SlotScore {
    bool sigmoid, renorm;
    float shift, mx, inv;  // mx, inv: a softmax's maximum and 1 / sum over all experts
    __device__ __forceinline__ float operator()(float v) const {
        if (renorm) return sigmoid ? exp_of_difference(fminf(v, 0.f), shift) / (1.f + expf(-fabsf(v))) : exp_of_difference(v, shift);
        return sigmoid ? 1.f / (1.f + expf(-v)) : exp_of_difference(v, mx) * inv;
    }
};

// Are the scores of two experts with equal fp32 values certainly equal, or only near?
__device__ __forceinline__ bool same_inputs(const RouteArgs& p, const float* row, int a, int b) {
    return row[a] == row[b] && (!p.bias || p.bias[a] == p.bias[b]);
}

__device__ __forceinline__ bool available(const RouteArgs& p, const float* row, int e) {
    return isfinite(row[e]) && (!p.bias || isfinite(p.bias[e]));
}

// The choice for token t by a whole wavefront, with 64-bit scores. A dropped expert's key is NaN, which
// no comparison prefers.
__device__ __forceinline__ void choose_exact(const RouteArgs& p, int t, double* key, double* gval, uint8_t* gkept,
                                             uint16_t* sel) {
    const int lane = lane_id();
    const float* row = p.logits + (int64_t)t * p.E;
    double mx = -INFINITY, sum = 0;
    if (!p.sigmoid) {
        for (int e = lane; e < p.E; e += 64)
            if (isfinite(row[e])) mx = fmax(mx, (double)row[e]);
        for (int o = 32; o > 0; o >>= 1) mx = fmax(mx, __shfl_xor(mx, o, 64));
        for (int e = lane; e < p.E; e += 64)
            if (isfinite(row[e])) sum += exp((double)row[e] - mx);
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
    }
    auto score = [&](int e) -> double {
        return p.sigmoid ? 1.0 / (1.0 + exp(-(double)row[e])) : exp((double)row[e] - mx) / sum;
    };
    const bool by_score = p.bias || (p.groups > 1 && p.top == 2);
    wave_lds_sync();
    for (int e = lane; e < p.E; e += 64) {
        double v = -INFINITY;
        if (available(p, row, e)) v = by_score ? score(e) + (p.bias ? (double)p.bias[e] : 0.0) : (double)row[e];
        key[e] = v;
    }
    wave_lds_sync();
    if (p.groups > 1) {
        const int gs = p.E / p.groups;
        if (lane < p.groups) {
            double a = -INFINITY, b = -INFINITY;
            for (int e = lane * gs; e < (lane + 1) * gs; ++e) {
                const double v = key[e];
                b = fmax(b, fmin(a, v));
                a = fmax(a, v);
            }
            gval[lane] = p.top == 2 && b > -INFINITY ? a + b : a;
        }
        wave_lds_sync();
        if (lane < p.groups) {
            const double v = gval[lane];
            int rank = 0;
            for (int g = 0; g < p.groups; ++g) rank += gval[g] > v || (gval[g] == v && g < lane);
            gkept[lane] = rank < p.kept;
        }
        wave_lds_sync();
        for (int e = lane; e < p.E; e += 64) {
            if (!gkept[(uint32_t)e * p.group_mul >> 22]) key[e] = NAN;
            else if (!p.bias && key[e] > -INFINITY) key[e] = row[e];  // within the groups the logits decide
        }
        wave_lds_sync();
    }
    for (int j = 0; j < p.k; ++j) {
        double bv = -INFINITY;
        int be = 0x7fffffff;
        for (int e = lane; e < p.E; e += 64) {
            const double v = key[e];
            if (v > bv || (v == bv && e < be)) {
                bv = v;
                be = e;
            }
        }
        for (int o = 32; o > 0; o >>= 1) {
            const double ov = __shfl_xor(bv, o, 64);
            const int oe = __shfl_xor(be, o, 64);
            if (ov > bv || (ov == bv && oe < be)) {
                bv = ov;
                be = oe;
            }
        }
        if (lane == 0) {
            sel[j] = (uint16_t)be;
            key[be] = NAN;
        }
        wave_lds_sync();
    }
}

template <int L, int PER>
__global__ void __launch_bounds__(kScoresThreads) route_scores_kernel(RouteArgs p) {
    constexpr int TW = 64 / L, TB = kScoresThreads / L;  // tokens a wavefront, a workgroup and pass
    __shared__ RouteLds<L, PER> s_lds[kScoresThreads / 64];
    __shared__ int32_t s_cnt[MOE_MAX_E];
    const int lane = lane_id(), gl = lane % L, tw = lane / L;
    RouteLds<L, PER>& lds = s_lds[threadIdx.x >> 6];
    const int E = p.E, k = p.k;
    if (p.hist) {
        for (int e = threadIdx.x; e < E; e += kScoresThreads) s_cnt[e] = 0;
        for (int64_t r = (int64_t)blockIdx.x * kScoresThreads + threadIdx.x; r < p.M_cap;
             r += (int64_t)gridDim.x * kScoresThreads)
            p.src_of[r] = -1;
        __syncthreads();
    }
    const bool whole = (E & 3) == 0 && ((uintptr_t)p.logits & 15) == 0;  // rows in 16-byte pieces
    const bool by_score = p.bias != nullptr;
    auto expert = [&](int i) { return 4 * (gl + L * (i >> 2)) + (i & 3); };
    // every lane of a workgroup runs the token loop equally often; a token past the end is idle
    const int64_t t0 = (int64_t)blockIdx.x * p.CT, t1 = min((int64_t)p.T, t0 + p.CT);
    for (int64_t tb = t0; tb < t1; tb += TB) {
        const int64_t t = tb + threadIdx.x / L;
        const bool live = t < t1;
        const float* row = p.logits + (live ? t : t0) * E;
        float x[PER], key[PER];
        bool bad = false;
#pragma unroll
        for (int q = 0; q < PER / 4; ++q) {
            const int e = expert(4 * q);
            if (whole) {
                const float4 v = e < E ? *(const float4*)(row + e) : make_float4(0, 0, 0, 0);
                x[4 * q] = v.x, x[4 * q + 1] = v.y, x[4 * q + 2] = v.z, x[4 * q + 3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[4 * q + j] = e + j < E ? row[e + j] : 0.f;
            }
        }
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool fin = isfinite(x[i]);
            bad |= live && !fin && expert(i) < E;
            if (!fin || expert(i) >= E) x[i] = -INFINITY;  // never preferred
            mx = fmaxf(mx, x[i]);
        }
        if (__ballot(bad) != 0ull && lane == 0 && p.err_word) atomicOr(p.err_word, MOE_ERRBIT_NONFINITE_LOGIT);
        mx = lanes_max<L>(mx);
        // a score is p.sigmoid ? logistic(x) : exp(x - mx) * inv
        float inv = 1.f;
        if (!p.sigmoid) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) sum += x[i] > -INFINITY ? __expf(x[i] - mx) : 0.f;
            sum = lanes_sum<L>(sum);
            inv = sum > 0.f ? 1.f / sum : 0.f;
        }
        auto score = [&](float v) { return p.sigmoid ? logistic(v) : __expf(v - mx) * inv; };
        // How far apart two fp32 values have to be for their order to be that of the exact ones: a score is
        // off by at most 8 steps of 2^-24 of itself (exponential, sum, reciprocal, product) and its sum with
        // the bias by one of 2^-24 of that; twice, and doubled for the margin.
        const float smax = p.sigmoid ? 1.f : inv;
        auto near = [&](float v) { return v > -INFINITY ? 0x1p-19f * smax + 0x1p-21f * fabsf(v) : 0.f; };
        bool doubt = false;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            key[i] = x[i];
            if (by_score) {
                const int e = expert(i);
                const float b = e < E ? p.bias[e] : 0.f;
                key[i] = x[i] > -INFINITY && isfinite(b) ? score(x[i]) + b : kUnavailable;
            }
        }
        if (p.groups > 1) {
            const bool exact = !by_score && p.top == 1;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (expert(i) < E)
                    lds.key[tw][expert(i)] = by_score || exact || !(x[i] > -INFINITY) ? key[i] : score(x[i]);
            }
            wave_lds_sync();
            const int gs = E / p.groups;
            for (int g = gl; g < p.groups; g += L) {
                float a = -INFINITY, b = -INFINITY;
                for (int e = g * gs; e < (g + 1) * gs; ++e) {
                    const float v = lds.key[tw][e];
                    b = fmaxf(b, fminf(a, v));
                    a = fmaxf(a, v);
                }
                lds.gval[tw][g] = p.top == 2 && b > -INFINITY ? a + b : a;
            }
            wave_lds_sync();
            for (int g = gl; g < p.groups; g += L) {
                const float v = lds.gval[tw][g];
                int rank = 0;
                bool close = false;
                for (int o = 0; o < p.groups; ++o) {
                    const float u = lds.gval[tw][o];
                    rank += u > v || (u == v && o < g);
                    close |= o != g && fabsf(u - v) <= 2.f * near(v);  // not where both are -inf
                }
                lds.gkept[tw][g] = rank < p.kept;
                // a pair on two sides of the border holds one that is kept and near another
                doubt |= !exact && close && rank < p.kept;
            }
            wave_lds_sync();
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = expert(i);
                if (e >= E || !lds.gkept[tw][(uint32_t)e * p.group_mul >> 22]) key[i] = NAN;  // dropped
            }
            wave_lds_sync();
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (expert(i) >= E) key[i] = NAN;
        }
        // a value that at least k keys reach: the k-th largest of the lanes' maxima
        float most = -INFINITY, least = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) most = fmaxf(most, key[i]);  // not the NaN
        for (int r = 0; r < k; ++r) {
            least = lanes_max<L>(most);
            if (most == least) most = -INFINITY;
        }
        const float floor_ = by_score ? least - near(least) : least;
        int mine = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) mine += key[i] >= floor_ ? 1 : 0;
        int at = mine;  // inclusive prefix over the token's lanes
#pragma unroll
        for (int o = 1; o < L; o <<= 1) {
            const int u = __shfl_up(at, o, L);
            if (gl >= o) at += u;
        }
        const int m = __shfl(at, L - 1, L);
        at -= mine;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (key[i] >= floor_) lds.cand[tw][at++] = make_uint2(__float_as_uint(key[i]), (uint32_t)expert(i));
        }
        wave_lds_sync();
        for (int c = gl; c < m; c += L) {
            const uint2 own = lds.cand[tw][c];
            const float v = __uint_as_float(own.x);
            const float d = near(v);
            int rank = 0;
            bool close = false;
            for (int j = 0; j < m; ++j) {
                const uint2 o = lds.cand[tw][j];
                const float u = __uint_as_float(o.x);
                rank += u > v || (u == v && o.y < own.y);
                if (by_score && fabsf(u - v) <= d && j != c) close |= !(u == v && same_inputs(p, row, (int)o.y, (int)own.y));
            }
            if (rank < k) {
                lds.sel[tw][rank] = (uint16_t)own.y;
                doubt |= close;
            }
        }
        // the tokens in doubt, one after the other, by the whole wavefront
        uint64_t todo = __ballot(doubt && live);
        while (todo) {
            const int w = (__ffsll((unsigned long long)todo) - 1) / L;
            wave_lds_sync();
            choose_exact(p, (int)(tb + (threadIdx.x >> 6) * TW + w), lds.exact, lds.gexact, lds.gkept[w], lds.sel[w]);
            todo &= L == 64 ? 0ull : ~(((1ull << (L & 63)) - 1) << (w * L));
        }
        wave_lds_sync();
        // weights, slot by slot
        float xs = -INFINITY;
        for (int j = gl; j < k; j += L) {
            const int e = lds.sel[tw][j];
            if (live && available(p, row, e)) xs = fmaxf(xs, row[e]);
        }
        xs = lanes_max<L>(xs);
        const SlotScore slot{p.sigmoid != 0, p.renorm != 0, p.sigmoid ? fminf(xs, 0.f) : xs, mx, inv};
        auto weight = [&](int e) { return available(p, row, e) ? slot(row[e]) : 0.f; };
        float total = 0.f;
        if (p.renorm) {
            for (int j = gl; j < k; j += L) total += live ? weight(lds.sel[tw][j]) : 0.f;
            total = lanes_sum<L>(total);
        }
        const float f = !p.renorm ? p.scale : total > 0.f ? p.scale / total : 0.f;
        for (int j = gl; j < k; j += L) {
            if (!live) continue;
            const int e = lds.sel[tw][j];
            p.topk_idx[t * k + j] = e;
            p.topk_w[t * k + j] = f * weight(e);
            if (p.hist) atomicAdd(&s_cnt[e], 1);
        }
        wave_lds_sync();  // the next tokens may overwrite the lists
    }
    if (p.hist) {
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += kScoresThreads) p.hist[(int64_t)blockIdx.x * E + e] = s_cnt[e];
    }
}

// ---- backward --------------------------------------------------------------
struct RouteBwdArgs {
    const float* logits;
    const float* bias;
    const int32_t* topk_idx;
    const float* ds;
    int T, E, k;
    int sigmoid, renorm;
    float scale;
    float* dlogits;
};

// dlogits from dL/dw of the chosen experts. With p_j their scores (0 for one without a finite logit and
// bias), S their sum, r_j = p_j / S:
//   renormalised     dL/dl_j = scale r_j (1 - p_j) (ds_j - sum_i r_i ds_i)  (sigmoid; a softmax without 1 - p_j)
//   sigmoid, plain   dL/dl_j = scale ds_j p_j (1 - p_j)
//   softmax, plain   dL/dl_e = scale p_e (g_e - sum_j p_j ds_j), g_e = ds_j for a chosen one, else 0
// and 0 for every other expert. L lanes a token; the slots' values go through an LDS row.
template <int L, int PER>
__global__ void __launch_bounds__(256) route_scores_bwd_kernel(RouteBwdArgs p) {
    __shared__ __align__(16) float s_row[256 / L][L * PER];
    const int gl = lane_id() % L;
    const int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    const bool live = t < p.T;
    const int E = p.E, k = p.k;
    float* g = s_row[threadIdx.x / L];
    const float* row = p.logits + (live ? t : 0) * E;
    const bool whole = (E & 3) == 0 && (((uintptr_t)p.logits | (uintptr_t)p.dlogits) & 15) == 0;
    auto expert = [&](int i) { return 4 * (gl + L * (i >> 2)) + (i & 3); };
#pragma unroll
    for (int q = 0; q < PER / 4; ++q) *(float4*)(g + expert(4 * q)) = make_float4(0, 0, 0, 0);
    const bool dense = !p.sigmoid && !p.renorm;
    float x[PER], mx = -INFINITY, inv = 0.f;
    if (dense) {
#pragma unroll
        for (int q = 0; q < PER / 4; ++q) {
            const int e = expert(4 * q);
            if (whole) {
                const float4 v = e < E ? *(const float4*)(row + e) : make_float4(0, 0, 0, 0);
                x[4 * q] = v.x, x[4 * q + 1] = v.y, x[4 * q + 2] = v.z, x[4 * q + 3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[4 * q + j] = e + j < E ? row[e + j] : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (!isfinite(x[i]) || expert(i) >= E) x[i] = -INFINITY;
            mx = fmaxf(mx, x[i]);
        }
        mx = lanes_max<L>(mx);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            x[i] = x[i] > -INFINITY ? __expf(x[i] - mx) : 0.f;
            sum += x[i];
        }
        sum = lanes_sum<L>(sum);
        inv = sum > 0.f ? 1.f / sum : 0.f;
    }
    auto slot = [&](int j) -> int {  // the expert of slot j, or -1: none that has a gradient
        if (!live) return -1;
        const int e = p.topk_idx[t * k + j];
        if ((uint32_t)e >= (uint32_t)E) return -1;
        return isfinite(row[e]) && (!p.bias || isfinite(p.bias[e])) ? e : -1;
    };
    float xs = -INFINITY;
    if (p.renorm) {
        for (int j = gl; j < k; j += L) {
            const int e = slot(j);
            if (e >= 0) xs = fmaxf(xs, row[e]);
        }
        xs = lanes_max<L>(xs);
    }
    const SlotScore weight{p.sigmoid != 0, p.renorm != 0, p.sigmoid ? fminf(xs, 0.f) : xs, mx, inv};
    float total = 1.f, dot = 0.f;
    if (p.renorm) {
        total = 0.f;
        for (int j = gl; j < k; j += L) {
            const int e = slot(j);
            if (e >= 0) total += weight(row[e]);
        }
        total = lanes_sum<L>(total);
    }
    for (int j = gl; j < k; j += L) {
        const int e = slot(j);  // divided, not times a reciprocal: a lone weight is 1 and has no gradient
        if (e >= 0) dot = fmaf(weight(row[e]) / total, p.ds[t * k + j], dot);
    }
    dot = lanes_sum<L>(dot);
    wave_lds_sync();
    for (int j = gl; j < k; j += L) {
        const int e = slot(j);
        if (e < 0) continue;
        const float v = row[e], d = p.ds[t * k + j];
        if (dense) {
            g[e] = d;
        } else {
            const float w = weight(v) / total;
            g[e] = p.scale * w * (p.sigmoid ? 1.f / (1.f + expf(v)) : 1.f) * (p.renorm ? d - dot : d);
        }
    }
    wave_lds_sync();
    if (!live) return;
    float* out = p.dlogits + t * E;
#pragma unroll
    for (int q = 0; q < PER / 4; ++q) {
        const int e = expert(4 * q);
        float4 v = *(const float4*)(g + e);
        if (dense) {
            v.x = p.scale * x[4 * q] * inv * (v.x - dot);
            v.y = p.scale * x[4 * q + 1] * inv * (v.y - dot);
            v.z = p.scale * x[4 * q + 2] * inv * (v.z - dot);
            v.w = p.scale * x[4 * q + 3] * inv * (v.w - dot);
        }
        if (whole) {
            if (e < E) *(float4*)(out + e) = v;
        } else {
            if (e < E) out[e] = v.x;
            if (e + 1 < E) out[e + 1] = v.y;
            if (e + 2 < E) out[e + 2] = v.z;
            if (e + 3 < E) out[e + 3] = v.w;
        }
    }
}

// ---- launch ----------------------------------------------------------------
// 16 lanes a token up to 256 experts and 16 choices, else 64.
template <class F>
static void by_experts(int E, int k, F&& f) {
    using std::integral_constant;
    if (E <= 256 && k <= 16) {
        if (E <= 64) f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
        else if (E <= 128) f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
        else f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    } else if (E <= 256) {
        f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    } else if (E <= 512) {
        f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
    } else {
        f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
    }
}

// Two kernels where a chunk's workgroup of the second can afford to read all chunks' counts (the limits of
// moe_route_counts), a chunk being at most 64 tokens; else choice, counts, their scan and the ranks.
struct ScoresPlan {
    bool fused;
    int CT, nchunks;
};
static ScoresPlan scores_plan(int T, int k, int E) {
    const int tb = kScoresThreads / (E <= 256 && k <= 16 ? 16 : 64);
    for (int ct = tb; ct <= 64; ct *= 2) {
        const int64_t nc = ((int64_t)T + ct - 1) / ct;
        if (layout_fused_fits(nc, E)) return {true, ct, (int)nc};
    }
    return {false, tb, (int)(((int64_t)T * k + kChunkPairs - 1) / kChunkPairs)};
}

size_t route_scores_workspace_bytes(int T, int k, int E) {
    const ScoresPlan pl = scores_plan(T, k, E);
    return (pl.fused ? 1 : 2) * (size_t)pl.nchunks * E * sizeof(int32_t);
}

int launch_route_scores(const RouteCall& c, hipStream_t s) {
    const ScoresPlan pl = scores_plan(c.T, c.k, c.E);
    RouteArgs p{};
    p.logits = c.logits, p.bias = c.bias, p.T = c.T, p.E = c.E, p.k = c.k;
    p.sigmoid = c.sigmoid, p.groups = c.groups, p.kept = c.kept, p.top = c.top, p.renorm = c.renorm, p.scale = c.scale;
    const uint32_t gs = (uint32_t)(c.E / c.groups);
    p.group_mul = ((1u << 22) + gs - 1) / gs;
    p.topk_idx = c.topk_idx, p.topk_w = c.topk_w, p.err_word = c.err_word;
    p.CT = pl.CT;
    if (pl.fused) p.hist = (int32_t*)c.ws, p.src_of = c.src_of, p.M_cap = c.M_cap;
    const unsigned grid = (unsigned)(((int64_t)c.T + pl.CT - 1) / pl.CT);
    by_experts(c.E, c.k, [&](auto A, auto B) {
        route_scores_kernel<decltype(A)::value, decltype(B)::value><<<grid, kScoresThreads, 0, s>>>(p);
    });
    if (pl.fused)
        launch_layout_fused(c.topk_idx, c.T, c.k, c.E, pl.CT, pl.nchunks, (const int32_t*)c.ws, c.counts, c.offsets,
                            c.row_of, c.src_of, s);
    else
        launch_layout(c.topk_idx, c.T, c.k, c.E, pl.nchunks, (int32_t*)c.ws, c.counts, c.offsets, c.row_of, c.src_of,
                      c.M_cap, s);
    return hipGetLastError() == hipSuccess ? 0 : -4;
}

int launch_route_scores_bwd(const float* logits, const float* bias, const int32_t* topk_idx, const float* ds, int T,
                            int E, int k, int sigmoid, int renorm, float scale, float* dlogits, hipStream_t s) {
    const RouteBwdArgs p{logits, bias, topk_idx, ds, T, E, k, sigmoid, renorm, scale, dlogits};
    by_experts(E, k, [&](auto A, auto B) {
        constexpr int L = decltype(A)::value, PER = decltype(B)::value;
        const unsigned grid = (unsigned)(((int64_t)T + 256 / L - 1) / (256 / L));
        route_scores_bwd_kernel<L, PER><<<grid, 256, 0, s>>>(p);
    });
    return hipGetLastError() == hipSuccess ? 0 : -4;
}

}  // namespace moe
