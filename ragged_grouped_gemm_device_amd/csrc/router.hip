// The router with scores, a balance bias, groups of experts and renormalised weights, and its
// gradient (gfx950).
//
//   s = sigmoid(l) or softmax(l); c = s + b (b a bias that takes part in the choice alone);
//   a group of E / G neighbouring experts is worth its best c, or the sum of its two best;
//   the k best c within the best groups, ties to the lower index; w_j = scale s_j (/ sum_i s_i).
//
// The choice is that of 64-bit arithmetic at fp32 cost: scores are formed in fp32, whose error is
// bounded; a token with two values nearer than that bound where their order matters is chosen again with
// 64-bit scores, by a wavefront of its own (normal logits, sigmoid with a bias: 1 to 2 tokens in 1000 for k = 8 of
// up to 256 experts, 1 in 100 for 32 of 256, 7 in 100 for 64 of 1024; a softmax's fewer), and so is one with fewer
// than k experts available, or with more nearly equal ones than are ranked. Without a bias the logits themselves
// are compared, which is exact.
//
// Choosing k of E: L = 16 lanes hold a token (four tokens a wavefront; 64 lanes beyond 256 experts
// or 16 choices). k rounds of a maximum over the lanes' own maxima give a value that at least k
// experts reach and, the lanes being as random samples, few others (about k + 4 of 256 for k = 8);
// those are gathered in LDS and each counts the ones ahead of it. A round costs four DPP steps, not
// a pass over all E. Where fewer than k lanes hold an available expert (few experts, or few groups kept), all
// available ones are candidates; where more than 64 would be, the bound is found by halving its range. 131072 tokens,
// sigmoid with bias: 4 of 8 experts 38 us (2 of 8: 33), 8 of 64 in 3 of 8 groups 76 (in 4: 83), 16 of 256 173 (8:
// 85), 64 of 512 1.6 ms.
#include <algorithm>
#include <cfloat>

#include "block_common.hpp"
#include "launch.hpp"
#include "route_common.hpp"

namespace moe {

constexpr int kScoresThreads = 1024;  // 64 tokens a pass and workgroup with 16 lanes a token
constexpr int kScoresGroups = 256;    // workgroups at most: one a compute unit
constexpr int kMaxCand = 64;          // candidates that are ranked in fp32

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
    int32_t* hist;      // [workgroups, E]
    int32_t* src_of;
    int64_t M_cap;
};

// LDS of a wavefront: its tokens' choice values (or all 64-bit ones of a token), the candidates, the groups'
// values, and the chosen experts.
template <int L, int PER>
struct __align__(16) RouteLds {
    static constexpr int kTokens = 64 / L, kRow = L * PER, kSel = (L == 16 ? 16 : kRouteMaxTopk) + 2;
    union {
        float key[kTokens][kRow];
        double exact[kRow];
    };
    union {
        int who[kTokens][kMaxCand];  // candidates
        int chosen[kRouteMaxTopk];
    };
    uint64_t cand[kTokens][kMaxCand];  // their order: see order_of
    union {
        float gval[kTokens][kRouteMaxGroups];
        double gexact[kRouteMaxGroups];
        uint64_t sel[kTokens][kSel];  // the first k + 1 candidates
    };
    uint8_t gkept[kRouteMaxGroups];
};

// Integers in the order of the floats, and back. (-0 comes before 0: good for a bound, not for a choice.)
__device__ __forceinline__ int ordered(float v) {
    const int u = __float_as_int(v);
    return u ^ (int)((uint32_t)(u >> 31) >> 1);
}
__device__ __forceinline__ float from_ordered(int u) { return __int_as_float(u ^ (int)((uint32_t)(u >> 31) >> 1)); }

// One number in which larger keys, and of equal ones lower experts, are larger; 0 sorts behind them all.
__device__ __forceinline__ uint64_t order_of(float key, int e) {
    const uint32_t k = (uint32_t)ordered(key + 0.f) ^ 0x80000000u;  // -0 + 0 = 0
    return (uint64_t)k << 32 | (uint32_t)(0xffff - e);
}
__device__ __forceinline__ float key_of(uint64_t o) { return from_ordered((int)((uint32_t)(o >> 32) ^ 0x80000000u)); }
__device__ __forceinline__ int expert_of(uint64_t o) { return 0xffff - (int)(uint32_t)o; }

// The larger of two numbers of which none is a NaN: fmaxf first makes both quiet, one more instruction each.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, INFINITY); }
__device__ __forceinline__ float smaller(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, -INFINITY); }

template <int CTRL>
__device__ __forceinline__ int lane_dpp_i(int v) { return __builtin_amdgcn_mov_dpp(v, CTRL, 0xF, 0xF, true); }

template <int L>
__device__ __forceinline__ int lanes_max_i(int v) {
    v = max(v, lane_dpp_i<0xB1>(v));
    v = max(v, lane_dpp_i<0x4E>(v));
    v = max(v, lane_dpp_i<0x141>(v));
    v = max(v, lane_dpp_i<0x140>(v));
    if constexpr (L == 64) {
        v = max(v, __shfl_xor(v, 16, 64));
        v = max(v, __shfl_xor(v, 32, 64));
    }
    return v;
}

// Inclusive prefix sum over the lanes of a group (row shifts bring 0 in from outside a row).
template <int L>
__device__ __forceinline__ int lanes_scan(int v, int gl) {
    v += lane_dpp_i<0x111>(v);
    v += lane_dpp_i<0x112>(v);
    v += lane_dpp_i<0x114>(v);
    v += lane_dpp_i<0x118>(v);
    if constexpr (L == 64) {
        const int a = __shfl(v, 15, 64), b = __shfl(v, 31, 64), c = __shfl(v, 47, 64);
        v += (gl >= 16 ? a : 0) + (gl >= 32 ? b : 0) + (gl >= 48 ? c : 0);
    }
    return v;
}

// exp(a - b) with the rounding of the difference made good: it would be an error of up to 2^-24 |a - b| of
// the result. Below -104 the result is 0 in fp32, and there the difference itself may overflow (its rounding is
// then a NaN).
__device__ __forceinline__ float exp_of_difference(float a, float b) {
    const float d = a - b, bb = d - a;
    const float e = (a - (d - bb)) - (b + bb);
    return d > -104.f ? expf(d) * (1.f + e) : 0.f;
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

__device__ __forceinline__ bool available(const RouteArgs& p, const float* row, int e) {
    return isfinite(row[e]) && (!p.bias || isfinite(p.bias[e]));
}

// Token t by a whole wavefront, with 64-bit scores: its choice, weights and counts. A dropped expert's key is
// NaN, which no comparison prefers. sel: LDS of kRouteMaxTopk experts.
__device__ __forceinline__ void route_exact(const RouteArgs& p, int64_t t, double* key, double* gval, uint8_t* gkept,
                                            int* sel, int32_t* cnt) {
    const int lane = lane_id();
    const float* row = p.logits + t * p.E;
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
        const double x = row[e];
        const double v = exp(p.sigmoid ? -x : x - mx);
        return p.sigmoid ? 1.0 / (1.0 + v) : v / sum;
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
            sel[j] = be;
            key[be] = NAN;
        }
        wave_lds_sync();
    }
    const bool mine = lane < p.k;
    const int e = mine ? sel[lane] : 0;
    const bool ok = mine && available(p, row, e);
    double w = 0;
    if (p.renorm) {  // over the best chosen logit, so that scores that underflow keep their ratios
        const double x = ok ? (double)row[e] : -INFINITY;
        double xs = x;
        for (int o = 32; o > 0; o >>= 1) xs = fmax(xs, __shfl_xor(xs, o, 64));
        if (ok) w = p.sigmoid ? exp(fmin(x, 0.0) - fmin(xs, 0.0)) / (1.0 + exp(-fabs(x))) : exp(x - xs);
        double total = w;
        for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o, 64);
        if (ok) w /= total;
    } else if (ok) {
        w = score(e);
    }
    if (mine) {
        p.topk_idx[t * p.k + lane] = e;
        p.topk_w[t * p.k + lane] = (float)(p.scale * w);
        atomicAdd(&cnt[e], 1);
    }
    wave_lds_sync();
}

// SIGMOID: the scores; BIAS: there is one, so that scores and not logits are compared. 131072 x 256, k = 8, sigmoid
// with bias and groups: 91 us (134 MB of logits, 1.5 TB/s); 16 x 256: 9.3. Bound by its instructions and their
// latency (about 880 vector instructions for the four tokens of a wavefront, those in doubt included; four wavefronts
// a SIMD by registers and LDS), so the steps are written to be few: values that
// take no part are -inf, not NaN; maxima are integers where lanes exchange them; the candidates are found from
// a bit mask a lane; their order is one 64-bit comparison.
template <int L, int PER, bool SIGMOID, bool BIAS>
__global__ void __launch_bounds__(kScoresThreads) route_scores_kernel(RouteArgs p) {
    constexpr int TB = kScoresThreads / L;  // tokens a workgroup and pass
    __shared__ RouteLds<L, PER> s_lds[kScoresThreads / 64];
    __shared__ int32_t s_cnt[MOE_MAX_E];
    const int lane = lane_id(), gl = lane % L, tw = lane / L;
    RouteLds<L, PER>& lds = s_lds[threadIdx.x >> 6];
    const int E = p.E, k = p.k;
    const bool whole = (E & 3) == 0 && (((uintptr_t)p.logits | (uintptr_t)p.bias) & 15) == 0;  // rows in 16-byte pieces
    auto expert = [&](int i) { return 4 * (gl + L * (i >> 2)) + (i & 3); };
    // a row of E values, 16 bytes at a time, -inf past its end; other rows by way of LDS
    auto load_row = [&](const float* row, float (&v)[PER]) {
        if (!whole) {
            wave_lds_sync();
            for (int e = gl; e < ((E + 3) & ~3); e += L) lds.key[tw][e] = e < E ? row[e] : -INFINITY;
            wave_lds_sync();
        }
#pragma unroll
        for (int q = 0; q < PER / 4; ++q) {
            const int e = expert(4 * q);
            float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (e < E) f = whole ? *(const float4*)(row + e) : *(const float4*)&lds.key[tw][e];
            v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
        }
        if (!whole) wave_lds_sync();
    };
    int absent = 0;  // values that this lane holds past the last expert
#pragma unroll
    for (int i = 0; i < PER; ++i) absent += expert(i) >= E;
    const int64_t t0 = (int64_t)blockIdx.x * p.CT, t1 = min((int64_t)p.T, t0 + p.CT);
    const int64_t mine = t0 + threadIdx.x / L;  // this group's first token
    float x[PER], bias[PER];
    if (whole && mine - tw < t1) load_row(p.logits + min(mine, t1 - 1) * E, x);
    if constexpr (BIAS) {
        load_row(p.bias, bias);
#pragma unroll
        for (int i = 0; i < PER; ++i) bias[i] = isfinite(bias[i]) ? bias[i] : -INFINITY;
    }
    for (int e = threadIdx.x; e < E; e += kScoresThreads) s_cnt[e] = 0;
    for (int64_t r = (int64_t)blockIdx.x * kScoresThreads + threadIdx.x; r < p.M_cap;
         r += (int64_t)gridDim.x * kScoresThreads)
        p.src_of[r] = -1;
    __syncthreads();
    const int gs = E / p.groups;
    // lanes that share a group's members, in whole 16-byte pieces
    int per_group = 1;
    while (2 * per_group * p.groups <= L && gs % (8 * per_group) == 0) per_group *= 2;
    // a wavefront's tokens leave the loop together (lane exchanges need all of them); one past the end is idle
    for (int64_t t = mine; t - tw < t1; t += TB) {
        const bool live = t < t1;
        const float* row = p.logits + min(t, t1 - 1) * E;
        if (!whole) load_row(row, x);
        // Opaque, so that what follows from it for each of PER values is formed where it is used: kept over the
        // loop, those indexes take more registers than there are.
        uint32_t mul = p.group_mul;
        asm volatile("" : "+s"(mul));
        float key[PER];
        int unfit = 0;
        float mx = -INFINITY, inv = 1.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool fin = fabsf(x[i]) < INFINITY;
            unfit += !fin;
            x[i] = fin ? x[i] : -INFINITY;  // never preferred
        }
        if (__ballot(live && unfit != absent) != 0ull && lane == 0 && p.err_word)
            atomicOr(p.err_word, MOE_ERRBIT_NONFINITE_LOGIT);
        if constexpr (!SIGMOID) {
#pragma unroll
            for (int i = 0; i < PER; ++i) mx = larger(mx, x[i]);
            mx = from_ordered(lanes_max_i<L>(ordered(mx)));
            const float shift = mx > -INFINITY ? mx : 0.f;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) sum += __expf(x[i] - shift);
            sum = lanes_sum<L>(sum);
            inv = sum > 0.f ? 1.f / sum : 0.f;
        }
        auto score = [&](float v) { return SIGMOID ? sigmoid_f(v) : __expf(v - mx) * inv; };
        // How far apart two fp32 values have to be for their order to be that of the exact ones: a score is
        // off by at most 8 steps of 2^-24 of the largest (exponential, sum, reciprocal, product) and its sum
        // with the bias by one of 2^-24 of that; twice, and doubled for the margin.
        const float smax = SIGMOID ? 1.f : inv;
        auto near = [&](float v) { return 0x1p-19f * smax + 0x1p-21f * fabsf(v); };
        bool doubt = false;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            key[i] = x[i];
            if constexpr (BIAS) {
                float c = score(x[i]) + bias[i];
                asm("" : "+v"(c));  // a selection, not a branch around the score
                key[i] = x[i] > -INFINITY ? c : -INFINITY;
            }
        }
        const bool plain = BIAS || p.top == 1;  // groups are valued by the keys themselves
#pragma unroll
        for (int q = 0; q < PER / 4; ++q) {
            float4 f = make_float4(key[4 * q], key[4 * q + 1], key[4 * q + 2], key[4 * q + 3]);
            if (p.groups > 1 && !plain) {
                auto valued = [&](float c) { return c > -INFINITY ? score(c) : c; };
                f = make_float4(valued(f.x), valued(f.y), valued(f.z), valued(f.w));
            }
            *(float4*)&lds.key[tw][expert(4 * q)] = f;
        }
        wave_lds_sync();
        if (p.groups > 1) {
            const bool exact = !BIAS && p.top == 1;
            const int g4 = (p.groups + 3) & ~3, part = gs / per_group;
            for (int j = gl; j < g4 * per_group; j += L) {
                const int g = j / per_group;
                float a = -INFINITY, b = -INFINITY;
                auto take = [&](float v) {
                    b = __builtin_amdgcn_fmed3f(a, b, v);
                    a = larger(a, v);
                };
                if (g < p.groups) {
                    const float* m = &lds.key[tw][j * part];
                    if ((part & 3) == 0) {
#pragma unroll 4
                        for (int i = 0; i < part; i += 4) {
                            const float4 f = *(const float4*)(m + i);
                            take(f.x), take(f.y), take(f.z), take(f.w);
                        }
                    } else {
#pragma unroll 4
                        for (int i = 0; i < part; ++i) take(m[i]);
                    }
                }
                for (int o = 1; o < per_group; o <<= 1) {  // partners are in the same turn: groups * per_group <= L
                    const float a2 = __shfl_xor(a, o, L), b2 = __shfl_xor(b, o, L);
                    b = larger(smaller(a, a2), larger(b, b2));
                    a = larger(a, a2);
                }
                const float worth = p.top == 2 && b > -INFINITY ? a + b : a;
                doubt |= b > -INFINITY && fabsf(worth) == INFINITY;  // past fp32, where the exact sums have an order
                if (j % per_group == 0) lds.gval[tw][g] = worth;
            }
            wave_lds_sync();
            uint64_t kept = 0;  // this token's groups
            for (int g0 = 0; g0 < p.groups; g0 += L) {
                const int g = g0 + gl;
                const float v = g < p.groups ? lds.gval[tw][g] : -INFINITY;
                const float d = 2.f * near(v);
                int rank = 0, close = 0;
#pragma unroll 2
                for (int o = 0; o < g4; o += 4) {
                    const float4 f = *(const float4*)&lds.gval[tw][o];
                    const float u[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        rank += (int)(u[j] > v) | ((int)(u[j] == v) & (int)(o + j < g));
                        close += fabsf(u[j] - v) <= d;  // itself; not where both are -inf
                    }
                }
                const bool keep = g < p.groups && rank < p.kept;
                // a pair on two sides of the border holds one that is kept and near another
                doubt |= !exact && keep && v > -INFINITY && close > 1;
                const uint64_t all = __ballot(keep);
                kept |= (L == 64 ? all : (all >> (lane & 48)) & 0xffffull) << g0;
            }
            auto dropped = [&](int i) { return !((kept >> (((uint32_t)expert(i) * mul >> 22) & 63)) & 1); };
            if ((gs & 3) == 0) {
#pragma unroll
                for (int q = 0; q < PER / 4; ++q) {
                    const bool drop = dropped(4 * q);
#pragma unroll
                    for (int j = 0; j < 4; ++j) key[4 * q + j] = drop ? -INFINITY : key[4 * q + j];
                }
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i) key[i] = dropped(i) ? -INFINITY : key[i];
            }
        }
        // the next tokens' logits, on the way while these are chosen
        if (whole && t + TB - tw < t1) load_row(p.logits + min(t + TB, t1 - 1) * E, x);
        // A value that at least k keys reach: the k-th largest of the lanes' maxima, their low bits the lane, so that
        // of equal ones a round takes out one. Where fewer lanes have any, all that are available.
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) top = larger(top, key[i]);
        int most = (ordered(top) & -L) | gl, least = most;
        for (int r = 0; r < k; ++r) {
            least = lanes_max_i<L>(most);
            most = most == least ? INT32_MIN : most;
        }
        const int lowest = ordered(-FLT_MAX);
        int reached = max(least & -L, lowest);
        uint32_t hits = 0;  // bit PER - 1 - i: key i
        int at = 0, m = 0;
        auto gather = [&](float from) {  // the keys from there on
            hits = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) hits = 2 * hits + (key[i] >= from ? 1u : 0u);
            const int n = __popc(hits);
            at = lanes_scan<L>(n, gl);
            m = L == 64 ? __shfl(at, 63, 64) : __shfl(at, 15, 16);
            at -= n;
        };
        auto from_reached = [&] {  // and those so near below that their order is not sure
            const float v = from_ordered(reached);
            return BIAS ? larger(v - near(v), -FLT_MAX) : v;
        };
        gather(from_reached());
        if (__ballot(m > kMaxCand) != 0ull) {
            // Too many to rank (k close to the lanes' number, or most lanes without a key): halve the range of
            // values, the last of which none reaches, until few more than k reach the bound.
            uint32_t span = (uint32_t)lanes_max_i<L>(ordered(top)) + 1u - (uint32_t)reached;
            while (__ballot(m > (k + kMaxCand) / 2 && span > 1) != 0ull) {
                const bool go = m > (k + kMaxCand) / 2 && span > 1;
                const int was = m, mid = reached + (int)(span / 2);
                gather(from_ordered(go ? mid : reached));
                const bool enough = m >= k;
                if (go) {
                    reached = enough ? mid : reached;
                    span = enough ? span - span / 2 : span / 2;
                    m = enough ? m : was;
                } else {
                    m = was;
                }
            }
            gather(from_reached());
        }
        // too few that are available: the exact form tells those apart that are kept from those that are not;
        // too many: nearly equal values
        const bool odd = m < k || m > kMaxCand;
        if (odd) hits = 0, m = 0;
        while (hits) {
            const int b = 31 - __clz((int)hits), i = PER - 1 - b;
            hits ^= 1u << b;
            lds.who[tw][at++] = expert(i);
        }
        wave_lds_sync();
        // The candidates' order. Their keys are in LDS, but as scores where groups are valued so and logits compared.
        const bool reread = !BIAS && p.groups > 1 && !plain;
        for (int c = gl; c < m; c += L) {
            const int e = lds.who[tw][c];
            lds.cand[tw][c] = order_of(reread ? row[e] : lds.key[tw][e], e);
        }
        wave_lds_sync();
        for (int c = gl; c < m; c += L) {
            const uint64_t own = lds.cand[tw][c];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < m; ++j) rank += lds.cand[tw][j] > own;
            if (rank <= k) lds.sel[tw][rank] = own;
        }
        if (m == k && gl == 0) lds.sel[tw][k] = 0;  // none behind the last
        wave_lds_sync();
        // slot by slot: every lane has at most one
        const bool slots = gl < k && !odd;
        const uint64_t own = slots ? lds.sel[tw][gl] : 0, next = slots ? lds.sel[tw][gl + 1] : 0;
        const int e = expert_of(own);
        const float value = key_of(own);
        float logit = value;
        if (BIAS && slots) logit = row[e];
        if (BIAS && slots) doubt |= next != 0 && value - key_of(next) <= near(value);
        // a token in doubt is marked, and left for below
        const uint64_t any = __ballot(doubt || odd);
        const bool sure = live && (L == 64 ? any : (any >> (lane & 48)) & 0xffffull) == 0;
        const bool mine_ = slots && sure;
        const float xs = p.renorm ? lanes_max<L>(mine_ ? logit : -INFINITY) : 0.f;
        const SlotScore slot{SIGMOID, p.renorm != 0, SIGMOID ? fminf(xs, 0.f) : xs, mx, inv};
        float w = mine_ ? slot(logit) : 0.f;
        if (p.renorm) {
            const float total = lanes_sum<L>(w);
            w = total > 0.f ? w / total : 0.f;
        }
        if (mine_) {
            p.topk_idx[t * k + gl] = e;
            p.topk_w[t * k + gl] = p.scale * w;
            atomicAdd(&s_cnt[e], 1);
        } else if (live && !sure && gl == 0) {
            p.topk_idx[t * k] = -1;
        }
        wave_lds_sync();  // the next tokens may overwrite the lists
    }
    __syncthreads();
    // the tokens in doubt, 64 marks at a time; in a loop of its own, or its 64-bit values would take the
    // registers of the one above
    for (int64_t b = t0 + (threadIdx.x & ~63); b < t1; b += kScoresThreads) {
        uint64_t todo = __ballot(b + lane < t1 && p.topk_idx[(b + lane) * k] < 0);
        while (todo) {
            const int at = __ffsll((unsigned long long)todo) - 1;
            route_exact(p, b + at, lds.exact, lds.gexact, lds.gkept, lds.chosen, s_cnt);
            todo &= todo - 1;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kScoresThreads) p.hist[(int64_t)blockIdx.x * E + e] = s_cnt[e];
}

// The layout from the workgroups' counts, one workgroup of 16 wavefronts a chunk of CT tokens: it sums all
// counts (the experts' totals) and those before its own, forms the regions' starts, and ranks its pairs in
// order, each wavefront a sixteenth of them after those before it. Integer sums: the order does not matter. 131072 x 8
// of 256: 17.8 us; 16 tokens 5.1.
__global__ void __launch_bounds__(kScoresThreads) scores_layout_kernel(const int32_t* __restrict__ topk_idx, int T,
                                                                       int k, int E, int nbits, int CT, int nchunks,
                                                                       const int32_t* __restrict__ hist,
                                                                       int32_t* __restrict__ counts,
                                                                       int32_t* __restrict__ offsets,
                                                                       int32_t* __restrict__ row_of,
                                                                       int32_t* __restrict__ src_of) {
    constexpr int NW = kScoresThreads / 64;
    __shared__ int32_t s_tot[MOE_MAX_E], s_base[MOE_MAX_E];
    __shared__ int32_t s_q[NW][MOE_MAX_E];  // the wavefronts' counts, then their first rows
    const int tid = threadIdx.x, wave = tid >> 6, lane = lane_id(), c = blockIdx.x;
    s_tot[tid] = s_base[tid] = 0;
    for (int e = lane; e < E; e += 64) s_q[wave][e] = 0;
    __syncthreads();
    const int64_t p0 = (int64_t)c * CT * k, p1 = min((int64_t)T * k, p0 + (int64_t)CT * k);
    const int64_t len = (p1 - p0 + NW - 1) / NW;
    const int64_t q0 = min(p1, p0 + wave * len), q1 = min(p1, q0 + len);
    for (int64_t q = q0 + lane; q < q1; q += 64) atomicAdd(&s_q[wave][topk_idx[q]], 1);
    {
        // thread (e, part) sums the chunks part, part + parts, ... of expert e, 8 loads in flight
        const int parts = kScoresThreads / E, part = tid / E, e = tid - part * E;
        if (part < parts) {
            int32_t tot = 0, base = 0;
            for (int cb = part; cb < nchunks; cb += 8 * parts) {
                int32_t h[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int cc = cb + u * parts;
                    h[u] = cc < nchunks ? hist[(int64_t)cc * E + e] : 0;
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    tot += h[u];
                    base += cb + u * parts < c ? h[u] : 0;
                }
            }
            atomicAdd(&s_tot[e], tot);
            atomicAdd(&s_base[e], base);
        }
    }
    __syncthreads();
    // regions' starts by one wavefront, 16 experts a lane
    if (wave == 0) {
        constexpr int PL = MOE_MAX_E / 64;
        int32_t v[PL], run = 0;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            v[i] = (s_tot[PL * lane + i] + MOE_ALIGN_ROWS - 1) / MOE_ALIGN_ROWS * MOE_ALIGN_ROWS;
            run += v[i];
        }
        int32_t at = run;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int32_t u = __shfl_up(at, o, 64);
            if (lane >= o) at += u;
        }
        at -= run;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            const int e = PL * lane + i;
            s_base[e] += at;
            if (c == 0 && e < E) {
                counts[e] = s_tot[e];
                offsets[e] = at;
                if (e == E - 1) offsets[E] = at + v[i];
            }
            at += v[i];
        }
    }
    __syncthreads();
    for (int e = tid; e < E; e += kScoresThreads) {
        int32_t run = s_base[e];
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const int32_t h = s_q[w][e];
            s_q[w][e] = run;
            run += h;
        }
    }
    __syncthreads();
    rank_pairs(topk_idx, q0, q1, nbits, s_q[wave], row_of, src_of);
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
// and 0 for every other expert. L lanes a token, one slot each; the slots' values go through an LDS row. DENSE:
// the softmax that is not renormalised, the one form that reads all logits. Bound by the latency of a slot's
// loads (expert, then its logit) and the write of dlogits: 131072 x 256, sigmoid, renormalised 31 to
// 36 us (3.8 to 4.3 TB/s); DENSE 46, reading as much again.
template <int L, int PER, bool DENSE>
__global__ void __launch_bounds__(256) route_scores_bwd_kernel(RouteBwdArgs p) {
    __shared__ __align__(16) float s_row[256 / L][L * PER];
    const int gl = lane_id() % L;
    const int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    const bool live = t < p.T;
    const int E = p.E;
    float* g = s_row[threadIdx.x / L];
    const float* row = p.logits + (live ? t : 0) * E;
    const bool whole = (E & 3) == 0 && (((uintptr_t)p.logits | (uintptr_t)p.dlogits) & 15) == 0;
    auto expert = [&](int i) { return 4 * (gl + L * (i >> 2)) + (i & 3); };
    // this lane's slot; none that is out of range or unavailable has a gradient
    int e = -1;
    float v = 0.f, d = 0.f;
    if (live && gl < p.k) {
        e = p.topk_idx[t * p.k + gl];
        d = p.ds[t * p.k + gl];
        if ((uint32_t)e >= (uint32_t)E) e = -1;
    }
    if (e >= 0) {
        v = row[e];
        if (!isfinite(v) || (p.bias && !isfinite(p.bias[e]))) e = -1;
    }
    if (e < 0) d = 0.f;  // also where ds is not finite: the slot's weight is 0 whatever its expert gave
    float x[DENSE ? PER : 1], mx = -INFINITY, inv = 0.f;
    if constexpr (DENSE) {
        if (!whole) {
            for (int q = gl; q < E; q += L) g[q] = row[q];
            wave_lds_sync();
        }
#pragma unroll
        for (int q = 0; q < PER / 4; ++q) {
            const int c = expert(4 * q);
            float4 f = make_float4(0, 0, 0, 0);
            if (c < E) f = whole ? *(const float4*)(row + c) : *(const float4*)(g + c);
            x[4 * q] = f.x, x[4 * q + 1] = f.y, x[4 * q + 2] = f.z, x[4 * q + 3] = f.w;
        }
        if (!whole) wave_lds_sync();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            x[i] = isfinite(x[i]) && expert(i) < E ? x[i] : -INFINITY;
            mx = fmaxf(mx, x[i]);
        }
        mx = lanes_max<L>(mx);
        const float shift = mx > -INFINITY ? mx : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            x[i] = __expf(x[i] - shift);
            sum += x[i];
        }
        sum = lanes_sum<L>(sum);
        inv = sum > 0.f ? 1.f / sum : 0.f;
    }
#pragma unroll
    for (int q = 0; q < PER / 4; ++q) *(float4*)(g + expert(4 * q)) = make_float4(0, 0, 0, 0);
    const float xs = p.renorm ? lanes_max<L>(e >= 0 ? v : -INFINITY) : 0.f;
    const SlotScore score{p.sigmoid != 0, p.renorm != 0, p.sigmoid ? fminf(xs, 0.f) : xs, mx, inv};
    float w = e >= 0 ? score(v) : 0.f;
    if (p.renorm) {  // divided, not times a reciprocal: a lone weight is 1 and has no gradient
        const float total = lanes_sum<L>(w);
        w = e >= 0 ? w / total : 0.f;
    }
    const float dot = lanes_sum<L>(w * d);
    wave_lds_sync();
    if (e >= 0)
        g[e] = DENSE ? d : p.scale * w * (p.sigmoid ? 1.f / (1.f + expf(v)) : 1.f) * (p.renorm ? d - dot : d);
    wave_lds_sync();
    if (!live) return;
    float* out = p.dlogits + t * E;
#pragma unroll
    for (int q = 0; q < PER / 4; ++q) {
        const int c = expert(4 * q);
        float4 f = *(const float4*)(g + c);
        if constexpr (DENSE) {
            f.x = p.scale * x[4 * q] * inv * (f.x - dot);
            f.y = p.scale * x[4 * q + 1] * inv * (f.y - dot);
            f.z = p.scale * x[4 * q + 2] * inv * (f.z - dot);
            f.w = p.scale * x[4 * q + 3] * inv * (f.w - dot);
            if (!whole) *(float4*)(g + c) = f;
        }
        if (whole && c < E) *(float4*)(out + c) = f;
    }
    if (!whole) {
        wave_lds_sync();
        for (int q = gl; q < E; q += L) out[q] = g[q];
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

// Tokens a workgroup: whole passes, at most kScoresGroups workgroups.
static int scores_chunk(int T, int k, int E) {
    const int tb = kScoresThreads / (E <= 256 && k <= 16 ? 16 : 64);
    const int64_t passes = ((int64_t)T + (int64_t)tb * kScoresGroups - 1) / ((int64_t)tb * kScoresGroups);
    return (int)(tb * passes);
}

size_t route_scores_workspace_bytes(int T, int k, int E) {
    const int ct = scores_chunk(T, k, E);
    return (size_t)(((int64_t)T + ct - 1) / ct) * E * sizeof(int32_t);
}

int launch_route_scores(const RouteCall& c, hipStream_t s) {
    RouteArgs p{};
    p.logits = c.logits, p.bias = c.bias, p.T = c.T, p.E = c.E, p.k = c.k;
    p.sigmoid = c.sigmoid, p.groups = c.groups, p.kept = c.kept, p.top = c.top, p.renorm = c.renorm, p.scale = c.scale;
    const uint32_t gs = (uint32_t)(c.E / c.groups);
    p.group_mul = ((1u << 22) + gs - 1) / gs;
    p.topk_idx = c.topk_idx, p.topk_w = c.topk_w, p.err_word = c.err_word;
    p.CT = scores_chunk(c.T, c.k, c.E);
    p.hist = (int32_t*)c.ws, p.src_of = c.src_of, p.M_cap = c.M_cap;
    const int nchunks = (int)(((int64_t)c.T + p.CT - 1) / p.CT);
    by_experts(c.E, c.k, [&](auto A, auto B) {
        constexpr int L = decltype(A)::value, PER = decltype(B)::value;
        auto go = [&](auto kern) { kern<<<nchunks, kScoresThreads, 0, s>>>(p); };
        if (p.sigmoid) p.bias ? go(route_scores_kernel<L, PER, true, true>) : go(route_scores_kernel<L, PER, true, false>);
        else p.bias ? go(route_scores_kernel<L, PER, false, true>) : go(route_scores_kernel<L, PER, false, false>);
    });
    int nbits = 0;
    while ((1 << nbits) < c.E) ++nbits;
    scores_layout_kernel<<<nchunks, kScoresThreads, 0, s>>>(c.topk_idx, c.T, c.k, c.E, nbits, p.CT, nchunks, p.hist,
                                                            c.counts, c.offsets, c.row_of, c.src_of);
    return hipGetLastError() == hipSuccess ? 0 : -4;
}

int launch_route_scores_bwd(const float* logits, const float* bias, const int32_t* topk_idx, const float* ds, int T,
                            int E, int k, int sigmoid, int renorm, float scale, float* dlogits, hipStream_t s) {
    by_experts(E, k, [&](auto A, auto B) {
        constexpr int L = decltype(A)::value, PER = decltype(B)::value, TB = 256 / L;  // tokens a workgroup
        // 2^22 workgroups a launch: one of 2^32 threads and more would be cut off without an error
        const int64_t step = ((int64_t)1 << 22) * TB;
        for (int64_t t = 0; t < T; t += step) {
            const int n = (int)std::min(step, T - t);
            const RouteBwdArgs p{logits + t * E, bias, topk_idx + t * k, ds + t * k, n, E, k, sigmoid, renorm, scale, dlogits + t * E};
            const unsigned grid = (unsigned)((n + TB - 1) / TB);
            if (!sigmoid && !renorm) route_scores_bwd_kernel<L, PER, true><<<grid, 256, 0, s>>>(p);
            else route_scores_bwd_kernel<L, PER, false><<<grid, 256, 0, s>>>(p);
        }
    });
    return hipGetLastError() == hipSuccess ? 0 : -4;
}

}  // namespace moe
