// Router losses: the load-balance loss and the z loss of softmax routing, per
// sequence, with their gradient.
//
//   p = softmax(logits[t]); over the n_s live tokens of sequence s:
//   f_se = E c_se / (k n_s), c_se pairs routed to expert e; P_se = mean of p_e
//   B = mean over sequences with a live token of sum_e f_se P_se
//   Z = mean over all live tokens of (log sum_e exp(logits[t, e]))^2
//   loss = cb B + cz Z, f held constant in the gradient (counts have none):
//   dloss/dlogits[t, e] = cb / (S' n_s) p_e (f_se - sum_j f_sj p_j) + cz 2 lse / n p_e
//
// The forward cuts the tokens into chunks; a chunk walks the sequences it holds
// and leaves one row of partial sums (probabilities, counts, live tokens, lse^2)
// per (chunk, sequence) pair. Chunk c and sequence s use row c + s: walking the
// tokens, either c or s grows at each step, so rows are distinct and fewer than
// chunks + S. Sums are joined in a fixed order (no floating-point atomics): the
// same inputs give the same bits.
//
// Both directions are bound by HBM: the logits are read once (131072 x 256 in 64
// sequences: 33 us, 4.1 TB/s, near the rate of a kernel that only loads them, then 11 us
// of two small launches to join), and the gradient reads one matrix and writes one
// (58 us, 4.6 TB/s).
#include <algorithm>

#include "dense_common.hpp"

namespace moe {

struct BalanceArgs {
    const float* logits;
    const int32_t* topk_idx;
    const uint8_t* valid;
    const int32_t* seq;  // [S + 1] or nullptr: one sequence of all T tokens
    int T, E, k, S;
    int CT;  // tokens per chunk
    float* rows;  // [nchunks + S][2 E + 2]: probabilities, counts, live tokens, lse^2
    float* bal;   // [S][etiles] partial sums of f P
    float* zs;    // [S] lse^2
    float cb, cz;
    float* loss;
    int32_t* counts;
    float* prob;
    int32_t* tokens;
    int etiles;
    int alone;  // one workgroup does it all
    // backward
    const float* grad;
    int accumulate;
    float* dlogits;
    uint16_t* dlogits16;
    int stream;  // dlogits past the caches
};

// first and past-the-end token of sequence s, kept inside [0, T]
__device__ __forceinline__ int seq_at(const BalanceArgs& p, int s) {
    if (!p.seq) return s == 0 ? 0 : p.T;
    const int v = p.seq[s];
    return v < 0 ? 0 : v > p.T ? p.T : v;
}

// Calls f(s, a, b) for every run [a, b) of tokens of one sequence inside
// [t0, t1); s = -1 for tokens before the first or behind the last sequence.
template <class F>
__device__ __forceinline__ void for_sequences(const BalanceArgs& p, int t0, int t1, F&& f) {
    int lo = -1, hi = p.S;  // largest s with seq_at(s) <= t0
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq_at(p, mid) <= t0) lo = mid;
        else hi = mid;
    }
    int t = t0;
    for (int s = lo; t < t1; ++s) {
        const int e = s >= p.S ? t1 : min(t1, seq_at(p, s + 1));
        if (e > t) {
            f(s >= p.S ? -1 : s, t, e);
            t = e;
        }
    }
}

// Reductions over a token's group of G lanes (every lane gets the result): DPP
// quad permutes and row mirrors inside 16 lanes, lane exchanges beyond.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}
template <int G, class Op>
__device__ __forceinline__ float group_reduce(float v, Op op) {
    if constexpr (G >= 2) v = op(v, dpp<0xB1>(v));    // lane ^ 1
    if constexpr (G >= 4) v = op(v, dpp<0x4E>(v));    // lane ^ 2
    if constexpr (G >= 8) v = op(v, dpp<0x141>(v));   // the other quad of 8 lanes
    if constexpr (G >= 16) v = op(v, dpp<0x140>(v));  // the other half of 16 lanes
    if constexpr (G >= 32) v = op(v, __shfl_xor(v, 16, 64));
    if constexpr (G >= 64) v = op(v, __shfl_xor(v, 32, 64));
    return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
    return group_reduce<G>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
    return group_reduce<G>(v, [](float a, float b) { return a + b; });
}

// Expert of element i of lane gl: four neighbours a lane when rows are whole
// 16-byte pieces (V4), else one.
template <int G, bool V4>
__device__ __forceinline__ int expert_of(int gl, int i) {
    return V4 ? (i >> 2) * 4 * G + 4 * gl + (i & 3) : gl + G * i;
}

// One token's logits, PER a lane; experts past E and tokens past the run (on ==
// false) are -inf.
template <int G, int PER, bool V4>
__device__ __forceinline__ void token_load(const BalanceArgs& p, int t, int gl, bool on, float (&x)[PER]) {
    const float* row = p.logits + (int64_t)t * p.E;
    if constexpr (V4) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
            const int e = expert_of<G, true>(gl, i);
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (on && e < p.E) v = *(const float4*)(row + e);
            x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = expert_of<G, false>(gl, i);
            x[i] = on && e < p.E ? row[e] : -INFINITY;
        }
    }
}

// x becomes exp(x - max); returns whether the token has a finite logit. Non-finite
// logits, and all of a token that is not valid, count as -inf (probability 0), as in
// the router. (`valid` only comes in here: the loads do not wait for it.) The hardware exponential's argument x log2(e) is rounded once: 2^-24 |x| relative.
template <int G, int PER>
__device__ __forceinline__ bool token_softmax(float (&x)[PER], bool valid, float& inv, float& lse) {
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (!valid || !isfinite(x[i])) x[i] = -INFINITY;
        mx = fmaxf(mx, x[i]);
    }
    mx = group_max<G>(mx);
    const bool some = mx > -INFINITY;
    const float ref = some ? mx : 0.f;  // exp(-inf - 0) = 0
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        x[i] = __expf(x[i] - ref);
        s += x[i];
    }
    s = group_sum<G>(s);
    inv = some ? 1.f / s : 0.f;
    lse = some ? mx + logf(s) : 0.f;
    return some;
}

// Joins the chunks' rows of sequence s for experts [32 et, 32 et + 32); all 256
// threads of a workgroup, also one after another for several (s, et).
__device__ __forceinline__ void balance_join(const BalanceArgs& p, int s, int et) {
    __shared__ float s_p[8][33], s_z[4];
    __shared__ int s_c[8][33], s_n[4];
    const int tid = threadIdx.x, el = tid & 31, l = tid >> 5;
    const int e = et * 32 + el;
    const int a = seq_at(p, s), b = seq_at(p, s + 1);
    const int c0 = a / p.CT, c1 = b > a ? (b - 1) / p.CT + 1 : c0;
    const int64_t w = 2 * p.E + 2;
    float pe = 0.f, z = 0.f;
    int ce = 0, n = 0;
#pragma unroll 4
    for (int c = c0 + l; c < (e < p.E ? c1 : c0); c += 8) {
        const float* row = p.rows + (c + s) * w;
        pe += row[e];
        ce += ((const int32_t*)row)[p.E + e];
    }
    for (int c = c0 + tid; c < c1; c += 256) {
        const float* row = p.rows + (c + s) * w;
        n += ((const int32_t*)row)[2 * p.E];
        z += row[2 * p.E + 1];
    }
    s_p[l][el] = pe;
    s_c[l][el] = ce;
    z = wave_sum(z);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, 64);
    if ((tid & 63) == 0) {
        s_n[tid >> 6] = n;
        s_z[tid >> 6] = z;
    }
    __syncthreads();
    n = s_n[0] + s_n[1] + s_n[2] + s_n[3];
    if (tid < 64) {
        float v = 0.f;
        if (tid < 32 && e < p.E) {
            float sum = 0.f;
            int cnt = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                sum += s_p[q][el];
                cnt += s_c[q][el];
            }
            const float mean = n > 0 ? sum / (float)n : 0.f;
            p.counts[(int64_t)s * p.E + e] = cnt;
            p.prob[(int64_t)s * p.E + e] = mean;
            v = n > 0 ? (float)cnt * ((float)p.E / ((float)p.k * (float)n)) * mean : 0.f;
        }
        v = wave_sum(v);
        if (tid == 0) {
            p.bal[(int64_t)s * p.etiles + et] = v;
            if (et == 0) {
                p.tokens[s] = n;
                p.zs[s] = (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]);
            }
        }
    }
    __syncthreads();
}

// The losses from the joined sums (one workgroup of 256 threads).
__device__ __forceinline__ void balance_total(const BalanceArgs& p) {
    __shared__ double s_b[4], s_z[4];
    __shared__ int s_n[4], s_live[4];
    const int tid = threadIdx.x;
    double b = 0.0, z = 0.0;
    int n = 0, live = 0;
    for (int64_t i = tid; i < (int64_t)p.S * p.etiles; i += 256) b += p.bal[i];
    for (int s = tid; s < p.S; s += 256) {
        z += p.zs[s];
        const int m = p.tokens[s];
        n += m;
        live += m > 0;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        b += __shfl_xor(b, o, 64);
        z += __shfl_xor(z, o, 64);
        n += __shfl_xor(n, o, 64);
        live += __shfl_xor(live, o, 64);
    }
    if ((tid & 63) == 0) s_b[tid >> 6] = b, s_z[tid >> 6] = z, s_n[tid >> 6] = n, s_live[tid >> 6] = live;
    __syncthreads();
    if (tid == 0) {
        b = (s_b[0] + s_b[1]) + (s_b[2] + s_b[3]);
        z = (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]);
        n = s_n[0] + s_n[1] + s_n[2] + s_n[3];
        live = s_live[0] + s_live[1] + s_live[2] + s_live[3];
        const double bal = live ? b / live : 0.0, zl = n ? z / n : 0.0;
        // a term that is switched off stays out, also where it is infinite (logits of
        // 1e20 and more, such as a mask's lowest value in all of a row)
        p.loss[0] = (float)((p.cb != 0.f ? p.cb * bal : 0.0) + (p.cz != 0.f ? p.cz * zl : 0.0));
        p.loss[1] = (float)bal;
        p.loss[2] = (float)zl;
        p.tokens[p.S] = live;
        p.tokens[p.S + 1] = n;
    }
}

// At most kJoinBlocks workgroups: a launch of 2^32 threads and more is cut off without an error.
constexpr int64_t kJoinBlocks = 1 << 20;
__global__ void __launch_bounds__(256) balance_join_kernel(BalanceArgs p) {
    for (int64_t i = blockIdx.x; i < (int64_t)p.S * p.etiles; i += gridDim.x) {
        const int s = (int)i / p.etiles;
        balance_join(p, s, (int)i - s * p.etiles);
    }
}
__global__ void __launch_bounds__(256) balance_total_kernel(BalanceArgs p) { balance_total(p); }

// A group of G lanes per token, PER logits a lane. One workgroup alone (small inputs) goes on to join and finish.
template <int G, int PER, bool V4>
__global__ void __launch_bounds__(256) balance_chunk_kernel(BalanceArgs p) {
    __shared__ float s_p[4][G * PER];
    __shared__ int s_cnt[G * PER];
    __shared__ float s_z[4];
    __shared__ int s_n[4];
    constexpr int NG = 256 / G;  // tokens at a time
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int gl = lane % G, grp = tid / G;
    for (int e = tid; e < G * PER; e += 256) s_cnt[e] = 0;
    __syncthreads();
    const int c = blockIdx.x;
    const int t0 = c * p.CT, t1 = min(p.T, t0 + p.CT);
    for_sequences(p, t0, t1, [&](int s, int a, int b) {
        if (s < 0) return;
        float acc[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) acc[i] = 0.f;
        float z = 0.f;
        int n = 0;
        auto take = [&](int t, bool valid, int first, float (&x)[PER]) {
            float inv, lse;
            const bool some = token_softmax<G, PER>(x, valid, inv, lse);
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] += x[i] * inv;
            if (some) {
                if (gl == 0) {
                    z += lse * lse;
                    ++n;
                }
                if (first >= 0 && first < p.E) atomicAdd(&s_cnt[first], 1);
                for (int j = gl + G; j < p.k; j += G) {
                    const int e = p.topk_idx[(int64_t)t * p.k + j];
                    if (e >= 0 && e < p.E) atomicAdd(&s_cnt[e], 1);
                }
            }
        };
        // the loads of a group's next token are on their way while one is worked on
        struct Token {
            float x[PER];
            int first;
            bool valid;
        } u, v;
        auto fetch = [&](int t, Token& k) {
            const bool on = t < b;
            token_load<G, PER, V4>(p, on ? t : a, gl, on, k.x);
            k.first = on && gl < p.k ? p.topk_idx[(int64_t)t * p.k + gl] : -1;
            k.valid = !p.valid || (on && p.valid[t] != 0);
        };
        fetch(a + grp, u);
        for (int t = a + grp; t - grp < b; t += 2 * NG) {
            fetch(t + NG, v);
            take(t, u.valid, u.first, u.x);
            fetch(t + 2 * NG, u);
            take(t + NG, v.valid, v.first, v.x);
        }
        // over the wavefront's groups, then its 4 wavefronts
#pragma unroll
        for (int o = 32; o >= G; o >>= 1) {
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] += __shfl_xor(acc[i], o, 64);
            z += __shfl_xor(z, o, 64);
            n += __shfl_xor(n, o, 64);
        }
        if (lane < G) {
#pragma unroll
            for (int i = 0; i < PER; ++i) s_p[wave][expert_of<G, V4>(gl, i)] = acc[i];
        }
        if (lane == 0) {
            s_z[wave] = z;
            s_n[wave] = n;
        }
        __syncthreads();
        float* row = p.rows + (int64_t)(c + s) * (2 * p.E + 2);
        for (int e = tid; e < p.E; e += 256) {
            row[e] = (s_p[0][e] + s_p[1][e]) + (s_p[2][e] + s_p[3][e]);
            ((int32_t*)row)[p.E + e] = s_cnt[e];
            s_cnt[e] = 0;
        }
        if (tid == 0) {
            ((int32_t*)row)[2 * p.E] = s_n[0] + s_n[1] + s_n[2] + s_n[3];
            row[2 * p.E + 1] = (s_z[0] + s_z[1]) + (s_z[2] + s_z[3]);
        }
        __syncthreads();
    });
    if (p.alone) {
        for (int i = 0; i < p.S * p.etiles; ++i) balance_join(p, i / p.etiles, i % p.etiles);
        balance_total(p);
    }
}

// The gradient, one group of G lanes per token. f enters less its value at the
// largest logit: the gradient does not change (sum_e p_e = 1), and where one
// expert holds nearly all the probability, f_e - sum_j f_j p_j no longer cancels.
template <int G, int PER, bool V4>
__global__ void __launch_bounds__(256) balance_bwd_kernel(BalanceArgs p) {
    constexpr int NG = 256 / G;
    const int tid = threadIdx.x, lane = tid & 63;
    const int gl = lane % G, grp = tid / G;
    const int t0 = blockIdx.x * p.CT, t1 = min(p.T, t0 + p.CT);
    const float up = p.grad ? p.grad[0] : 1.f;
    const int live = p.tokens[p.S], ntot = p.tokens[p.S + 1];
    const float zc = ntot > 0 ? up * p.cz * 2.f / (float)ntot : 0.f;
    for_sequences(p, t0, t1, [&](int s, int a, int b) {
        const int n = s >= 0 ? p.tokens[s] : 0;
        const float fs = n > 0 ? (float)p.E / ((float)p.k * (float)n) : 0.f;
        const float bc = n > 0 ? up * p.cb / ((float)live * (float)n) : 0.f;
        float f[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = expert_of<G, V4>(gl, i);
            f[i] = s >= 0 && e < p.E ? (float)p.counts[(int64_t)s * p.E + e] * fs : 0.f;
        }
        auto give = [&](int t, bool valid, float (&x)[PER]) {
            float inv, lse;
            token_softmax<G, PER>(x, valid, inv, lse);
            float ref = -INFINITY;  // x = exp(logit - max) is 1 at the largest logit
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (x[i] == 1.f) ref = fmaxf(ref, f[i]);
            ref = group_max<G>(ref);
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                x[i] *= inv;
                if (x[i] > 0.f) dot += x[i] * (f[i] - ref);
            }
            dot = group_sum<G>(dot);
            const float zl = zc * lse;
#pragma unroll
            for (int i = 0; i < PER; ++i) x[i] = x[i] > 0.f ? x[i] * (bc * ((f[i] - ref) - dot) + zl) : 0.f;
            if (t >= b) return;
            if constexpr (V4) {
#pragma unroll
                for (int i = 0; i < PER; i += 4) {
                    const int e = expert_of<G, true>(gl, i);
                    if (e < p.E) {
                        const int64_t at = (int64_t)t * p.E + e;
                        float4 d = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                        if (p.accumulate) {
                            const float4 o = *(const float4*)(p.dlogits + at);
                            d.x += o.x, d.y += o.y, d.z += o.z, d.w += o.w;
                        }
                        if (p.stream) st_nt16(p.dlogits + at, d);
                        else *(float4*)(p.dlogits + at) = d;
                        if (p.dlogits16)
                            *(uint2*)(p.dlogits16 + at) = make_uint2(pack_bf16x2(d.x, d.y), pack_bf16x2(d.z, d.w));
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int e = expert_of<G, false>(gl, i);
                    if (e < p.E) {
                        const int64_t at = (int64_t)t * p.E + e;
                        const float d = p.accumulate ? x[i] + p.dlogits[at] : x[i];
                        p.dlogits[at] = d;
                        if (p.dlogits16) p.dlogits16[at] = (uint16_t)f32_to_bf16(d);
                    }
                }
            }
        };
        float u[PER], v[PER];
        bool uv, vv;
        auto fetch = [&](int t, float (&x)[PER], bool& valid) {
            const bool on = s >= 0 && t < b;
            token_load<G, PER, V4>(p, on ? t : a, gl, on, x);
            valid = !p.valid || (on && p.valid[t] != 0);
        };
        fetch(a + grp, u, uv);
        for (int t = a + grp; t - grp < b; t += 2 * NG) {
            fetch(t + NG, v, vv);
            give(t, uv, u);
            fetch(t + 2 * NG, u, uv);
            give(t + NG, vv, v);
        }
    });
}

// Lanes per token and logits per lane: up to 16 logits a lane, so that a wavefront
// works on several tokens at once and a reduction over a token takes few exchanges
// (E = 256: 16 lanes, 4 tokens a wavefront; with 64 lanes a token 79 us instead).
struct BalanceShape {
    int G, PER;
};
static BalanceShape balance_shape(int E) {
    if (E <= 16) return {4, 4};
    if (E <= 32) return {8, 4};
    if (E <= 64) return {16, 4};
    if (E <= 128) return {16, 8};
    if (E <= 256) return {16, 16};
    if (E <= 512) return {32, 16};
    return {64, MOE_MAX_E / 64};
}

// Tokens per chunk: about `most` workgroups of whole steps, but no more than a sequence's
// mean length, since a workgroup walks the sequences of its chunk one after the other
// (forward, backward of 128 x 64 in 64 sequences 9.5, 4.6 us; 91.3, 29.1 in one chunk).
static int balance_chunk(int T, int E, int S, int most) {
    const int step = 2 * 256 / balance_shape(E).G;
    const int ct = (T + most - 1) / most;
    return std::max(ct, std::min((ct + step - 1) / step * step, (T + S - 1) / S));
}

// The forward's: all tokens of one sequence where one workgroup passes over them in two
// steps: it joins and finishes, no further launch (256 x 8 7.2 us, 8.5 with three launches;
// 128 x 64, four steps, 10.2 alone, 8.8 with three).
static int balance_chunk(int T, int E, int S) {
    const int few = 4 * 256 / balance_shape(E).G;
    return S == 1 && T <= few ? few : balance_chunk(T, E, S, 1024);
}

static int balance_etiles(int E) { return (E + 31) / 32; }

size_t balance_workspace_bytes(int T, int E, int S) {
    const int ct = balance_chunk(T, E, S);
    const int64_t rows = ((int64_t)T + ct - 1) / ct + S;
    return (size_t)(rows * (2 * E + 2) + (int64_t)S * balance_etiles(E) + S) * sizeof(float);
}

template <bool V4, class F>
static void by_shape(int E, F&& f) {
    using std::integral_constant;
    const BalanceShape h = balance_shape(E);
    const std::bool_constant<V4> v{};
    if (h.G == 4) f(integral_constant<int, 4>{}, integral_constant<int, 4>{}, v);
    else if (h.G == 8) f(integral_constant<int, 8>{}, integral_constant<int, 4>{}, v);
    else if (h.G == 16 && h.PER == 4) f(integral_constant<int, 16>{}, integral_constant<int, 4>{}, v);
    else if (h.G == 16 && h.PER == 8) f(integral_constant<int, 16>{}, integral_constant<int, 8>{}, v);
    else if (h.G == 16) f(integral_constant<int, 16>{}, integral_constant<int, 16>{}, v);
    else if (h.G == 32) f(integral_constant<int, 32>{}, integral_constant<int, 16>{}, v);
    else f(integral_constant<int, 64>{}, integral_constant<int, 16>{}, v);
}

// Rows are read as 16-byte pieces when every row starts on one.
template <class F>
static void by_experts(int E, bool aligned, F&& f) {
    if (E % 4 == 0 && aligned) by_shape<true>(E, f);
    else by_shape<false>(E, f);
}

static bool on16(const void* p) { return ((uintptr_t)p & 15) == 0; }

int launch_balance_loss(const float* logits, const int32_t* topk_idx, const uint8_t* valid, const int32_t* seq,
                        int T, int E, int k, int S, float cb, float cz, float* loss, int32_t* counts,
                        float* prob, int32_t* tokens, void* ws, hipStream_t s) {
    BalanceArgs p{};
    p.logits = logits, p.topk_idx = topk_idx, p.valid = valid, p.seq = seq, p.T = T, p.E = E, p.k = k, p.S = S;
    p.CT = balance_chunk(T, E, S);
    const int nchunks = (T + p.CT - 1) / p.CT;
    p.etiles = balance_etiles(E);
    // one after the other, the joins of 32 experts each cost more than two launches from four
    // on (60 tokens: E = 64 8.2 us alone, 9.5 with three launches; E = 128 11.4, 10.0)
    p.alone = nchunks == 1 && p.etiles <= 2;
    p.rows = (float*)ws;
    p.bal = p.rows + (int64_t)(nchunks + S) * (2 * E + 2);
    p.zs = p.bal + (int64_t)S * p.etiles;
    p.cb = cb, p.cz = cz, p.loss = loss, p.counts = counts, p.prob = prob, p.tokens = tokens;
    by_experts(E, on16(logits), [&](auto G, auto PER, auto V4) {
        balance_chunk_kernel<decltype(G)::value, decltype(PER)::value, decltype(V4)::value><<<nchunks, 256, 0, s>>>(p);
    });
    if (!p.alone) {
        balance_join_kernel<<<(unsigned)std::min((int64_t)p.etiles * S, kJoinBlocks), 256, 0, s>>>(p);
        balance_total_kernel<<<1, 256, 0, s>>>(p);
    }
    return hipGetLastError() == hipSuccess ? 0 : -4;
}

int launch_balance_loss_bwd(const float* logits, const int32_t* counts, const int32_t* tokens,
                            const uint8_t* valid, const int32_t* seq, int T, int E, int k, int S, float cb,
                            float cz, const float* grad, int accumulate, float* dlogits, uint16_t* dlogits16,
                            hipStream_t s) {
    BalanceArgs p{};
    p.logits = logits, p.valid = valid, p.seq = seq, p.T = T, p.E = E, p.k = k, p.S = S;
    p.CT = balance_chunk(T, E, S, 2048);
    p.counts = const_cast<int32_t*>(counts), p.tokens = const_cast<int32_t*>(tokens);
    p.cb = cb, p.cz = cz, p.grad = grad, p.accumulate = accumulate, p.dlogits = dlogits, p.dlogits16 = dlogits16;
    p.stream = (int64_t)T * E * 4 >= kDenseStreamBytes;
    const int nchunks = (T + p.CT - 1) / p.CT;
    by_experts(E, on16(logits) && on16(dlogits) && ((uintptr_t)dlogits16 & 7) == 0, [&](auto G, auto PER, auto V4) {
        balance_bwd_kernel<decltype(G)::value, decltype(PER)::value, decltype(V4)::value><<<nchunks, 256, 0, s>>>(p);
    });
    return hipGetLastError() == hipSuccess ? 0 : -4;
}

}  // namespace moe
