// The norms before and after a MoE block (gfx950).
//
//   before: s = x + r (rounded to bf16: what the residual stream holds), y = s rho w,
//           rho = 1 / sqrt(mean(s^2) + eps)
//   after:  v = sum_j w_j Y[row_j] (rounded to bf16, as moe_combine), out = x + scale gate (v rho w)
//   back through a norm y = s rho w, with h = s rho and g = dy w:
//           ds = rho (g - h mean(g h)),  dw = sum over rows of dy h
//
// All are bound by HBM traffic: a row stays in registers between its statistics and its
// output, so every tensor is read once and written once. 32768 x 8192 with the residual: forward 366 us (5.9
// TB/s), backward 420 (5.1); 16384 x 7168 of 8 experts with a full gate: forward 558 (5.0), backward 228 (5.1). A large
// copy reaches 5.0 to 5.1. Past 8192 columns a thread of a gradient holds eight pieces of a row and their sums, so that two
// wavefronts (one behind the block) fit a SIMD and its loads are exposed: 16384 x 16384 forward 400 (5.4) and 373 (5.7),
// backward 617 (3.5) and 792 (3.4).
#include <algorithm>

#include "block_common.hpp"

namespace moe {

// TPR threads hold a row, NC chunks of 8 values each; a workgroup of 256 holds 256 / TPR rows.
constexpr int kNormThreads = 256;

// Sum over a row's TPR threads, the same in all of them. `part` is LDS of the workgroup that no
// wavefront still reads: callers in a loop alternate two.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
    v = lanes_sum<64>(v);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = (part[0] + part[1]) + (part[2] + part[3]);
    }
    return v;
}

// sigmoid(v) and its derivative, e / (1 + e)^2 with e = exp(-|v|): no cancellation far from zero. The hardware's
// reciprocal is good to one unit of fp32; a division by the rounding rules takes ten instructions, and with two a
// value a full gate's backward pass was bound by arithmetic (16384 x 7168: 359 us, so 290).
struct Sigmoid {
    float value, slope;
};
__device__ __forceinline__ Sigmoid sigmoid_of(float v) {
    const float e = __expf(-fabsf(v)), q = __builtin_amdgcn_rcpf(1.f + e);
    return {v < 0.f ? e * q : q, e * q * q};
}

template <int TPR, int NC>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_kernel(NormFwd p) {
    __shared__ float s_part[4];
    const int tid = threadIdx.x % TPR;
    const int64_t t = (int64_t)blockIdx.x * (kNormThreads / TPR) + threadIdx.x / TPR;
    const int cpr = p.d / 8;
    const bool live = t < p.T;
    const int64_t row = t * cpr;
    uint4 v[NC];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = tid + TPR * i;
        v[i] = make_uint4(0, 0, 0, 0);
        if (live && c < cpr) {
            v[i] = ((const uint4*)p.x)[row + c];
            if (p.res) {
                float a[8], b[8];
                unpack8(v[i], a);
                unpack8(((const uint4*)p.res)[row + c], b);
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] += b[j];
                v[i] = pack8(a);
            }
            if (p.total) ((uint4*)p.total)[row + c] = v[i];
        }
        float a[8];
        unpack8(v[i], a);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(a[j], a[j], ss);
    }
    const float r = rsqrtf(row_sum<TPR>(ss, s_part) / (float)p.d + p.eps);
    if (live && tid == 0 && p.rstd) p.rstd[t] = r;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = tid + TPR * i;
        if (live && c < cpr) {
            float a[8], w[8];
            unpack8(v[i], a);
            unpack8(((const uint4*)p.w)[c], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = a[j] * r * w[j];
            ((uint4*)p.y)[row + c] = pack8(a);
        }
    }
}

// A workgroup walks rows and keeps its column sums of dw in registers; part: [parts, d], joined by norm_join_kernel
// (11 us for 1024 parts).
template <int TPR, int NC>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_kernel(NormBwd p, float* part) {
    __shared__ float s_part[2][4];
    const int tid = threadIdx.x % TPR;
    constexpr int RPB = kNormThreads / TPR;
    const int64_t me = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR, n = (int64_t)gridDim.x * RPB;
    const int cpr = p.d / 8;
    float dw[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    int turn = 0;
    // every row group of a workgroup takes as many turns (the sums below may hold a barrier)
    for (int64_t t0 = (int64_t)blockIdx.x * RPB; t0 < p.T; t0 += n, turn ^= 1) {
        const int64_t t = t0 + threadIdx.x / TPR;
        const bool live = t < p.T;
        const int64_t row = t * cpr;
        const float r = live ? p.rstd[t] : 0.f;
        uint4 x[NC], dy[NC];
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = tid + TPR * i;
            if (live && c < cpr) {
                x[i] = ((const uint4*)p.x)[row + c];
                dy[i] = ((const uint4*)p.dy)[row + c];
                float a[8], b[8], w[8];
                unpack8(x[i], a);
                unpack8(dy[i], b);
                unpack8(((const uint4*)p.w)[c], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float bh = b[j] * (a[j] * r);
                    dw[i][j] += bh;
                    m = fmaf(bh, w[j], m);
                }
            }
        }
        const float mean = row_sum<TPR>(m, s_part[turn]) / (float)p.d;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = tid + TPR * i;
            if (live && c < cpr) {
                float a[8], b[8], w[8];
                unpack8(x[i], a);
                unpack8(dy[i], b);
                unpack8(((const uint4*)p.w)[c], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] = r * (b[j] * w[j] - a[j] * r * mean);
                if (p.dres) {
                    unpack8(((const uint4*)p.dres)[row + c], b);
#pragma unroll
                    for (int j = 0; j < 8; ++j) a[j] += b[j];
                }
                ((uint4*)p.dx)[row + c] = pack8(a);
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = tid + TPR * i;
        if (c < cpr) {
            float* o = part + me * p.d + 8 * c;
            *(float4*)o = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            *(float4*)(o + 4) = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
}

template <int TPR, int NC>
__global__ void __launch_bounds__(kNormThreads) post_norm_fwd_kernel(PostNormFwd p) {
    __shared__ float s_part[4];
    const int tid = threadIdx.x % TPR;
    const int64_t t = (int64_t)blockIdx.x * (kNormThreads / TPR) + threadIdx.x / TPR;
    const int cpr = p.d / 8;
    const bool live = t < p.T;
    const int64_t row = t * cpr;
    uint4 v[NC];
    float ss = 0.f;
    if (!p.row_of) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = tid + TPR * i;
            v[i] = live && c < cpr ? ((const uint4*)p.y)[row + c] : make_uint4(0, 0, 0, 0);
        }
    } else {
        // the sum over the token's experts in ascending order, as moe_combine takes it
        float acc[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
        for (int q = 0; live && q < p.k; ++q) {
            const int64_t src = (int64_t)p.row_of[t * p.k + q] * cpr;
            const float wq = p.topk_w ? p.topk_w[t * p.k + q] : 1.f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = tid + TPR * i;
                if (c < cpr) {
                    float f[8];
                    unpack8(((const uint4*)p.y)[src + c], f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(wq, f[j], acc[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = tid + TPR * i;
            v[i] = pack8(acc[i]);
            if (p.total && live && c < cpr) ((uint4*)p.total)[row + c] = v[i];
        }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        float a[8];
        unpack8(v[i], a);
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(a[j], a[j], ss);
    }
    const float r = rsqrtf(row_sum<TPR>(ss, s_part) / (float)p.d + p.eps);
    if (!live) return;
    if (tid == 0 && p.rstd) p.rstd[t] = r;
    float g1 = 1.f;
    if (p.gate && p.gate_cols == 1) {
        g1 = bf16_to_f32(p.gate[t]);
        if (p.sigmoid) g1 = sigmoid_of(g1).value;
    }
    g1 *= p.scale;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = tid + TPR * i;
        if (c < cpr) {
            float a[8], w[8], x[8];
            unpack8(v[i], a);
            unpack8(((const uint4*)p.w)[c], w);
            unpack8(((const uint4*)p.x)[row + c], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = a[j] * r * w[j] * g1;
            if (p.gate_cols > 1) {
                float g[8];
                unpack8(((const uint4*)p.gate)[row + c], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] *= p.sigmoid ? sigmoid_of(g[j]).value : g[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] += x[j];
            ((uint4*)p.out)[row + c] = pack8(a);
        }
    }
}

// Through out = x + scale gate(c) (y rho w); the gradient of x is dout itself. A row's loads are all on their way before
// the first is used, at two wavefronts a SIMD (16384 x 7168 with a full gate: 229 us, 5.1 TB/s; 290 with loads and
// arithmetic mixed at three. norm_bwd_kernel, with less to hold, is better mixed, at four: 428 against 518 us).
template <int TPR, int NC>
__global__ void __launch_bounds__(kNormThreads) post_norm_bwd_kernel(PostNormBwd p, float* part) {
    __shared__ float s_part[2][4];
    const int tid = threadIdx.x % TPR;
    constexpr int RPB = kNormThreads / TPR;
    const int64_t me = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR, n = (int64_t)gridDim.x * RPB;
    const int cpr = p.d / 8;
    float dw[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * RPB; t0 < p.T; t0 += n, turn ^= 1) {
        const int64_t t = t0 + threadIdx.x / TPR;
        const bool live = t < p.T;
        const int64_t row = t * cpr;
        const float r = live ? p.rstd[t] : 0.f;
        float g1 = 1.f, slope = 1.f;  // a token's gate and its derivative
        if (p.gate_cols == 1 && live) {
            g1 = bf16_to_f32(p.gate[t]);
            if (p.sigmoid) {
                const Sigmoid s = sigmoid_of(g1);
                g1 = s.value, slope = s.slope;
            }
        }
        uint4 y[NC], dv[NC], gt[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {  // all on their way before the first is used
            const int c = tid + TPR * i;
            if (live && c < cpr) {
                y[i] = ((const uint4*)p.y)[row + c];
                dv[i] = ((const uint4*)p.dout)[row + c];
                if (p.gate_cols > 1) gt[i] = ((const uint4*)p.gate)[row + c];
            }
        }
        float u[NC][8];  // the gradient of h: scale dout w, times the gate where there is one a channel
        float m = 0.f;   // sum of u h
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = tid + TPR * i;
            if (live && c < cpr) {
                float a[8], b[8], w[8];
                unpack8(y[i], a);
                unpack8(dv[i], b);
                unpack8(((const uint4*)p.w)[c], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    a[j] *= r;
                    b[j] *= p.scale;
                }
                if (p.gate_cols > 1) {
                    float g[8], dg[8];
                    unpack8(gt[i], g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        Sigmoid s = {g[j], 1.f};
                        if (p.sigmoid) s = sigmoid_of(g[j]);
                        dg[j] = b[j] * a[j] * w[j] * s.slope;
                        b[j] *= s.value;
                    }
                    if (p.dgate) ((uint4*)p.dgate)[row + c] = pack8(dg);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dw[i][j] = fmaf(b[j] * a[j], g1, dw[i][j]);
                    u[i][j] = b[j] * w[j];
                    m = fmaf(u[i][j], a[j], m);
                }
            }
        }
        m = row_sum<TPR>(m, s_part[turn]);
        if (p.gate_cols == 1 && p.dgate && live && tid == 0) ((float*)p.dgate)[t] = m * slope;
        const float mean = m * g1 * r / (float)p.d;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = tid + TPR * i;
            if (live && c < cpr) {
                float a[8];
                unpack8(y[i], a);
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] = r * (u[i][j] * g1 - a[j] * mean);
                ((uint4*)p.dy)[row + c] = pack8(a);
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = tid + TPR * i;
        if (c < cpr) {
            float* o = part + me * p.d + 8 * c;
            *(float4*)o = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            *(float4*)(o + 4) = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
}

// dw[c] = sum of the parts' column sums, in a fixed order: 16 columns and 16 part lanes a
// workgroup, so that few columns still fill the chip.
__global__ void __launch_bounds__(256) norm_join_kernel(const float* __restrict__ part, int parts, int d,
                                                        float* __restrict__ out) {
    __shared__ float s_v[16][17];
    const int cl = threadIdx.x & 15, l = threadIdx.x >> 4;
    const int c = blockIdx.x * 16 + cl;
    float v = 0.f;
    if (c < d) {
#pragma unroll 4
        for (int k = l; k < parts; k += 16) v += part[(int64_t)k * d + c];
    }
    s_v[l][cl] = v;
    __syncthreads();
    if (l == 0 && c < d) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) t += s_v[k][cl];
        out[c] = t;
    }
}

// How a width is held: 64 threads a row up to 1024 columns, else 256.
struct NormShape {
    int tpr, nc;
};
static NormShape norm_shape(int d) {
    const int cpr = d / 8;
    if (cpr <= 64) return {64, 1};
    if (cpr <= 128) return {64, 2};
    const int nc = (cpr + 255) / 256;
    return {256, nc <= 1 ? 1 : nc <= 2 ? 2 : nc <= 4 ? 4 : 8};
}

template <class F>
static void norm_dispatch(int d, F&& f) {
    const NormShape sh = norm_shape(d);
    auto go = [&](auto A, auto B) { f(A, B); };
    using std::integral_constant;
    if (sh.tpr == 64 && sh.nc == 1) go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (sh.tpr == 64) go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else if (sh.nc == 1) go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (sh.nc == 2) go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (sh.nc == 4) go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
    else go(integral_constant<int, 256>{}, integral_constant<int, 8>{});
}

// Workgroups of a backward pass: about four rows each, 1024 at most.
static int norm_bwd_groups(int T, int d) {
    const int rpb = kNormThreads / norm_shape(d).tpr;
    const int64_t groups = ((int64_t)T + rpb - 1) / rpb;
    return (int)std::min<int64_t>(1024, (groups + 3) / 4);
}
static int norm_parts(int T, int d) { return norm_bwd_groups(T, d) * (kNormThreads / norm_shape(d).tpr); }

size_t norm_workspace_bytes(int T, int d) {
    const int parts = norm_parts(T, d);
    return parts > 1 ? (size_t)parts * d * sizeof(float) : 0;
}

static int done() { return hipGetLastError() == hipSuccess ? 0 : -4; }

// The rows in launches of at most kNormGroups workgroups, f(first row, rows): one of 2^32 threads and more would be cut
// off without an error.
constexpr int64_t kNormGroups = 1 << 22;
template <class F>
static void by_rows(int T, int rows_per_group, F&& f) {
    const int64_t step = kNormGroups * rows_per_group;
    for (int64_t t = 0; t < T; t += step) f(t, (int)std::min(step, T - t));
}
template <class E>
static E* at_row(E* p, int64_t offset) { return p ? p + offset : p; }

int launch_norm_fwd(const NormFwd& p, hipStream_t s) {
    norm_dispatch(p.d, [&](auto A, auto B) {
        constexpr int TPR = decltype(A)::value, NC = decltype(B)::value, RPB = kNormThreads / TPR;
        by_rows(p.T, RPB, [&](int64_t t, int rows) {
            NormFwd q = p;
            const int64_t o = t * p.d;
            q.T = rows, q.x = p.x + o, q.res = at_row(p.res, o), q.total = at_row(p.total, o), q.y = p.y + o, q.rstd = at_row(p.rstd, t);
            norm_fwd_kernel<TPR, NC><<<(unsigned)((rows + RPB - 1) / RPB), kNormThreads, 0, s>>>(q);
        });
    });
    return done();
}

int launch_post_norm_fwd(const PostNormFwd& p, hipStream_t s) {
    norm_dispatch(p.d, [&](auto A, auto B) {
        constexpr int TPR = decltype(A)::value, NC = decltype(B)::value, RPB = kNormThreads / TPR;
        by_rows(p.T, RPB, [&](int64_t t, int rows) {
            PostNormFwd q = p;
            const int64_t o = t * p.d;
            if (!p.row_of) q.y = p.y + o;  // else the experts' rows, wherever they are
            q.row_of = at_row(p.row_of, t * p.k), q.topk_w = at_row(p.topk_w, t * p.k), q.gate = at_row(p.gate, t * p.gate_cols);
            q.T = rows, q.x = p.x + o, q.total = at_row(p.total, o), q.out = p.out + o, q.rstd = at_row(p.rstd, t);
            post_norm_fwd_kernel<TPR, NC><<<(unsigned)((rows + RPB - 1) / RPB), kNormThreads, 0, s>>>(q);
        });
    });
    return done();
}

template <class P, class L>
static int norm_bwd_any(const P& p, void* ws, hipStream_t s, L&& launch) {
    const int groups = norm_bwd_groups(p.T, p.d), parts = norm_parts(p.T, p.d);
    float* part = !p.dw ? nullptr : parts > 1 ? (float*)ws : p.dw;
    launch(groups, part);
    if (p.dw && parts > 1)
        norm_join_kernel<<<(unsigned)((p.d + 15) / 16), 256, 0, s>>>(part, parts, p.d, p.dw);
    return done();
}

int launch_norm_bwd(const NormBwd& p, void* ws, hipStream_t s) {
    return norm_bwd_any(p, ws, s, [&](int groups, float* part) {
        norm_dispatch(p.d, [&](auto A, auto B) {
            norm_bwd_kernel<decltype(A)::value, decltype(B)::value><<<groups, kNormThreads, 0, s>>>(p, part);
        });
    });
}

int launch_post_norm_bwd(const PostNormBwd& p, void* ws, hipStream_t s) {
    return norm_bwd_any(p, ws, s, [&](int groups, float* part) {
        norm_dispatch(p.d, [&](auto A, auto B) {
            post_norm_bwd_kernel<decltype(A)::value, decltype(B)::value><<<groups, kNormThreads, 0, s>>>(p, part);
        });
    });
}

}  // namespace moe
