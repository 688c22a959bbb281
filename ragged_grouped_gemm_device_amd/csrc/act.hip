// Elementwise passes of the dense linear layer's backward, and the restoring of
// 8-bit checkpoints.
//
//   moe_act_bwd        dz = dy * f'(z), a = f(z), dbias = column sums of dz, with z
//                      read as bf16 or straight from its MXFP8 checkpoint
//   moe_dequant_mxfp8  bf16 values of row-wise MXFP8 codes
//
// All are bound by HBM traffic: 16-byte accesses, one pass.
#include <algorithm>

#include "dense_common.hpp"

namespace moe {

struct ActArgs {
    const uint16_t* dy;  // [T, NO], or nullptr: only a
    const uint16_t* z;   // [T, N], or nullptr: z_q, z_s
    const uint8_t* z_q;
    const uint8_t* z_s;
    int T, N;
    uint16_t* dz;  // [T, N] or nullptr
    uint16_t* a;   // [T, NO] or nullptr
    float* part;   // [row chunks, N] column sums, or nullptr
    int rows;      // rows per chunk
};

__device__ __forceinline__ void unpack8(uint4 w, float* v) {
    unpack_bf16x4(make_uint2(w.x, w.y), v);
    unpack_bf16x4(make_uint2(w.z, w.w), v + 4);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

// A workgroup takes 32 groups of 8 output columns (gated: with their 8 gate and
// 8 up columns) and `rows` rows, 8 rows at a time; a thread keeps its columns'
// sums of dz (fp32, before the rounding) in registers over the rows, joined over
// the 8 row lanes in LDS in a fixed order. dz leaves as bf16 because both gradient
// products read it on the bf16 matrix cores: each of its values moves by up to 2^-8, and
// dx and dw, an fp32 dw too, are with it off by 0.23 to 0.24% in norm (0.17% from
// rounding dx or dw itself to bf16). An fp32 dz would need the products on fp32 matrix
// instructions, a sixteenth of the bf16 rate.
template <int ACT, bool Z8>
__global__ void __launch_bounds__(256) act_bwd_kernel(ActArgs p) {
    constexpr bool G = ACT < 2;
    constexpr int H = G ? 2 : 1;
    __shared__ float s_sum[8][32][8 * H + 1];
    const int gl = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int NO = G ? p.N / 2 : p.N;
    const int g = blockIdx.x * 32 + gl;
    const bool live = g < NO / 8;
    const int c0 = G ? (g >> 2) * 64 + (g & 3) * 8 : g * 8;
    const int64_t r0 = (int64_t)blockIdx.y * p.rows;
    const int64_t r1 = min(r0 + p.rows, (int64_t)p.T);
    float sum[H][8];
#pragma unroll
    for (int u = 0; u < H; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[u][i] = 0.f;
    for (int64_t m = r0 + rl; live && m < r1; m += 8) {
        float d[8], z[H][8], o[H][8], a[8];
        if (p.dy) unpack8(*(const uint4*)(p.dy + m * NO + 8 * g), d);
        else {
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = 0.f;
        }
        if constexpr (ACT != 3) {
#pragma unroll
            for (int u = 0; u < H; ++u) {
                const int col = c0 + 32 * u;
                if constexpr (Z8) {
                    const uint2 q = *(const uint2*)(p.z_q + m * p.N + col);
                    const float sc = e8m0_value(p.z_s[m * (p.N / 32) + col / 32]);
                    e4m3x4_value(q.x, sc, z[u]);
                    e4m3x4_value(q.y, sc, z[u] + 4);
                } else {
                    unpack8(*(const uint4*)(p.z + m * p.N + col), z[u]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (G) {
                float f, df;
                dense_act_grad<ACT>(z[0][i], f, df);
                a[i] = f * z[1][i];
                o[0][i] = d[i] * z[1][i] * df;
                o[1][i] = d[i] * f;
            } else if constexpr (ACT == 3) {
                a[i] = 0.f;
                o[0][i] = d[i];
            } else {
                float df;
                dense_act_grad<ACT>(z[0][i], a[i], df);
                o[0][i] = d[i] * df;
            }
        }
#pragma unroll
        for (int u = 0; u < H; ++u) {
            if (p.dz) *(uint4*)(p.dz + m * p.N + c0 + 32 * u) = pack8(o[u]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[u][i] += o[u][i];
        }
        if (ACT != 3 && p.a) *(uint4*)(p.a + m * NO + 8 * g) = pack8(a);
    }
    if (!p.part) return;
#pragma unroll
    for (int u = 0; u < H; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) s_sum[rl][gl][8 * u + i] = sum[u][i];
    __syncthreads();
    for (int q = threadIdx.x; q < 32 * 8 * H; q += 256) {
        const int gq = q / (8 * H), iq = q % (8 * H);
        const int gg = blockIdx.x * 32 + gq;
        if (gg >= NO / 8) continue;
        float v = 0.f;
#pragma unroll
        for (int l = 0; l < 8; ++l) v += s_sum[l][gq][iq];
        const int col = (G ? (gg >> 2) * 64 + (gg & 3) * 8 : gg * 8) + (iq >> 3) * 32 + (iq & 7);
        p.part[(int64_t)blockIdx.y * p.N + col] = v;
    }
}

// dbias[c] = sum of the chunks' column sums, in a fixed order: 16 columns and 16
// chunk lanes per workgroup, so that few columns still fill the chip.
__global__ void __launch_bounds__(256) colsum_kernel(const float* __restrict__ part, int chunks, int N,
                                                     float* __restrict__ out) {
    __shared__ float s_v[16][17];
    const int cl = threadIdx.x & 15, l = threadIdx.x >> 4;
    const int c = blockIdx.x * 16 + cl;
    float v = 0.f;
    if (c < N) {
#pragma unroll 4
        for (int k = l; k < chunks; k += 16) v += part[(int64_t)k * N + c];
    }
    s_v[l][cl] = v;
    __syncthreads();
    if (l == 0 && c < N) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) t += s_v[k][cl];
        out[c] = t;
    }
}

// 8 codes a thread: 8 bytes in, one 16-byte store. NT: streaming stores, for outputs
// past kDenseStreamBytes, which the last-level cache would not hold for their reader
// ([32768, 4096]: 64.2 us, 6.3 TB/s; 68.6 with plain stores, 72.8 with 16 codes a
// thread). Bound by HBM.
template <bool NT>
__global__ void __launch_bounds__(256) dequant_mxfp8_kernel(const uint8_t* __restrict__ q,
                                                            const uint8_t* __restrict__ s, int64_t n8,
                                                            uint16_t* __restrict__ out) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
        const uint2 w = ((const uint2*)q)[i];
        const float sc = e8m0_value(s[i >> 2]);
        float v[8];
        e4m3x4_value(w.x, sc, v);
        e4m3x4_value(w.y, sc, v + 4);
        if constexpr (NT) st_nt16((uint4*)out + i, pack8(v));
        else ((uint4*)out)[i] = pack8(v);
    }
}

// Row chunks of moe_act_bwd, at least 8 rows each: about 8192 workgroups, but fewer
// where each leaves a row of column sums, 1024 of the gated form and 2048 of the others,
// whose threads have half as much in flight. [16384, 4096] SwiGLU without dbias 59.5 us
// with 1024 workgroups, 61.0, 56.0, 52.2 with 2048, 4096, 8192; with dbias 62.3, 64.5,
// 62.3, 62.7. SiLU with dbias 73.3, 68.5, 71.5, 68.8.
static void act_chunks(int T, int N, bool gated, bool sums, int& rows, int& chunks) {
    const int64_t tiles = ((gated ? N / 2 : N) / 8 + 31) / 32;
    const int64_t target = !sums ? 8192 : gated ? 1024 : 2048;
    const int64_t r = ((int64_t)T * tiles + target - 1) / target;
    rows = (int)std::max<int64_t>(8, (r + 7) / 8 * 8);
    chunks = (T + rows - 1) / rows;
}

size_t act_part_bytes(int T, int N) {
    size_t most = 0;
    for (int gated = 0; gated < 2; ++gated) {
        int rows, chunks;
        act_chunks(T, N, gated, true, rows, chunks);
        most = std::max(most, chunks > 1 ? (size_t)chunks * N * sizeof(float) : 0);
    }
    return most;
}

int launch_act_bwd(const uint16_t* dy, const uint16_t* z, const uint8_t* z_q, const uint8_t* z_s, int T, int N,
                   int act, uint16_t* dz, uint16_t* a, float* dbias, void* ws, hipStream_t s) {
    const bool gated = act < 2;
    int rows, chunks;
    act_chunks(T, N, gated, dbias != nullptr, rows, chunks);
    ActArgs p{};
    p.dy = dy, p.z = z, p.z_q = z_q, p.z_s = z_s, p.T = T, p.N = N, p.dz = dz, p.a = a, p.rows = rows;
    p.part = !dbias ? nullptr : chunks > 1 ? (float*)ws : dbias;
    const dim3 grid((unsigned)(((gated ? N / 2 : N) / 8 + 31) / 32), (unsigned)chunks);
    auto go = [&](auto A) {
        constexpr int ACT = decltype(A)::value;
        if (ACT != 3 && !z) act_bwd_kernel<ACT, ACT != 3><<<grid, 256, 0, s>>>(p);
        else act_bwd_kernel<ACT, false><<<grid, 256, 0, s>>>(p);
    };
    switch (act) {
        case 0: go(std::integral_constant<int, 0>{}); break;
        case 1: go(std::integral_constant<int, 1>{}); break;
        case 2: go(std::integral_constant<int, 2>{}); break;
        case 3: go(std::integral_constant<int, 3>{}); break;
        case 4: go(std::integral_constant<int, 4>{}); break;
        default: go(std::integral_constant<int, 5>{}); break;
    }
    if (dbias && chunks > 1)
        colsum_kernel<<<(unsigned)((N + 15) / 16), 256, 0, s>>>((const float*)ws, chunks, N, dbias);
    return hipGetLastError() == hipSuccess ? 0 : -4;
}

int launch_dequant_mxfp8(const uint8_t* q, const uint8_t* sc, int64_t R, int C, uint16_t* out, hipStream_t s) {
    const int64_t n8 = R * (C / 8);
    const unsigned blocks = (unsigned)std::min<int64_t>((n8 + 255) / 256, (int64_t)1 << 20);
    if (n8 * 16 >= kDenseStreamBytes) dequant_mxfp8_kernel<true><<<blocks, 256, 0, s>>>(q, sc, n8, out);
    else dequant_mxfp8_kernel<false><<<blocks, 256, 0, s>>>(q, sc, n8, out);
    return hipGetLastError() == hipSuccess ? 0 : -4;
}

}  // namespace moe
