// 4-bit blocks: quantisation of bf16 matrices, row-wise or transposed, and back (gfx950).
//
// A block is 32 values; its E8M0 scale is the smallest power of two 2^e with amax <= 6 * 2^e, so that no
// value is clipped (as the 8-bit blocks' scale, with E4M3's 448), its codes are E2M1 (1 sign, 2
// exponent, 1 fraction bit), v / 2^e rounded to the nearest, ties to the even code. E2M1 has no NaN: a
// block with a NaN or an infinity takes scale 255, E8M0's NaN, and is NaN as a whole wherever it is read.
// gfx950's packed conversion divides by the scale and rounds so for every bf16 value (checked over
// all of them).
//
// Both directions are bound by HBM: 2 bytes in and 17/32 out a value, or the reverse. 8 x 7168 x 4096 values: by
// columns 122 us (4.9 TB/s), restored 101 (5.9); by rows 16384 x 7168 53 (5.6) and 131072 x 2048 114 (5.9), restored 44
// and 96 (6.8, 7.1: the codes come from the last-level cache); 1021 x 2880: 3.1 us by rows, 3.4 restored, a launch's time.
#include <algorithm>

#include "block_common.hpp"
#include "dense_common.hpp"

namespace moe {

// E8M0 code of a block from the bf16 bits of its largest magnitude (sign cleared): amax = (1 + M/128)
// 2^(E-127) and 6 = 1.5 * 2^2, so e = E - 127 - 2, plus one above 1.5 (M > 64), at least -127.
__device__ __forceinline__ uint32_t mx4_scale(uint32_t amax) {
    const int E = (int)(amax >> 7);
    if (E == 0xff) return 255;
    return (uint32_t)max(0, E - 2 + ((amax & 0x7fu) > 64u ? 1 : 0));
}

// The codes of 8 values (4 words of bf16 pairs) under scale code sc, first value in the low half byte.
__device__ __forceinline__ uint32_t mx4_codes(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t sc) {
    const float f = e8m0_value(sc);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, a), f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, b), f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, c), f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, d), f, 3);
    return sc == 255 ? 0u : w;
}

__device__ __forceinline__ uint32_t magnitude8(uint4 v) {
    const uint32_t m = max_u16x2(max_u16x2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                 max_u16x2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    return max(m & 0xffffu, m >> 16);
}

// Row-wise: 8 values a thread, four threads a block; 16 bytes in, 4 out, both whole lines a wavefront.
__global__ void __launch_bounds__(256) quant_mxfp4_row_kernel(const uint4* __restrict__ src, int64_t n8,
                                                              uint32_t* __restrict__ q, uint8_t* __restrict__ s) {
    const int64_t step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += step) {  // whole blocks leave together
        const uint4 v = src[i];
        uint32_t m = magnitude8(v);
        m = max(m, xor_lane<1>(m));
        m = max(m, xor_lane<2>(m));
        const uint32_t sc = mx4_scale(m);
        q[i] = mx4_codes(v.x, v.y, v.z, v.w, sc);
        if ((i & 3) == 0) s[i >> 2] = (uint8_t)sc;
    }
}

// Transposed: a workgroup takes 256 rows x 64 columns, a thread 8 rows x 8 columns (columns 8 (l & 7) +
// [0, 8), rows 8 (8 w + l / 8) + [0, 8)), so that the four threads of a 32-row block are two lane exchanges
// apart and a column's 256 codes are one 128-byte line. Codes and scales are turned in LDS (16-byte pieces
// XOR-swizzled by the column group).
__global__ void __launch_bounds__(256) quant_mxfp4_col_kernel(const uint16_t* __restrict__ src, int64_t R, int C,
                                                              uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
    __shared__ __align__(16) uint8_t s_q[64 * 128];
    __shared__ __align__(16) uint8_t s_s[64 * 8];
    const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int cc = l & 7, rg = 8 * w + (l >> 3);
    const int c0 = blockIdx.x * 64, c = c0 + 8 * cc;
    const int64_t r0 = (int64_t)blockIdx.y * 256, r = r0 + 8 * rg;
    src += (int64_t)blockIdx.z * R * C;
    q += (int64_t)blockIdx.z * R * C / 2;
    s += (int64_t)blockIdx.z * R * C / 32;
    const bool ok = c < C && r < R;  // rows come in blocks of 32, columns in eights
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ok ? *(const uint4*)(src + (r + i) * C + c) : make_uint4(0, 0, 0, 0);
    auto word = [&](int i, int p) -> uint32_t { return p == 0 ? v[i].x : p == 1 ? v[i].y : p == 2 ? v[i].z : v[i].w; };
    uint32_t m[4];  // largest magnitudes of columns (2p, 2p + 1)
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        m[p] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m[p] = max_u16x2(m[p], word(i, p) & 0x7fff7fffu);
        m[p] = max_u16x2(m[p], xor_lane<8>(m[p]));
        m[p] = max_u16x2(m[p], xor_lane<16>(m[p]));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t sc = mx4_scale((j & 1) ? m[j >> 1] >> 16 : m[j >> 1] & 0xffffu);
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;  // the column's halves of two rows
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __builtin_amdgcn_perm(word(2 * i + 1, j >> 1), word(2 * i, j >> 1), sel);
        const int col = 8 * cc + j;
        *(uint32_t*)(s_q + col * 128 + (((rg >> 2) ^ cc) << 4) + (rg & 3) * 4) = mx4_codes(p[0], p[1], p[2], p[3], sc);
        if ((rg & 3) == 0) s_s[col * 8 + (rg >> 2)] = (uint8_t)sc;
    }
    __syncthreads();
    const int64_t rb = R / 32;
#pragma unroll
    for (int it = 0; it < 2; ++it) {
        const int i = it * 256 + threadIdx.x, col = i >> 3, g = i & 7;  // piece g: rows 32 g .. 32 g + 31
        if (c0 + col < C && r0 + 32 * g < R)
            *(uint4*)(q + (int64_t)(c0 + col) * (R / 2) + r0 / 2 + 16 * g) =
                *(const uint4*)(s_q + col * 128 + ((g ^ (col >> 3)) << 4));
    }
    if ((R & 255) == 0 && ((uintptr_t)s & 7) == 0) {
        if (threadIdx.x < 64 && c0 + (int)threadIdx.x < C)
            *(uint2*)(s + (int64_t)(c0 + threadIdx.x) * rb + r0 / 32) = *(const uint2*)(s_s + 8 * threadIdx.x);
    } else {
        for (int i = threadIdx.x; i < 512; i += 256) {
            const int col = i >> 3, g = i & 7;
            if (c0 + col < C && r0 + 32 * g < R) s[(int64_t)(c0 + col) * rb + r0 / 32 + g] = s_s[i];
        }
    }
}

// 8 values a thread: 4 bytes in, one 16-byte store. NT: past the caches, for outputs that these would not
// hold for their reader (from kDenseStreamBytes, as the 8-bit blocks').
template <bool NT>
__global__ void __launch_bounds__(256) dequant_mxfp4_kernel(const uint32_t* __restrict__ q,
                                                            const uint8_t* __restrict__ s, int64_t n8,
                                                            uint4* __restrict__ out) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
        const uint32_t w = q[i], sc = s[i >> 2];
        const float f = e8m0_value(sc);
        uint4 v;
        v.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 0));
        v.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 1));
        v.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 2));
        v.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 3));
        if (sc == 255) v = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
        if constexpr (NT) st_nt16(out + i, v);
        else out[i] = v;
    }
}

int launch_quant_mxfp4(const uint16_t* src, int batch, int64_t R, int C, int mode, uint8_t* q_row, uint8_t* s_row,
                       uint8_t* q_col, uint8_t* s_col, hipStream_t s) {
    if (mode & 1) {
        const int64_t n8 = (int64_t)batch * R * (C / 8);
        const unsigned blocks = (unsigned)std::min<int64_t>((n8 + 255) / 256, (int64_t)1 << 20);
        quant_mxfp4_row_kernel<<<blocks, 256, 0, s>>>((const uint4*)src, n8, (uint32_t*)q_row, s_row);
    }
    if (mode & 2) {
        const dim3 grid((C + 63) / 64, (unsigned)((R + 255) / 256), batch);
        quant_mxfp4_col_kernel<<<grid, 256, 0, s>>>(src, R, C, q_col, s_col);
    }
    return hipGetLastError() == hipSuccess ? 0 : -4;
}

int launch_dequant_mxfp4(const uint8_t* q, const uint8_t* sc, int64_t R, int C, uint16_t* out, hipStream_t s) {
    const int64_t n8 = R * (C / 8);
    const unsigned blocks = (unsigned)std::min<int64_t>((n8 + 255) / 256, (int64_t)1 << 20);
    if (n8 * 16 >= kDenseStreamBytes)
        dequant_mxfp4_kernel<true><<<blocks, 256, 0, s>>>((const uint32_t*)q, sc, n8, (uint4*)out);
    else
        dequant_mxfp4_kernel<false><<<blocks, 256, 0, s>>>((const uint32_t*)q, sc, n8, (uint4*)out);
    return hipGetLastError() == hipSuccess ? 0 : -4;
}

}  // namespace moe
