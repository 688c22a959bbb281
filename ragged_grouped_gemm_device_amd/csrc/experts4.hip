// The experts' product with 4-bit weights (gfx950): y[R_e] = f(X[R_e] W_e), W_e given as MXFP4 rows
// [N, K] (blocks along K), X as bf16, MXFP8 or MXFP4, sums in fp32.
//
// Two kernels. experts4_tile_kernel: tiles of BM rows x 256 columns over LDS slabs, for experts with many
// rows, bound by the matrix cores. experts4_rows_kernel: weights straight from HBM into the matrix
// instruction's operands, for few rows (single tokens, decode batches), bound by the read of W.
//
// 8- and 4-bit operands go into v_mfma_scale as they are, with their block scales. bf16 rows need bf16
// weights: a code times its scale is one, exactly, and gfx950 converts two in one instruction; 8
// conversions feed 8 MFMAs of a wavefront.
#include <algorithm>

#include "block_common.hpp"
#include "dense_common.hpp"

namespace moe {

constexpr int kBf16 = 0, kMx8 = 1, kMx4 = 2;  // formats of X
constexpr int kWaitLgkmcnt0 = 0xC07F;         // s_waitcnt lgkmcnt(0) alone

struct Experts4Args {
    const uint8_t* x;       // rows of K bf16, K bytes or K / 2 bytes
    const uint8_t* xs;      // block scales [rows, K / 32]; formats 1, 2
    const int32_t* src_of;  // nullable: rows are those of the experts' buffer
    int k;
    int64_t rows;           // rows of x
    const uint8_t *wq, *ws;
    const int32_t *offsets, *counts;
    int E, N, K, act;
    uint16_t* y;
};

__device__ __forceinline__ int64_t x_row_bytes(int fmt, int K) { return fmt == kBf16 ? 2 * (int64_t)K : fmt == kMx8 ? K : K / 2; }

// f of one output, or of a gate and its up value
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case 0: f(std::integral_constant<int, 0>{}); break;
        case 1: f(std::integral_constant<int, 1>{}); break;
        case 2: f(std::integral_constant<int, 2>{}); break;
        case 3: f(std::integral_constant<int, 3>{}); break;
        case 4: f(std::integral_constant<int, 4>{}); break;
        default: f(std::integral_constant<int, 5>{}); break;
    }
}

// 8 bf16 weights from 8 codes (a word) and their block's scale
__device__ __forceinline__ bf16x8_t weights8(uint32_t w, float s) {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    return bf16x8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

__device__ __forceinline__ i32x8_t operand4(uint4 v) { return i32x8_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0}; }
__device__ __forceinline__ i32x8_t operand8(uint4 a, uint4 b) {
    return i32x8_t{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// ------------------------------------------------------------------ few rows
// A workgroup takes 64 columns of one expert and 16 RT of its rows; its NW wavefronts split K in blocks of 256
// and join in LDS. In a 16 x 16 x 128 product lane l supplies row l & 15 of W and of X and one 32-value block of
// each, lane group l / 16 the blocks 2 (l / 16) + s of a block's two steps s; with bf16 a 32-value block is used
// in four 16 x 16 x 32 products, a word of W in each.
// W goes through LDS, though no lane shares it: read straight into that layout, neighbouring lanes would ask
// for different rows, four lines for every four lanes, and the load path, not HBM, would be the bound (3.1 to
// 4.2 TB/s in the forms tried; copies of whole 128-byte lines: see below). Each wavefront copies its own blocks,
// 64 rows of 128 bytes, one ahead of the one it multiplies, and waits for no other. X, a few rows, comes
// straight from the caches: lanes without a row ask for nothing. The scales of W's rows, 8 bytes of a line a
// block, are laid into LDS once for 8192 of K.
// One token, 8 of 32 experts: 7168 x 4096 SwiGLU 24 to 26 us (4.8 to 5.1 TB/s, a large copy's rate), 2048 x 7168 15.7 to
// 17.1 (3.7 to 4.0); 16 tokens, all experts, 7168 x 4096: 88 to 100 (5.0 to 5.6). With 32 bf16 rows one register goes to
// scratch.
constexpr int kScaleChunk = 256;  // scale bytes of a row in LDS; 16-byte pieces XOR-swizzled by the row

template <int F, int RT, int NW>
__global__ void __launch_bounds__(NW * 64, 2) experts4_rows_kernel(Experts4Args p) {
    constexpr int kLd = 68;  // floats a row of the join: 64 and a pad against bank conflicts
    constexpr int kX = F == kBf16 ? 4 : F == kMx8 ? 2 : 1;  // 16-byte pieces of a 32-value block of X
    constexpr int kXBlock = F == kBf16 ? 512 : F == kMx8 ? 256 : 128;  // bytes of 256 of K
    __shared__ __attribute__((aligned(1024))) uint8_t s_w[NW][2][64 * 128];  // then the join
    __shared__ __align__(16) uint8_t s_sc[64 * kScaleChunk];
    static_assert(sizeof(float) * 16 * RT * kLd <= sizeof(s_w[0]), "the join fits the blocks");
    auto s_red = [&](int w, int row, int c) { return (float*)&s_w[w][0][0] + row * kLd + c; };
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    // the blockIdx.y-th expert that has rows
    int e = -1, m = 0;
    for (int base = 0, left = blockIdx.y; base < p.E; base += 64) {
        const int c = base + lane < p.E ? p.counts[base + lane] : 0;
        uint64_t some = __ballot(c > 0);
        const int n = __popcll(some);
        if (left < n) {
            while (left--) some &= some - 1;
            const int at = __ffsll((unsigned long long)some) - 1;
            e = base + at;
            m = __shfl(c, at, 64);
            break;
        }
        left -= n;
    }
    e = __builtin_amdgcn_readfirstlane(e);
    m = __builtin_amdgcn_readfirstlane(m);
    if (e < 0) return;
    const int n0 = blockIdx.x * 64;
    const int K = p.K, KB = K / 32, cols = min(p.N - n0, 64);
    const int64_t wrow = (int64_t)e * p.N + n0;
    const uint8_t* wsc = p.ws + wrow * KB;
    // rows past the last column: past the resource, zeros; past K: another row's codes, finite, under scales of
    // 0 and times zeros of X
    const i32x4_t rw = rsrc_words(p.wq + wrow * (K / 2), (uint32_t)cols * (K / 2));
    const uint32_t lds = (uint32_t)(uintptr_t)(LDS_AS char*)(&s_w[wave][0][0]);
    const uint32_t wo = (lane >> 3) * (uint32_t)(K / 2);
    auto copy_w = [&](int block, int buf) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = 8 * i + (lane >> 3);
            lds_copy16(rw, lds + buf * 8192 + i * 1024, wo + 4 * i * (uint32_t)K + 128 * block + (((lane & 7) ^ kmaj_swz(row)) << 4));
        }
    };
    const int64_t xb = x_row_bytes(F, K);
    for (int first = blockIdx.z * 16 * RT; first < m; first += gridDim.z * 16 * RT) {
        const int row0 = p.offsets[e] + first, rows = min(m - first, 16 * RT);
        const int64_t base = p.src_of ? 0 : row0, space = p.src_of ? p.rows : rows;
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x + base * xb, clamp_records(space * xb));
        const __amdgpu_buffer_rsrc_t rxs = make_rsrc(F == kBf16 ? p.x : p.xs + base * KB, clamp_records(space * KB));
        f32x4_t acc[4][RT];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < RT; ++i) acc[j][i] = (f32x4_t){};
        uint32_t xrow[RT];  // this lane's rows; kMasked: none
        for (int kb = 0; kb < KB; kb += kScaleChunk) {
            const int nkb = min(KB - kb, kScaleChunk), nb = (nkb + 7) / 8, kb8 = kb / 8;
            const int b0 = nb * wave / NW, b1 = nb * (wave + 1) / NW;
            if (b0 < b1) copy_w(kb8 + b0, 0);
            if (kb == 0) {
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const int at = 16 * i + r;
                    xrow[i] = at >= rows ? kMasked : (uint32_t)(p.src_of ? p.src_of[row0 + at] / p.k : at);
                }
            }
            struct XBlock {
                u32x4_nt_t x[RT][2][kX];
                int s[RT][2];
            };
            auto load_x = [&](XBlock& b, int at) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const bool has = xrow[i] != kMasked;
#pragma unroll
                        for (int q = 0; q < kX; ++q) {
                            // an 8-bit lane's two pieces are halves of the blocks that lane groups g / 2 and 2 + g / 2 have of W
                            const int of = F == kMx8 ? 2 * (g >> 1) + 4 * q + s : 2 * g + s;
                            const uint32_t o = F == kMx8 ? 64 * (g >> 1) + 16 * (g & 1) + 128 * q + 32 * s : 32 * kX * g + 16 * kX * s + 16 * q;
                            b.x[i][s][q] = __builtin_amdgcn_raw_buffer_load_b128(
                                rx, has && 8 * at + of < nkb ? xrow[i] * (uint32_t)xb + o : kMasked, kXBlock * (kb8 + at), 0);
                        }
                        b.s[i][s] = 0;
                        if constexpr (F != kBf16)
                            b.s[i][s] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
                                rxs, has && 8 * at + 2 * g + s < nkb ? xrow[i] * (uint32_t)KB + 2 * g + s : kMasked, kb + 8 * at, 0);
                    }
                }
            };
            XBlock xn;
            if (b0 < b1) load_x(xn, b0);
            // W's scales, NW threads a row, 16 bytes each and turn, all loads out before the first is waited for;
            // zeros past K and past the last column
            constexpr int kTurns = kScaleChunk / (16 * NW);
            const int srow = threadIdx.x / NW, part = threadIdx.x % NW;
            uint4 sv[kTurns];
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {
                const int c = 16 * (part + NW * i), n = min(16, nkb - c);
                sv[i] = make_uint4(0, 0, 0, 0);
                if (srow < cols && n > 0) {
                    const uint8_t* src = wsc + (int64_t)srow * KB + kb + c;
                    if ((int64_t)(srow + 1) * KB + 16 <= (int64_t)cols * KB || n == 16) {
                        __builtin_memcpy(&sv[i], src, 16);  // past its row's end: the next rows'
                    } else {
                        uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            if (q < n) v[q >> 2] |= (uint32_t)src[q] << (8 * (q & 3));
                        sv[i] = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {
                const int c = 16 * (part + NW * i), n = nkb - c;
                auto keep = [&](uint32_t v, int at) { return n >= at + 4 ? v : n <= at ? 0u : v & ((1u << (8 * (n - at))) - 1u); };
                if (c < 8 * nb)
                    *(uint4*)(s_sc + srow * kScaleChunk + (c ^ ((srow & 15) << 4))) =
                        make_uint4(keep(sv[i].x, 0), keep(sv[i].y, 4), keep(sv[i].z, 8), keep(sv[i].w, 12));
            }
            __syncthreads();
            for (int b = b0; b < b1; ++b) {
                const int buf = (b - b0) & 1;
                // the block and its X are here (their copies and loads are the only ones out)
                __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
                const XBlock x = xn;
                if (b + 1 < b1) {
                    copy_w(kb8 + b + 1, buf ^ 1);
                    load_x(xn, b + 1);
                }
                const uint8_t* sw = s_w[wave][buf];
                uint32_t sc[4];  // two steps' scales
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sc[j] = *(const uint16_t*)(s_sc + (16 * j + r) * kScaleChunk + ((8 * b + 2 * g) ^ (r << 4)));
#pragma unroll
                for (int s = 0; s < 2; ++s) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const u32x4_nt_t w = *(const u32x4_nt_t*)(sw + kmaj_byte(16 * j + r, 2 * g + s));
                        if constexpr (F == kBf16) {
                            // the conversion reads a float's exponent alone
                            const float f = __uint_as_float(s ? sc[j] << 15 : sc[j] << 23);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const bf16x8_t v = weights8(w[q], f);
#pragma unroll
                                for (int i = 0; i < RT; ++i)
                                    acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8_t, x.x[i][s][q]),
                                                                                        acc[j][i], 0, 0, 0);
                            }
                        } else {
                            const i32x8_t v = operand4(__builtin_bit_cast(uint4, w));
#pragma unroll
                            for (int i = 0; i < RT; ++i) {
                                i32x8_t u;
                                if constexpr (F == kMx8)
                                    u = operand8(__builtin_bit_cast(uint4, x.x[i][s][0]), __builtin_bit_cast(uint4, x.x[i][s][1]));
                                else
                                    u = operand4(__builtin_bit_cast(uint4, x.x[i][s][0]));
                                // byte s of W's scales
                                acc[j][i] = s ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, u, acc[j][i], 4, F == kMx8 ? 0 : 4, 1,
                                                                                                 (int)sc[j], 0, x.s[i][s])
                                              : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, u, acc[j][i], 4, F == kMx8 ? 0 : 4, 0,
                                                                                                 (int)sc[j], 0, x.s[i][s]);
                            }
                        }
                    }
                }
                // every read of this buffer has come back before the next turn's copies into it
                __builtin_amdgcn_s_waitcnt(kWaitLgkmcnt0);
                __builtin_amdgcn_sched_barrier(0);
            }
            __syncthreads();  // the scales, or the last blocks, are read
        }
        // lane: row l & 15 of X, columns 16 j + 4 (l / 16) + [0, 4)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < RT; ++i) *(f32x4_t*)s_red(wave, 16 * i + r, 16 * j + 4 * g) = acc[j][i];
        __syncthreads();
        with_act(p.act, [&](auto A) {
            constexpr int ACT = decltype(A)::value;
            constexpr bool G = ACT < 2;
            constexpr int Q = G ? 8 : 16;  // quads of outputs a row
            const int NO = G ? p.N / 2 : p.N;
            for (int i = threadIdx.x; i < rows * Q; i += NW * 64) {
                const int row = i / Q, c = 4 * (i % Q);
                if (n0 / (G ? 2 : 1) + c >= NO) continue;
                f32x4_t a = {}, u = {};
#pragma unroll
                for (int v = 0; v < NW; ++v) {
                    a += *(const f32x4_t*)s_red(v, row, c);
                    if constexpr (G) u += *(const f32x4_t*)s_red(v, row, c + 32);
                }
                f32x4_t o;
#pragma unroll
                for (int q = 0; q < 4; ++q) o[q] = G ? dense_act<ACT>(a[q]) * u[q] : dense_act<ACT>(a[q]);
                *(uint2*)(p.y + (int64_t)(row0 + row) * NO + n0 / (G ? 2 : 1) + c) =
                    make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
            }
        });
        __syncthreads();  // read out before the next rows' blocks
    }
}

// ------------------------------------------------------------------ tiles
// What a format's slab holds: KS elements of K, 128 bytes a row of X (whole lines: in slabs of half the width, four in
// a ring, every line was fetched twice and the 4-bit form lost 13%) and WROW a row of W.
template <int F>
struct Slab {
    static constexpr int KS = F == kBf16 ? 64 : F == kMx8 ? 128 : 256;
    static constexpr int WROW = KS / 2, WCH = WROW / 16;  // 16-byte pieces a row of W: 2, 4, 8
    static constexpr int SPG = 512 / KS;                  // slabs that 16 scale bytes of a row serve, a group
};

// byte offset of 16-byte piece c of row r, rows of CH pieces: pieces are XOR-swizzled so that the rows of
// one 256-byte bank window and the next differ (128-byte rows: as the grouped GEMMs' slabs)
template <int CH>
__device__ __forceinline__ int slab_swz(int r) {
    return CH == 8 ? (r >> 1) & 7 : CH == 4 ? (r >> 2) & 3 : (r >> 3) & 1;
}
template <int CH>
__device__ __forceinline__ int slab_byte(int r, int c) {
    return r * CH * 16 + ((c ^ slab_swz<CH>(r)) << 4);
}

// s_waitcnt vmcnt(n) alone
constexpr int wait_vmcnt(int n) { return 0x0F70 | (n & 15) | (n >> 4 << 14); }

// Tiles of BMX rows x 256 columns, 2 x 4 wavefronts, each every other block of 32 rows and 64 columns; two slabs in LDS, the
// next on its way by copies that pass no registers while one is multiplied. The slabs of all of a workgroup's tiles are
// one sequence, so that the next tile's first arrives during the last's epilogue. 16384 tokens x 8 of 32 experts,
// 7168 x 4096, SwiGLU, by box and run: 4-bit rows 1990 to 2160 us (3560 to 3870 TFLOP/s), 8-bit 3130 to 3230 (2380 to
// 2460), bf16 5980 to 6300 (1220 to 1290, as a large library product). bf16 is bound by the matrix cores; in the 4-bit form they are busy 46% at the 1.8 GHz that the
// power limit leaves: multiplying alone took 1588 us, copying alone 1650, neither quite hidden behind the other.
// Tiles of fewer rows wait for W from HBM: there (kEarly) a slab's copies go out before the one they replace is multiplied to
// its end, as soon as all wavefronts have its last fragments: a barrier more a slab, and 7 to 11% less time (32 rows
// an expert, bf16: 210 -> 190 us, 4-bit 107 -> 98); with 256 rows the time did not fall (0 to +3%).
// Tried without gain: four slabs of 64-byte rows, 4 wavefronts of 128 x 128.
template <int F, int BMX, bool GLU>
__global__ void __launch_bounds__(512, 1) experts4_tile_kernel(Experts4Args p) {
    using SL = Slab<F>;
    constexpr int TM = BMX / 64;        // 32-row tiles a wavefront (2 x 4 wavefronts)
    constexpr int XB = BMX * 128, WB = 256 * SL::WROW;
    constexpr int XL = XB / 8192, WL = WB / 8192;  // copies of 16 bytes a thread
    constexpr bool kEarly = BMX < 256;  // copies go out before the slab they replace is multiplied to its end
    // a slab, or the epilogue's 4 KiB of each of the 8 wavefronts
    __shared__ __attribute__((aligned(1024))) uint8_t s_ab[2][XB + WB > 32768 ? XB + WB : 32768];
    __shared__ __attribute__((aligned(1024))) uint8_t s_sc[3][(BMX + 256) * 16];  // groups of scales
    __shared__ int s_tiles[MOE_MAX_E + 1];       // first large tile of every expert
    __shared__ uint16_t s_small[MOE_MAX_E + 1];  // its small one, if the next expert's is another
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int K = p.K, KB = K / 32, ntn = (p.N + 255) / 256;
    const int64_t xb = x_row_bytes(F, K);
    const int wb = K / 2;
    // Experts' last tiles with at most half the rows are small, and come after all others: workgroups take tiles in turn,
    // the small ones level out what they have.
    for (int e = tid; e < p.E; e += 512) {
        const int c = p.counts[e], left = c % BMX;
        s_tiles[e + 1] = c / BMX + (left > BMX / 2);
        s_small[e + 1] = left > 0 && left <= BMX / 2;
    }
    if (tid == 0) s_tiles[0] = s_small[0] = 0;
    __syncthreads();
    if (tid < 64) {
        int carry = 0, carry_small = 0;
        for (int base = 0; base < p.E; base += 64) {
            const int e = base + lane + 1;
            int v = e <= p.E ? s_tiles[e] : 0, u = e <= p.E ? s_small[e] : 0;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int v2 = __shfl_up(v, o, 64), u2 = __shfl_up(u, o, 64);
                if (lane >= o) v += v2, u += u2;
            }
            if (e <= p.E) s_tiles[e] = v + carry, s_small[e] = (uint16_t)(u + carry_small);
            carry += __shfl(v, 63, 64);
            carry_small += __shfl(u, 63, 64);
        }
    }
    __syncthreads();
    const int large = s_tiles[p.E], mtiles = large + s_small[p.E], total = mtiles * ntn;
    const int nbl = gridDim.x;  // a multiple of 8
    auto logical = [&](int round) { return round * nbl + (blockIdx.x & 7) * (nbl >> 3) + (blockIdx.x >> 3); };
    struct Tile {
        int e, row0, rows, n0;
    };
    auto get_tile = [&](int tt) -> Tile {
        constexpr int G = 8;  // bands of 8 M tiles: an XCD's neighbouring tiles share operand panels in its L2
        const int band = tt / (G * ntn), within = tt - band * G * ntn, bm = min(G, mtiles - band * G);
        const int mt = band * G + within % bm;
        const bool small = mt >= large;
        int e = 0;  // experts whose tiles all come before
        for (int base = 0; base < p.E; base += 64) {
            const int at = min(base + lane, p.E - 1) + 1;
            const bool before = small ? s_small[at] <= mt - large : s_tiles[at] <= mt;
            e += __popcll(__ballot(base + lane < p.E && before));
        }
        Tile t;
        t.e = e;
        // scalar loads: they wait for no copies
        const int count = ((const __attribute__((address_space(4))) int32_t*)p.counts)[e];
        const int skip = small ? count / BMX * BMX : __builtin_amdgcn_readfirstlane(mt - s_tiles[e]) * BMX;
        t.row0 = ((const __attribute__((address_space(4))) int32_t*)p.offsets)[e] + skip;
        t.rows = min(count - skip, BMX);
        t.n0 = __builtin_amdgcn_readfirstlane(within / bm * 256);
        return t;
    };
    // What a thread copies of a tile: its rows of X (offsets from the tile's or, gathered, x's base; rows past
    // the expert's last are its last again, and not stored), of W, and one row's scales.
    constexpr int WR = 512 / SL::WCH;  // rows of W a copy; of X, 64
    const int xc = (tid & 7) ^ slab_swz<8>(tid >> 3);  // the piece of a 128-byte row, the same in every copy
    const int wc = (tid & (SL::WCH - 1)) ^ slab_swz<SL::WCH>(tid / SL::WCH);
    const uint32_t wo = (uint32_t)(tid / SL::WCH) * wb + wc * 16;
    struct Src {
        i32x4_t rx, rw;
        uint32_t xo[XL];  // the rows, or the slots they come from; from the tile's first copies on, byte offsets
        int row;          // of this thread's scales
        const uint8_t* sc;  // threads [0, 256) W's rows, then X's
    };
    const bool scaled = tid < 256 + (F == kBf16 ? 0 : BMX);
    auto begin = [&](const Tile& t) -> Src {
        Src s;
        const int cols = min(p.N - t.n0, 256);
        const int64_t base = p.src_of ? 0 : t.row0;
        s.rx = rsrc_from(p.x, p.rows * xb, base * xb);
        const int64_t n0 = (int64_t)t.e * p.N + t.n0;
        s.rw = rsrc_words(p.wq + n0 * wb, clamp_records((int64_t)cols * wb));  // rows past the last column: zeros
        auto row_of = [&](int r) {
            const int row = min(r, t.rows - 1);
            return p.src_of ? p.src_of[t.row0 + row] : row;
        };
#pragma unroll
        for (int i = 0; i < XL; ++i) s.xo[i] = (uint32_t)row_of((tid >> 3) + 64 * i);
        s.row = min(tid & 255, cols - 1);
        s.sc = p.ws + n0 * KB;
        if (F != kBf16 && tid >= 256) {
            s.row = row_of(tid - 256);
            s.sc = p.xs + base * KB;
        }
        return s;
    };
    auto resolve = [&](Src& s) {
#pragma unroll
        for (int i = 0; i < XL; ++i) s.xo[i] = (uint32_t)((p.src_of ? s.xo[i] / (uint32_t)p.k : s.xo[i]) * xb) + xc * 16;
        s.sc += (int64_t)(F != kBf16 && tid >= 256 && p.src_of ? s.row / p.k : s.row) * KB;
    };
    auto issue = [&](const Src& s, int kt, int buf) {
        const uint32_t l0 = (uint32_t)(uintptr_t)(LDS_AS char*)(&s_ab[buf][0]) + wave * 1024;
        const uint32_t xk = (uint32_t)kt * 128, wk = (uint32_t)kt * SL::WROW;
        const bool xin = (int64_t)xk + xc * 16 < xb, win = (int)wk + wc * 16 < wb;  // past K: zeros
#pragma unroll
        for (int i = 0; i < XL; ++i) lds_copy16(s.rx, l0 + i * 8192, xin ? s.xo[i] + xk : kMasked);
#pragma unroll
        for (int i = 0; i < WL; ++i) lds_copy16(s.rw, l0 + XB + i * 8192, win ? wo + i * WR * (uint32_t)wb + wk : kMasked);
    };
    // Two groups of this thread's row of scales (1024 of K), zeros past its end, through registers, since rows
    // start at any byte. A thread's 16 bytes cost a line of their own, so a group at a time they were a third of all
    // line reads; three places hold the group in use and the next two.
    uint4 held[2];
    auto load_scales = [&](const Src& s, int at) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int n = min(16, KB - at - 16 * g);
            held[g] = make_uint4(0, 0, 0, 0);
            if (n == 16) {
                __builtin_memcpy(&held[g], s.sc + at + 16 * g, 16);
            } else if (n > 0) {
                uint32_t b[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (i < n) b[i >> 2] |= (uint32_t)s.sc[at + 16 * g + i] << (8 * (i & 3));
                held[g] = make_uint4(b[0], b[1], b[2], b[3]);
            }
        }
    };
    int t = logical(0);
    if (t >= total) return;
    Tile tl = get_tile(t);
    const int nk = (K + SL::KS - 1) / SL::KS;
    // The slabs of all this workgroup's tiles are one sequence; the next to copy:
    Src asrc = begin(tl);
    int akt = 0, around = 0, abuf = 0, aslot = 0, fetched = 0;  // groups of scales on their way
    bool amore = true;
    auto advance = [&]() {
        akt = 0;
        const int tn = logical(++around);
        amore = tn < total;
        if (amore) asrc = begin(get_tile(tn));
    };
    // its scales, where it begins a pair of groups
    auto fetch_scales = [&]() {
        if (kEarly && akt == nk) advance();
        if (!amore) return;
        if (akt == 0) resolve(asrc);
        if (akt % (2 * SL::SPG) == 0) {
            fetched = min(2, (nk - akt + SL::SPG - 1) / SL::SPG);
            if (scaled) load_scales(asrc, akt / SL::SPG * 16);
        }
    };
    auto store_scales = [&]() {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            if (g >= fetched) break;
            if (scaled) *(uint4*)(s_sc[aslot] + tid * 16) = held[g];
            aslot = aslot == 2 ? 0 : aslot + 1;
        }
        fetched = 0;
    };
    auto copy_slab = [&]() {
        if (!amore) return;
        issue(asrc, akt, abuf);
        abuf ^= 1;
        ++akt;
        if (!kEarly && akt == nk) advance();  // its rows' loads have a slab's time
    };
    auto barrier = [&]() {  // no wait for copies in it
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < 1 + kEarly; ++i) {
        fetch_scales();
        store_scales();
        copy_slab();
    }
    __builtin_amdgcn_s_waitcnt(0);
    barrier();
    int buf = 0, slot = 2, round = 0;
    // A tile whose wavefronts have NB blocks of 32 rows each, then its epilogue.
    auto tile = [&](auto Blocks) {
        constexpr int NB = decltype(Blocks)::value;
        int ln = lane;  // opaque, or the addresses of all forms are kept in registers over the tiles
        asm volatile("" : "+v"(ln));
        const int h = ln >> 5, lr = ln & 31;
        const int wrow = wn * 64 + lr, xrow = wm * 32 + lr;  // a wavefront's blocks of 32 rows: every other one
        f32x16_t acc[NB][2];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = (f32x16_t){};
        for (int kt = 0; kt < nk; ++kt) {
            // sent early, copies take the place of this slab, the tile's last one excepted: the epilogue's stage
            if (!kEarly || kt + 1 < nk) fetch_scales();
            const bool early = kEarly && kt + 1 < nk && amore;
            if (!kEarly) copy_slab();
            const int sub = kt % SL::SPG;
            if (sub == 0) slot = slot == 2 ? 0 : slot + 1;
            const uint8_t* sX = s_ab[buf];
            const uint8_t* sW = s_ab[buf] + XB;
            const uint8_t* sc = s_sc[slot] + sub * (SL::KS / 32);
            auto release = [&]() {  // once all have read their last fragments
                if (!early) return;
                __builtin_amdgcn_s_waitcnt(kWaitLgkmcnt0);
                barrier();
                store_scales();
                copy_slab();
            };
            if constexpr (F == kBf16) {
                // W's piece h of a row (K 32 h ..) is one scale block: step q takes its word q, X's piece 4 h + q
                uint4 fw[2];
                float fs[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    fw[j] = *(const uint4*)(sW + slab_byte<2>(wrow + 32 * j, h));
                    fs[j] = __uint_as_float((uint32_t)sc[(wrow + 32 * j) * 16 + h] << 23);  // its exponent alone is read
                }
                bf16x8_t fx[2][NB];
                auto load_x = [&](int q) {
#pragma unroll
                    for (int i = 0; i < NB; ++i) fx[q & 1][i] = *(const bf16x8_t*)(sX + slab_byte<8>(xrow + 64 * i, 4 * h + q));
                };
                load_x(0);
                static_for<4>([&](auto Q) {
                    if constexpr (Q < 3) load_x(Q + 1);
                    else if constexpr (kEarly) release();
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t word = Q == 0 ? fw[j].x : Q == 1 ? fw[j].y : Q == 2 ? fw[j].z : fw[j].w;
                        const bf16x8_t v = weights8(word, fs[j]);
#pragma unroll
                        for (int i = 0; i < NB; ++i)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, fx[Q & 1][i], acc[i][j], 0, 0, 0);
                    }
                    __builtin_amdgcn_sched_barrier(0);  // the compiler would put the loads off to their use
                });
            } else {
                constexpr int NS = SL::KS / 64;  // steps of 64
                // scale words of 128 of K, shifted by the lane half's block: byte 0 serves the word's first
                // step, byte 2 its second
                uint32_t ss[2][NS / 2], sx[NB][NS / 2];
#pragma unroll
                for (int u = 0; u < NS / 2; ++u) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) ss[j][u] = *(const uint32_t*)(sc + (wrow + 32 * j) * 16 + 4 * u) >> (8 * h);
#pragma unroll
                    for (int i = 0; i < NB; ++i) sx[i][u] = *(const uint32_t*)(sc + (256 + xrow + 64 * i) * 16 + 4 * u) >> (8 * h);
                }
                auto frag_w = [&](int j, int s) { return *(const uint4*)(sW + slab_byte<SL::WCH>(wrow + 32 * j, 2 * s + h)); };
                auto frag_x = [&](int i, int s) {
                    if constexpr (F == kMx4) return *(const uint4*)(sX + slab_byte<8>(xrow + 64 * i, 2 * s + h));
                    else return operand8(*(const uint4*)(sX + slab_byte<8>(xrow + 64 * i, 4 * s + h)),
                                         *(const uint4*)(sX + slab_byte<8>(xrow + 64 * i, 4 * s + 2 + h)));
                };
                uint4 fw[2];
                std::conditional_t<F == kMx4, uint4, i32x8_t> fx[NB];
                auto operand = [](auto v) {
                    if constexpr (F == kMx4) return operand4(v);
                    else return v;
                };
#pragma unroll
                for (int j = 0; j < 2; ++j) fw[j] = frag_w(j, 0);
#pragma unroll
                for (int i = 0; i < NB; ++i) fx[i] = frag_x(i, 0);
                static_for<NS>([&](auto S) {
                    constexpr bool more = S + 1 < NS;
                    if constexpr (!more && kEarly) release();
                    static_for<2>([&](auto J) {
                        static_for<NB>([&](auto I) {
                            acc[I][J] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                operand4(fw[J]), operand(fx[I]), acc[I][J], 4, F == kMx4 ? 4 : 0, 2 * (S & 1), (int)ss[J][S / 2], 2 * (S & 1),
                                (int)sx[I][S / 2]);
                            if constexpr (more && J == 1) fx[I] = frag_x(I, S + 1);
                        });
                        if constexpr (more) fw[J] = frag_w(J, S + 1);
                    });
                    __builtin_amdgcn_sched_barrier(0);  // or the sums move to other registers at the release
                });
            }
            // pinned before the wait below (the compiler would sink them past it)
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) asm volatile("" : "+v"(acc[i][j]));
            buf ^= 1;
            if (kt + 1 < nk) {
                // the next slab is here; one sent early may still be on its way
                if (early) __builtin_amdgcn_s_waitcnt(wait_vmcnt(XL + WL));
                else __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
                if (!kEarly) store_scales();
                __builtin_amdgcn_s_waitcnt(kWaitLgkmcnt0);
                barrier();
            }
        }
        // Epilogue: lane = row, columns 8 q + 4 h + s of each 32-wide tile; 32 rows at a time through this
        // wavefront's 4 KiB of the slab no longer read, so that stores cover whole rows.
        __syncthreads();  // the last slab is read out
        uint8_t* stg = &s_ab[buf ^ 1][0] + wave * 4096;
        with_act(p.act, [&](auto A) {
            constexpr int ACT = decltype(A)::value;
            if constexpr ((ACT < 2) == GLU) {
                const int NO = GLU ? p.N / 2 : p.N;
                constexpr int PC = GLU ? 4 : 8;  // 16-byte pieces a row
                const int col0 = (tl.n0 + wn * 64) / (GLU ? 2 : 1);
                static_for<NB>([&](auto I) {
                    static_for<GLU ? 1 : 2>([&](auto J) {
                        static_for<4>([&](auto Q) {
                            float o[4];
#pragma unroll
                            for (int s = 0; s < 4; ++s) {
                                o[s] = dense_act<ACT>(acc[I][J][4 * Q + s]);
                                if constexpr (GLU) o[s] *= acc[I][1][4 * Q + s];
                            }
                            *(uint2*)(stg + slab_byte<PC>(lr, 4 * J + Q) + 8 * h) =
                                make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
                        });
                    });
                    wave_lds_sync();
                    static_for<PC / 2>([&](auto It) {
                        const int R = It * (64 / PC) + ln / PC, c = ln % PC;
                        const uint4 v = *(const uint4*)(stg + slab_byte<PC>(R, c));
                        const int m = 64 * I + 32 * wm + R, col = col0 + 8 * c;
                        if (m < tl.rows && col < NO) st_nt16(p.y + (int64_t)(tl.row0 + m) * NO + col, v);
                    });
                    wave_lds_sync();
                });
            }
        });
    };
    for (;;) {
        // Experts' last tiles hold what is left of their rows: a quarter or half of the work where that is enough. Each
        // form passes the same barriers, so the wavefronts' halves need not take the same one.
        const int blocks = (tl.rows - 32 * wm + 63) / 64;
        if (blocks <= 1) tile(std::integral_constant<int, 1>{});
        else if (blocks <= 2 && TM > 2) tile(std::integral_constant<int, 2>{});
        else tile(std::integral_constant<int, TM>{});
        const int tn = logical(++round);
        if (tn >= total) break;
        tl = get_tile(tn);
        if (kEarly) fetch_scales();
        __builtin_amdgcn_s_waitcnt(0);
        if (!kEarly) store_scales();
        __syncthreads();  // the next tile's first slab is here, and the stage read out
        if (kEarly) {
            store_scales();
            copy_slab();
            __builtin_amdgcn_s_waitcnt(kWaitLgkmcnt0);
            barrier();
        }
    }
}

// ------------------------------------------------------------------ launch
// Which kernel, by the mean rows of an expert that has any (the counts are the device's; any choice is right). All of
// 32 experts of 7168 x 4096 with SwiGLU, us, 4-bit rows / bf16 rows (where the card's memory lands moves some by a tenth):
//   mean rows        8         16         32         48         64         96        128        256
//   rows, 16     90 / 105  123 / 172  213 / 318  298 / 463
//   rows, 32     92 / 123   97 / 156  149 / 277  203 / 392  257 / 514
//   tiles, 64    96 / 186   96 / 190   98 / 189  100 / 195  159 / 325  161 / 349  198 / 448  300 / 717
//   tiles, 128  105 / 217  106 / 225  106 / 232  108 / 237  112 / 237  114 / 246  168 / 360  234 / 540
//   tiles, 256  111 / 226  111 / 235  112 / 243  114 / 247  116 / 249  121 / 263  130 / 296  205 / 480
// (64 rows stop paying where most experts have more.)
// Few tiles leave compute units idle: then smaller ones (1024 tokens x 2 of 8 experts, 2048 x 2048, 8-bit rows: 256 rows 31,
// 128 rows 25, 64 rows 31 us), or the other kernel, which has four times the workgroups (512 tokens x 1 of 4,
// 1024 x 1024, bf16: 10.3 against 15.0 us of 64 rows). Its wavefronts split K in eight instead of four where columns and
// experts give fewer workgroups than compute units (with more, four are faster: one token, 8 of 32, 2048 x 7168: 16.0
// against 22.5 us).
template <int F>
static void experts4_any(const Experts4Args& a, int T, int k, hipStream_t s) {
    using std::integral_constant;
    const int64_t pairs = (int64_t)T * k;
    const int active = (int)std::min<int64_t>(a.E, pairs);
    const double mean = (double)pairs / active;
    const int64_t ntn = (a.N + 255) / 256;
    auto filled = [&](int bm) { return ((int64_t)mean + bm - 1) / bm * active * ntn; };  // tiles of bm rows
    int bm = mean <= 50 ? 64 : mean <= 110 ? 128 : 256;
    while (bm > 64 && filled(bm) < 128) bm /= 2;
    auto rows = [&](auto R, auto W) {
        constexpr int RT = decltype(R)::value, NW = decltype(W)::value;
        const dim3 grid((a.N + 63) / 64, active, (unsigned)((std::min(T, (int)(2 * mean + 1)) + 16 * RT - 1) / (16 * RT)));
        experts4_rows_kernel<F, RT, NW><<<grid, NW * 64, 0, s>>>(a);
    };
    auto tiles = [&](auto B) {
        constexpr int BMX = decltype(B)::value;
        const int64_t bound = (pairs / BMX + active) * ntn;
        const int grid = persistent_grid(bound);
        if (a.act < 2) experts4_tile_kernel<F, BMX, true><<<grid, 512, 0, s>>>(a);
        else experts4_tile_kernel<F, BMX, false><<<grid, 512, 0, s>>>(a);
    };
    if (mean <= 10 || T <= 16) {
        if ((int64_t)active * ((a.N + 63) / 64) <= 256) rows(integral_constant<int, 1>{}, integral_constant<int, 8>{});
        else rows(integral_constant<int, 1>{}, integral_constant<int, 4>{});
    } else if (mean <= 24 || filled(64) < 128) {
        rows(integral_constant<int, 2>{}, integral_constant<int, 4>{});
    } else if (bm == 64) {
        tiles(integral_constant<int, 64>{});
    } else if (bm == 128) {
        tiles(integral_constant<int, 128>{});
    } else {
        tiles(integral_constant<int, 256>{});
    }
}

int launch_experts4(const Experts4Call& c, hipStream_t s) {
    Experts4Args a{};
    a.x = (const uint8_t*)c.x, a.xs = c.x_s, a.src_of = c.src_of, a.k = c.k, a.rows = c.src_of ? c.T : c.M_cap;
    a.wq = c.w_q, a.ws = c.w_s, a.offsets = c.offsets, a.counts = c.counts;
    a.E = c.E, a.N = c.N, a.K = c.K, a.act = c.act, a.y = c.y;
    if (c.fmt == kBf16) experts4_any<kBf16>(a, c.T, c.k, s);
    else if (c.fmt == kMx8) experts4_any<kMx8>(a, c.T, c.k, s);
    else experts4_any<kMx4>(a, c.T, c.k, s);
    return hipGetLastError() == hipSuccess ? 0 : -4;
}

}  // namespace moe
