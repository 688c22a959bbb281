// Dense linear layer on gfx950 bf16 MFMA (v_mfma_f32_32x32x16_bf16): the router
// projection and the shared expert that run beside the routed experts.
//
//   forward  y  = f(x W + b) + r     A = x [T, K] K-major,  B = W [K, N] N-major
//   dgrad    dx = dz W^T + r         A = dz [T, N] K-major, B = W read along its rows, K-major
//   wgrad    dw = x^T dz (+ dw)      A = x, B = dz, both with the reduction (tokens) outermost
//
// One kernel template: a workgroup owns a BM x BN tile, its wavefronts 32 TM x
// 64 pieces of it (fp32 accumulators in the MFMA layout); K moves in slabs of 64
// through ST LDS stages filled by direct global -> LDS copies. With ST = 2 the kernel
// is persistent; with ST = 3 or 4 a workgroup has one tile and keeps two or three slabs
// on their way, which hides the copies' latency where no second workgroup shares the
// compute unit. Buffer bounds turn everything past the matrices' rows into zeros and a
// lane whose columns lie past the end uses an offset past every buffer, so any T >= 1
// and any K, N that are multiples of 8 take the same path.
//
// The epilogue adds the bias to the fp32 accumulators (z), optionally stores z as
// bf16 or as MXFP8 codes of its bf16 value, applies the activation to the fp32 z,
// adds the residual and rounds once.
//
// Bounds: the matrix cores at the clock that the power allows where tiles fill the chip
// (forward 32768 x 8192 x 4096 SwiGLU with 8-bit z 1716 us, 1282 TFLOP/s, 71% of the MFMA
// cycles at 1.72 GHz, where the vendor library's bare product takes 1653; dgrad and wgrad
// 16384 x 7168 x 4096 738 and 838 us, 631 and 1030 there); the wait for slab copies with
// one or two workgroups a compute unit (1000 x 2880 x 5760 GeGLU 47 us, 27% of the MFMA
// cycles); the read of W with few rows (the small products below).
#include <algorithm>

#include "dense_common.hpp"

namespace moe {

struct DenseArgs {
    const uint16_t* A;
    int64_t lda;
    const uint8_t* a_q;  // A as an 8-bit checkpoint instead: codes [K, M], scales [K, M / 32]
    const uint8_t* a_s;
    const uint16_t* B;
    int64_t ldb;
    int M, N, K;  // rows and columns of the product, reduction length
    int ntm, ntn;
    int splits, split_slabs;  // K slabs per split
    const uint16_t* bias;     // [N] or nullptr
    const uint16_t* res;      // [M, NO] or nullptr (NO: columns of the output)
    void* out;                // [M, NO] bf16, or fp32 when out_f32
    int out_f32, accumulate;
    uint16_t* z;   // [M, N] or nullptr
    uint8_t* z_q;  // [M, N] codes, [M, N / 32] scales, or nullptr
    uint8_t* z_s;
    float* part;  // [splits, M, N] raw sums instead of an epilogue, or nullptr
    // with tail_splits > 1: tiles from tail_first on have K cut into tail_splits pieces of
    // tail_slabs, whose raw sums go to part as [piece][tile - tail_first][rows, columns]
    int tail_first, tail_splits, tail_slabs;
    int stream;   // outputs past the caches
};

__device__ __forceinline__ void dense_st16(bool stream, void* at, uint4 v) {
    if (stream) st_nt16(at, v);
    else *(uint4*)at = v;
}

template <int ACT>
constexpr bool kGated = ACT == 0 || ACT == 1;

// 16-byte chunk swizzle of row k in an MN-major slab of W columns: a transpose
// read touches 4 neighbouring k rows, 64 bytes each; the XOR spreads them over
// the four 64-byte quarters of LDS's 256-byte bank window.
template <int W>
__device__ __forceinline__ int mn_swz(int k) {
    if constexpr (W == 256) return (k & 7) << 2;
    else return (k & 3) << 2;
}

// Row-wise MXFP8 block of a 32 x 32 block held the MFMA way, as mx_rowq32, for
// rows that may lie past the matrix: every lane takes part in the exchanges and
// only the lanes of a real row store.
__device__ __forceinline__ void mx_rowq32_if(const uint32_t pk[8], int lane, bool ok, uint8_t* q, uint8_t* sc) {
    uint32_t am = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) am = max_u16x2(am, pk[r] & 0x7fff7fffu);
    uint32_t amax = max(am & 0xffffu, am >> 16);
    amax = max(amax, (uint32_t)__shfl_xor((int)amax, 32, 64));
    const int e = mx_block_exp(amax);
    const float inv = mx_inv_scale(e);
    uint32_t w[4];
#pragma unroll
    for (int Q = 0; Q < 4; ++Q)
        w[Q] = e4m3x4(bf16_lo(pk[2 * Q]) * inv, bf16_hi(pk[2 * Q]) * inv, bf16_lo(pk[2 * Q + 1]) * inv,
                      bf16_hi(pk[2 * Q + 1]) * inv);
    const int h = (lane >> 5) & 1;
    const uint32_t g0 = h ? w[0] : w[2], g1 = h ? w[1] : w[3];
    const auto s0 = __builtin_amdgcn_permlane32_swap(g0, g0, false, false);
    const auto s1 = __builtin_amdgcn_permlane32_swap(g1, g1, false, false);
    const uint32_t r0 = h ? s0[0] : s0[1], r1 = h ? s1[0] : s1[1];
    if (ok) {
        *(uint4*)(q + 16 * h) = h ? make_uint4(r0, w[2], r1, w[3]) : make_uint4(w[0], r0, w[1], r1);
        if (h == 0) *sc = (uint8_t)(e + 127);
    }
}

// 8 output values v of row m, columns [col, col + 8): residual, accumulation, one rounding.
__device__ __forceinline__ void dense_store8(const DenseArgs& p, int64_t at, float* v) {
    if (p.res) {
        const uint4 r = *(const uint4*)(p.res + at);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] += bf16_lo(w[i]);
            v[2 * i + 1] += bf16_hi(w[i]);
        }
    }
    if (p.out_f32) {
        float4* o = (float4*)((float*)p.out + at);
        if (p.accumulate) {
            const float4 a = o[0], b = o[1];
            v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
            v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
        }
        dense_st16(p.stream, o, __builtin_bit_cast(uint4, make_float4(v[0], v[1], v[2], v[3])));
        dense_st16(p.stream, o + 1, __builtin_bit_cast(uint4, make_float4(v[4], v[5], v[6], v[7])));
    } else {
        dense_st16(p.stream, (uint16_t*)p.out + at,
                   make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                              pack_bf16x2(v[6], v[7])));
    }
}

// 16 columns of an 8-bit checkpoint's row on their way into an LDS slab: codes and
// scale in registers, then two 16-byte pieces of bf16 (exact: 4 significant bits).
struct Codes16 {
    uint4 q;
    uint32_t s;
};
__device__ __forceinline__ Codes16 codes16_load(const DenseArgs& p, int64_t row, int col) {
    Codes16 c{make_uint4(0, 0, 0, 0), 127};
    if (row < p.K && col < p.M) {
        c.q = *(const uint4*)(p.a_q + row * p.lda + col);
        c.s = p.a_s[row * (p.lda / 32) + col / 32];
    }
    return c;
}
__device__ __forceinline__ void codes16_store(const Codes16& c, uint8_t* lo, uint8_t* hi) {
    const float sc = e8m0_value(c.s);
    float v[16];
    e4m3x4_value(c.q.x, sc, v);
    e4m3x4_value(c.q.y, sc, v + 4);
    e4m3x4_value(c.q.z, sc, v + 8);
    e4m3x4_value(c.q.w, sc, v + 12);
    *(uint4*)lo = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                             pack_bf16x2(v[6], v[7]));
    *(uint4*)hi = make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]),
                             pack_bf16x2(v[14], v[15]));
}

// Wait until at most N vector-memory operations are in flight and every LDS
// operation has completed, then the workgroup barrier.
template <int N>
__device__ __forceinline__ void wait_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// The epilogue's other form: the raw sums of a piece of K, to `out` [row][col] of row
// length `ld`.
template <int TM, int TN>
__device__ __forceinline__ void dense_raw_sums(const DenseArgs& p, f32x16_t (&acc)[TM][TN], uint8_t* stg, float* out,
                                               int64_t ld, int mb, int col0, int lane) {
    const int h = lane >> 5, r = lane & 31;
    static_for<TM>([&](auto I) {
        if (mb + 32 * I >= p.M) return;
        static_for<TN>([&](auto J) {
            static_for<4>([&](auto Q) {
                const int ch = 8 * J + 2 * Q + h;
                *(float4*)(stg + r * 256 + ((ch ^ (r & 15)) << 4)) = make_float4(
                    acc[I][J][4 * Q], acc[I][J][4 * Q + 1], acc[I][J][4 * Q + 2], acc[I][J][4 * Q + 3]);
            });
        });
        wave_lds_sync();
        static_for<8>([&](auto It) {
            const int R = 4 * It + (lane >> 4), c = lane & 15;
            const float4 v = *(const float4*)(stg + R * 256 + ((c ^ (R & 15)) << 4));
            const int m = mb + 32 * I + R, col = col0 + 4 * c;
            if (m < p.M && col < p.N) *(float4*)(out + (int64_t)m * ld + col) = v;
        });
        wave_lds_sync();
    });
}

// The epilogue of one wavefront's piece of a tile. Lane l holds row l & 31 of each 32
// x 32 block and, in register 4 Q + s, column 8 Q + 4 h + s, h = l >> 5. Values leave
// through the wavefront's 8 KiB of the LDS stage `stg` that the tile no longer reads
// (the next tile's first slab goes to the other one), so that a store instruction
// covers whole row runs; 16-byte chunks are XOR-swizzled by the row.
template <int DBM, int DBN, int WMW, int WNW, int TM, int TN, int ACT, bool TAIL>
__device__ __forceinline__ void dense_epilogue(const DenseArgs& p, f32x16_t (&acc)[TM][TN], uint8_t* stg, int m0,
                                               int n0, int split, int tail, int wm, int wn, int lane) {
    // every wavefront has read the last slab out of the stage
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
    const int h = lane >> 5, r = lane & 31;
    const int col0 = n0 + wn * 64;
    if (col0 >= p.N) return;
    const int mb0 = m0 + wm * 32 * TM;
    if (TAIL && tail >= 0)
        return dense_raw_sums(p, acc, stg, p.part + (int64_t)tail * DBM * DBN - ((int64_t)m0 * DBN + n0), DBN, mb0,
                              col0, lane);
    if (ACT == 3 && p.splits > 1)
        return dense_raw_sums(p, acc, stg, p.part + (int64_t)split * p.M * p.N, p.N, mb0, col0, lane);
    const int NO = kGated<ACT> ? p.N / 2 : p.N;
    static_for<TM>([&](auto I) {
        const int mb = mb0 + 32 * I;
        if (mb >= p.M) return;
        if (p.bias) {
            static_for<TN>([&](auto J) {
                static_for<4>([&](auto Q) {
                    const int col = col0 + 32 * J + 8 * Q + 4 * h;
                    if (col < p.N) {
                        float b[4];
                        unpack_bf16x4(*(const uint2*)(p.bias + col), b);
#pragma unroll
                        for (int s = 0; s < 4; ++s) acc[I][J][4 * Q + s] += b[s];
                    }
                });
            });
        }
        if (ACT != 3 && (p.z || p.z_q)) {
            uint32_t pk[TN][8];
            static_for<TN>([&](auto J) {
                static_for<8>([&](auto R8) { pk[J][R8] = pack_bf16x2(acc[I][J][2 * R8], acc[I][J][2 * R8 + 1]); });
            });
            if (p.z_q) {
                static_for<TN>([&](auto J) {
                    const int cb = col0 + 32 * J;
                    if (cb < p.N)
                        mx_rowq32_if(pk[J], lane, mb + r < p.M, p.z_q + (int64_t)(mb + r) * p.N + cb,
                                     p.z_s + (int64_t)(mb + r) * (p.N / 32) + cb / 32);
                });
            }
            if (p.z) {
                static_for<TN>([&](auto J) {
                    static_for<4>([&](auto Q) {
                        const int ch = 4 * J + Q;
                        *(uint2*)(stg + r * 128 + ((ch ^ ((r >> 1) & 7)) << 4) + 8 * h) =
                            make_uint2(pk[J][2 * Q], pk[J][2 * Q + 1]);
                    });
                });
                wave_lds_sync();
                static_for<4>([&](auto It) {
                    const int R = 8 * It + (lane >> 3), c = lane & 7;
                    const uint4 v = *(const uint4*)(stg + R * 128 + ((c ^ ((R >> 1) & 7)) << 4));
                    const int m = mb + R, col = col0 + 8 * c;
                    if (m < p.M && col < p.N) dense_st16(p.stream, p.z + (int64_t)m * p.N + col, v);
                });
                wave_lds_sync();
            }
        }
        if constexpr (kGated<ACT>) {
            static_for<4>([&](auto Q) {
                float v[4];
#pragma unroll
                for (int s = 0; s < 4; ++s) v[s] = dense_act<ACT>(acc[I][0][4 * Q + s]) * acc[I][1][4 * Q + s];
                const int ch = 2 * Q + h;
                *(float4*)(stg + r * 128 + ((ch ^ (r & 7)) << 4)) = make_float4(v[0], v[1], v[2], v[3]);
            });
            wave_lds_sync();
            static_for<2>([&](auto It) {
                const int R = 16 * It + (lane >> 2), c = lane & 3;
                float v[8];
                *(float4*)v = *(const float4*)(stg + R * 128 + (((2 * c) ^ (R & 7)) << 4));
                *(float4*)(v + 4) = *(const float4*)(stg + R * 128 + (((2 * c + 1) ^ (R & 7)) << 4));
                const int m = mb + R;
                if (m < p.M) dense_store8(p, (int64_t)m * NO + col0 / 2 + 8 * c, v);
            });
        } else {
            static_for<TN>([&](auto J) {
                static_for<4>([&](auto Q) {
                    float v[4];
#pragma unroll
                    for (int s = 0; s < 4; ++s) v[s] = dense_act<ACT>(acc[I][J][4 * Q + s]);
                    const int ch = 8 * J + 2 * Q + h;
                    *(float4*)(stg + r * 256 + ((ch ^ (r & 15)) << 4)) = make_float4(v[0], v[1], v[2], v[3]);
                });
            });
            wave_lds_sync();
            static_for<4>([&](auto It) {
                const int R = 8 * It + (lane >> 3), c = lane & 7;
                float v[8];
                *(float4*)v = *(const float4*)(stg + R * 256 + (((2 * c) ^ (R & 15)) << 4));
                *(float4*)(v + 4) = *(const float4*)(stg + R * 256 + (((2 * c + 1) ^ (R & 15)) << 4));
                const int m = mb + R, col = col0 + 8 * c;
                if (m < p.M && col < p.N) dense_store8(p, (int64_t)m * NO + col, v);
            });
        }
        wave_lds_sync();
    });
}

template <int DBM, int DBN, int WMW, int WNW, int ST, bool A_KMAJ, bool B_KMAJ, int ACT, bool TAIL = false>
__global__ void __launch_bounds__(WMW * WNW * 64, ST > 2 ? 1 : 2) dense_gemm_kernel(DenseArgs p) {
    constexpr int NT = WMW * WNW * 64;
    constexpr int TM = DBM / (32 * WMW), TN = DBN / (32 * WNW);
    static_assert(TN == 2, "a wavefront owns 64 columns: 32 gate and 32 up columns of a gated layer");
    constexpr int ABYTES = DBM * 128, STAGE = (DBM + DBN) * 128;
    constexpr int LA = ABYTES / (NT * 16), LB = (STAGE - ABYTES) / (NT * 16);
    static_assert((ST == 2 ? 1 : ST) * STAGE >= WMW * WNW * 8192,
                  "the epilogue stages 8 KiB per wavefront, in one LDS stage where the next tile fills the other");
    __shared__ __attribute__((aligned(1024))) uint8_t s_ab[ST * STAGE];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WNW, wn = wave % WNW;

    // Tiles: splits outermost, then bands of 4 M tiles with the M tiles inner. The
    // kernel is persistent: round r covers tiles [r nb, (r + 1) nb), of which each XCD
    // (workgroups are dealt round robin to 8) takes a contiguous eighth, so that its
    // L2 holds a window's operand panels.
    // TAIL: a last round that would leave many compute units idle has its tiles' K cut
    // into pieces instead. A form of its own: with the raw sums' branch in it the
    // epilogue spills up to 34 registers (SwiGLU 32768 x 8192 x 4096: 1840 us, 1800).
    const int per = p.ntm * p.ntn;
    const int total = TAIL ? p.tail_first + (per - p.tail_first) * p.tail_splits : per * p.splits;
    const int nb = gridDim.x;  // a multiple of 8
    const int first = (blockIdx.x & 7) * (nb >> 3) + (blockIdx.x >> 3);
    const int slabs = (p.K + DBK - 1) / DBK;
    struct Tile {
        int m0, n0, split, tail, ks0, nk;
    };
    auto get_tile = [&](int tt) -> Tile {
        Tile tl;
        int t, each = p.split_slabs;
        if (TAIL) {
            const int v = tt - p.tail_first, rem = per - p.tail_first;
            tl.tail = v < 0 ? -1 : v;
            tl.split = v < 0 ? 0 : __builtin_amdgcn_readfirstlane(v / rem);
            t = v < 0 ? tt : p.tail_first + v - tl.split * rem;
            if (v >= 0) each = p.tail_slabs;
        } else {
            tl.tail = -1;
            tl.split = __builtin_amdgcn_readfirstlane(tt / per);
            t = tt - tl.split * per;
        }
        const int band = t / (4 * p.ntn), within = t - band * 4 * p.ntn;
        const int bm = min(4, p.ntm - band * 4);
        tl.m0 = __builtin_amdgcn_readfirstlane((band * 4 + within % bm) * DBM);
        tl.n0 = __builtin_amdgcn_readfirstlane((within / bm) * DBN);
        tl.ks0 = tl.split * each;
        tl.nk = min(each, slabs - tl.ks0);
        return tl;
    };

    // Operand sources: a 64-bit base per slab, 32-bit lane offsets inside it. Copy i
    // of the workgroup fills LDS chunks [i NT, (i + 1) NT) of 16 bytes in thread
    // order; each lane fetches whichever global chunk the swizzled layout has there.
    struct Src {
        const char* a_base;
        const char* b_base;
        int64_t a_bytes, b_bytes;
        uint32_t a_off, b_off;
    };
    constexpr int ACPR = A_KMAJ ? 8 : DBM / 8, BCPR = B_KMAJ ? 8 : DBN / 8;  // chunks per slab row
    const int a_r = tid / ACPR, b_r = tid / BCPR;
    const int a_c = (tid % ACPR) ^ (A_KMAJ ? kmaj_swz(a_r) : mn_swz<DBM>(a_r));
    const int b_c = (tid % BCPR) ^ (B_KMAJ ? kmaj_swz(b_r) : mn_swz<DBN>(b_r));
    const int64_t a_step = A_KMAJ ? DBK * 2 : (int64_t)DBK * p.lda * 2;
    const int64_t b_step = B_KMAJ ? DBK * 2 : (int64_t)DBK * p.ldb * 2;
    const uint32_t a_istep = (uint32_t)(NT / ACPR * p.lda * 2), b_istep = (uint32_t)(NT / BCPR * p.ldb * 2);
    auto make_src = [&](const Tile& tl) -> Src {
        Src sr;
        if constexpr (A_KMAJ) {
            sr.a_base = (const char*)(p.A + (int64_t)tl.m0 * p.lda);
            sr.a_bytes = (int64_t)min(p.M - tl.m0, DBM) * p.lda * 2;
            sr.a_off = (uint32_t)((a_r * p.lda + a_c * 8) * 2);
        } else {
            const int col = tl.m0 + a_c * 8;
            sr.a_base = (const char*)p.A;
            sr.a_bytes = (int64_t)p.K * p.lda * 2;
            sr.a_off = col < p.M ? (uint32_t)((a_r * p.lda + col) * 2) : kMasked;
        }
        if constexpr (B_KMAJ) {
            sr.b_base = (const char*)(p.B + (int64_t)tl.n0 * p.ldb);
            sr.b_bytes = (int64_t)min(p.N - tl.n0, DBN) * p.ldb * 2;
            sr.b_off = (uint32_t)((b_r * p.ldb + b_c * 8) * 2);
        } else {
            const int col = tl.n0 + b_c * 8;
            sr.b_base = (const char*)p.B;
            sr.b_bytes = (int64_t)p.K * p.ldb * 2;
            sr.b_off = col < p.N ? (uint32_t)((b_r * p.ldb + col) * 2) : kMasked;
        }
        return sr;
    };
    const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS_AS char*)&s_ab[0] + wave * 1024;
    // K slab `ks` (of the whole reduction) into LDS stage `st`: the A copies, the B
    // copies. In a last slab that ends inside, a K-major lane past K fetches nothing
    // (zeros); an operand with K outermost ends at its last row by the buffer bound.
    auto issue_a = [&](const Src& sr, int ks, int st) {
        const i32x4_t r = rsrc_from(sr.a_base, sr.a_bytes, (int64_t)ks * a_step);
        const bool out = A_KMAJ && a_c * 8 >= p.K - ks * DBK;
#pragma unroll
        for (int i = 0; i < LA; ++i)
            lds_copy16(r, lds0 + st * STAGE + i * NT * 16, out ? kMasked : sr.a_off + i * a_istep);
    };
    auto issue_b = [&](const Src& sr, int ks, int st) {
        const i32x4_t r = rsrc_from(sr.b_base, sr.b_bytes, (int64_t)ks * b_step);
        const bool out = B_KMAJ && b_c * 8 >= p.K - ks * DBK;
#pragma unroll
        for (int i = 0; i < LB; ++i)
            lds_copy16(r, lds0 + st * STAGE + ABYTES + i * NT * 16, out ? kMasked : sr.b_off + i * b_istep);
    };

    // MFMA operand of a 32-row (or 32-column) piece at K step ks: lane l holds index
    // l & 31 and k = 16 ks + 8 (l >> 5) + [0, 8)
    auto frag = [&](const uint8_t* s, auto KM, auto W, int base, int ks) -> bf16x8_t {
        if constexpr (decltype(KM)::value) {
            const int r = base + (lane & 31);
            return __builtin_bit_cast(bf16x8_t, *(const uint4*)(s + kmaj_byte(r, 2 * ks + (lane >> 5))));
        } else {
            constexpr int w = decltype(W)::value;
            const int lg = lane & 15;
            const int c = base + 16 * ((lane >> 4) & 1) + 4 * (lg & 3);
            const int k0 = 16 * ks + 8 * (lane >> 5) + (lg >> 2);
            const int o0 = k0 * (2 * w) + (((c >> 3) ^ mn_swz<w>(k0)) << 4) + (c & 7) * 2;
            const int k1 = k0 + 4;
            const int o1 = k1 * (2 * w) + (((c >> 3) ^ mn_swz<w>(k1)) << 4) + (c & 7) * 2;
            const bf16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LDS_AS bf16x4_t*)(s + o0));
            const bf16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LDS_AS bf16x4_t*)(s + o1));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };
    auto fragA = [&](int st, int i, int ks) {
        return frag(s_ab + st * STAGE, std::bool_constant<A_KMAJ>{}, std::integral_constant<int, DBM>{},
                    wm * 32 * TM + 32 * i, ks);
    };
    auto fragB = [&](int st, int j, int ks) {
        return frag(s_ab + st * STAGE + ABYTES, std::bool_constant<B_KMAJ>{}, std::integral_constant<int, DBN>{},
                    wn * 64 + 32 * j, ks);
    };
    bf16x8_t fa[2][TM], fb[2][TN];
    // the first MFMA row's operands; the other A fragments follow behind its MFMAs
    auto load_row0 = [&](int set, int st, int ks) {
        fb[set][0] = fragB(st, 0, ks);
        fa[set][0] = fragA(st, 0, ks);
        fb[set][1] = fragB(st, 1, ks);
    };
    f32x16_t acc[TM][TN];

    int tt = first;
    if (tt >= total) return;
    Tile tl = get_tile(tt);
    Src src = make_src(tl);
    int st = 0;  // LDS stage of the current slab
    issue_a(src, tl.ks0, 0);
    issue_b(src, tl.ks0, 0);
    if constexpr (ST > 2) {  // one tile per workgroup: its first slabs at once
        for (int k = 1; k < ST - 1 && k < tl.nk; ++k) {
            issue_a(src, tl.ks0 + k, k);
            issue_b(src, tl.ks0 + k, k);
        }
    }
    // wait for slab kt, leaving the copies of the slabs behind it in flight
    auto wait_slab = [&](int kt) {
        const int behind = min(ST - 2, tl.nk - 1 - kt);
        if (behind >= 2) wait_barrier<2 * (LA + LB)>();
        else if (behind == 1) wait_barrier<LA + LB>();
        else wait_barrier<0>();
    };
    for (;;) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = (f32x16_t){};
        // the next tile's first slab is fetched during this one's last
        const int tn = tt + nb;
        const bool have_next = ST == 2 && tn < total;
        Tile tl_next = tl;
        Src src_next = src;
        if (have_next) {
            tl_next = get_tile(tn);
            src_next = make_src(tl_next);
        }
        if constexpr (ST == 2) wait_barrier<0>();
        else wait_slab(0);  // the first slab has landed, the previous tile's staging is read out
        load_row0(0, st, 0);
        for (int kt = 0; kt < tl.nk; ++kt) {
            const bool last = kt + 1 == tl.nk;
            static_for<DBK / 16>([&](auto KS) {
                constexpr int ks = KS, c = ks & 1;
                // After the barrier all wavefronts ask LDS for fragments at once: only
                // the first row's operands go first, the rest and the next step's
                // behind its MFMAs; the next slab's A and B copies in two steps.
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[0][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[c][j], fa[c][0], acc[0][j], 0, 0, 0);
                if constexpr (ks == 0) {
#pragma unroll
                    for (int i = 1; i < TM; ++i) fa[0][i] = fragA(st, i, 0);
                }
                if constexpr (ks + 1 < DBK / 16) {
                    load_row0(c ^ 1, st, ks + 1);
#pragma unroll
                    for (int i = 1; i < TM; ++i) fa[c ^ 1][i] = fragA(st, i, ks + 1);
                }
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    acc[1][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[c][j], fa[c][1], acc[1][j], 0, 0, 0);
                if constexpr (ks == 0) {
                    if constexpr (ST == 2) {
                        if (!last) issue_a(src, tl.ks0 + kt + 1, st ^ 1);
                        else if (have_next) issue_a(src_next, tl_next.ks0, st ^ 1);
                    } else if (kt + ST - 1 < tl.nk) {
                        issue_a(src, tl.ks0 + kt + ST - 1, st == 0 ? ST - 1 : st - 1);  // the stage left last
                    }
                }
                if constexpr (ks == 1) {
                    if constexpr (ST == 2) {
                        if (!last) issue_b(src, tl.ks0 + kt + 1, st ^ 1);
                        else if (have_next) issue_b(src_next, tl_next.ks0, st ^ 1);
                    } else if (kt + ST - 1 < tl.nk) {
                        issue_b(src, tl.ks0 + kt + ST - 1, st == 0 ? ST - 1 : st - 1);  // the stage left last
                    }
                }
#pragma unroll
                for (int i = 2; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[c][j], fa[c][i], acc[i][j], 0, 0, 0);
                __builtin_amdgcn_s_setprio(0);
            });
            const int next = ST == 2 ? st ^ 1 : st + 1 == ST ? 0 : st + 1;
            if (!last) {
                if constexpr (ST == 2) wait_barrier<0>();
                else wait_slab(kt + 1);
                load_row0(0, next, 0);
            }
            st = next;
        }
        dense_epilogue<DBM, DBN, WMW, WNW, TM, TN, ACT, TAIL>(p, acc, s_ab + (ST == 2 ? st ^ 1 : 0) * STAGE + wave * 8192,
                                                              tl.m0, tl.n0, tl.split, tl.tail, wm, wn, lane);
        if (!have_next) break;
        tt = tn;
        tl = tl_next;
        src = src_next;
    }
}

// The epilogue on 8 columns of the output held by one thread: v[0] their sums over
// K (gated: v[0] the gate and v[1] the up columns); g counts groups of 8 output
// columns. With z_q, the 4 threads of a 32-column block are 4 neighbouring lanes.
template <int ACT>
__device__ __forceinline__ void dense_finish8(const DenseArgs& p, int64_t m, int g, float (*v)[8]) {
    constexpr int H = kGated<ACT> ? 2 : 1;
    const int NO = kGated<ACT> ? p.N / 2 : p.N;
    const int c0 = kGated<ACT> ? (g >> 2) * 64 + (g & 3) * 8 : g * 8;
#pragma unroll
    for (int u = 0; u < H; ++u) {
        const int col = c0 + 32 * u;
        if (p.bias) {
            float b[8];
            const uint4 w = *(const uint4*)(p.bias + col);
            unpack_bf16x4(make_uint2(w.x, w.y), b);
            unpack_bf16x4(make_uint2(w.z, w.w), b + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] += b[i];
        }
        if (ACT != 3 && (p.z || p.z_q)) {
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pk[i] = pack_bf16x2(v[u][2 * i], v[u][2 * i + 1]);
            if (p.z) *(uint4*)(p.z + m * p.N + col) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            if (p.z_q) {
                uint32_t am = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) am = max_u16x2(am, pk[i] & 0x7fff7fffu);
                uint32_t amax = max(am & 0xffffu, am >> 16);
                amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1, 64));
                amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2, 64));
                const int e = mx_block_exp(amax);
                const float inv = mx_inv_scale(e);
                uint2 q;
                q.x = e4m3x4(bf16_lo(pk[0]) * inv, bf16_hi(pk[0]) * inv, bf16_lo(pk[1]) * inv, bf16_hi(pk[1]) * inv);
                q.y = e4m3x4(bf16_lo(pk[2]) * inv, bf16_hi(pk[2]) * inv, bf16_lo(pk[3]) * inv, bf16_hi(pk[3]) * inv);
                *(uint2*)(p.z_q + m * p.N + col) = q;
                if ((g & 3) == 0) p.z_s[m * (p.N / 32) + col / 32] = (uint8_t)(e + 127);
            }
        }
    }
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (kGated<ACT>) y[i] = dense_act<ACT>(v[0][i]) * v[1][i];
        else y[i] = dense_act<ACT>(v[0][i]);
    }
    dense_store8(p, m * NO + 8 * g, y);
}

// Joins the K splits. A thread adds the partial sums of 8 output columns over every
// L-th split; the L lanes' sums meet in LDS, lane order; then the epilogue. L = 8
// where there are few outputs (one row), so that the splits' loads run side by side.
template <int ACT, int L>
__global__ void __launch_bounds__(256) dense_join_kernel(DenseArgs p) {
    constexpr int H = kGated<ACT> ? 2 : 1;
    constexpr int GB = 256 / L;  // groups per workgroup
    __shared__ float s_v[L > 1 ? L : 1][L > 1 ? GB * (8 * H + 1) : 1];
    const int ng = (kGated<ACT> ? p.N / 2 : p.N) / 8;
    const int gi = threadIdx.x % GB, l = threadIdx.x / GB;
    const int64_t idx = (int64_t)blockIdx.x * GB + gi;
    const bool on = idx < (int64_t)p.M * ng;  // with z_q: whole groups of 4 threads, ng % 4 == 0
    const int64_t m = on ? idx / ng : 0;
    const int g = on ? (int)(idx - m * ng) : 0;
    const int c0 = kGated<ACT> ? (g >> 2) * 64 + (g & 3) * 8 : g * 8;
    float v[2][8];
#pragma unroll
    for (int u = 0; u < H; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
    if (on) {
        const float* base = p.part + m * p.N + c0;
        const int64_t step = (int64_t)p.M * p.N;
#pragma unroll 4
        for (int s = l; s < p.splits; s += L) {
#pragma unroll
            for (int u = 0; u < H; ++u) {
                const float4* q = (const float4*)(base + s * step + 32 * u);
                const float4 a = q[0], b = q[1];
                v[u][0] += a.x, v[u][1] += a.y, v[u][2] += a.z, v[u][3] += a.w;
                v[u][4] += b.x, v[u][5] += b.y, v[u][6] += b.z, v[u][7] += b.w;
            }
        }
    }
    if constexpr (L > 1) {
#pragma unroll
        for (int i = 0; i < 8 * H; ++i) s_v[l][gi * (8 * H + 1) + i] = v[i >> 3][i & 7];
        __syncthreads();
        if (l > 0) return;
#pragma unroll
        for (int i = 0; i < 8 * H; ++i)
#pragma unroll
            for (int k = 1; k < L; ++k) v[i >> 3][i & 7] += s_v[k][gi * (8 * H + 1) + i];
    }
    if (on) dense_finish8<ACT>(p, m, g, v);
}

// Joins the pieces of the last round's tiles (256 x 256): a thread adds 8 output
// columns of a row (gated: their gate and up columns), piece order; then the epilogue.
// Bound by the pieces' read (192 tiles in 4 pieces, 201 MB: 39 us, 5.8 TB/s with the
// output's write).
template <int ACT>
__global__ void __launch_bounds__(256) dense_tail_join_kernel(DenseArgs p) {
    constexpr int H = kGated<ACT> ? 2 : 1, G = 32 / H;  // groups of 8 outputs in a tile's row
    constexpr int RB = 256 / G;                         // rows a workgroup
    const int rem = p.ntm * p.ntn - p.tail_first;
    const int r = blockIdx.x / (256 / RB);
    const int t = p.tail_first + r;
    const int band = t / (4 * p.ntn), within = t - band * 4 * p.ntn;
    const int bm = min(4, p.ntm - band * 4);
    const int row = blockIdx.x % (256 / RB) * RB + threadIdx.x / G, g = threadIdx.x % G;
    const int c = kGated<ACT> ? (g >> 2) * 64 + (g & 3) * 8 : g * 8;
    const int64_t m = (int64_t)(band * 4 + within % bm) * 256 + row;
    const int n0 = within / bm * 256;
    if (m >= p.M || n0 + c >= p.N) return;
    const float* at = p.part + ((int64_t)r * 256 + row) * 256 + c;
    const int64_t step = (int64_t)rem * 65536;
    float v[2][8] = {};
#pragma unroll 4
    for (int s = 0; s < p.tail_splits; ++s) {
#pragma unroll
        for (int u = 0; u < H; ++u) {
            const float4 a = *(const float4*)(at + s * step + 32 * u), b = *(const float4*)(at + s * step + 32 * u + 4);
            v[u][0] += a.x, v[u][1] += a.y, v[u][2] += a.z, v[u][3] += a.w;
            v[u][4] += b.x, v[u][5] += b.y, v[u][6] += b.z, v[u][7] += b.w;
        }
    }
    dense_finish8<ACT>(p, m, n0 / (8 * H) + g, v);
}

// ------------------------------------------------------------------ small products
// Few output tiles (single tokens, decode batches, small layers): here a product is
// the time to read its operands, W above all, and the latency of its K loop. A
// workgroup owns 64 columns (32 gate and 32 up columns of a gated layer), up to 64
// rows and a range of K; its 4 wavefronts take every fourth 64-deep slab of it, each
// through LDS stages of its own, so the loop has no barrier: a wavefront waits only
// for its own copies, ST - 1 slabs ahead of the one it multiplies. XC copies of 8
// rows (8 XC rows a tile) bring a K-major A, 8 copies an A with K outermost and B.
// The wavefronts' sums meet in LDS. A compute unit copies about 55 B a clock into
// LDS, so tiles this small reach 40% of the matrix rate at most, and larger products
// take the kernel above. [T = 1, K = 8192, N = 4096: 13.3 us, 5.0 TB/s of W; as 128 x
// 128 tiles 14.0 us and a join of 11.5 us over 16 splits.]
template <bool A_KMAJ, bool B_KMAJ, int XC, bool A8>
__global__ void __launch_bounds__(256, 1) dense_small_kernel(DenseArgs p, int act) {
    static_assert(A_KMAJ || XC == 8, "an A with K outermost comes 64 columns at a time");
    constexpr int MT = XC > 4 ? 2 : 1, ROWS = 8 * XC;
    constexpr int ST = XC == 1 ? 4 : XC <= 4 ? 3 : 2;
    constexpr int WB = 64 * 128, STAGE = WB + XC * 1024, CP = 8 + XC;
    __shared__ __attribute__((aligned(1024))) uint8_t s_ab[4 * ST * STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int per = p.ntm * p.ntn;
    const int split = __builtin_amdgcn_readfirstlane(blockIdx.x / per);
    const int t = blockIdx.x - split * per;
    const int m0 = __builtin_amdgcn_readfirstlane(t / p.ntn * ROWS);
    const int n0 = __builtin_amdgcn_readfirstlane(t % p.ntn * 64);
    const int slabs = (p.K + DBK - 1) / DBK;
    const int ks0 = split * p.split_slabs;
    const int nk = min(p.split_slabs, slabs - ks0);
    const int mine = nk > wave ? (nk - wave + 3) / 4 : 0;  // this wavefront's slabs: ks0 + wave + 4 j

    // copy i of a slab: 8 slab rows of 128 bytes, 8 lanes each; row kr + 8 i, chunk c
    const int kr = lane >> 3;
    const int kc = (lane & 7) ^ (((kr >> 1) & 1) << 2);  // K outermost: chunk, the same for every i
    const int a_col = m0 + kc * 8, b_col = n0 + kc * 8;
    const uint8_t* mem = s_ab + wave * ST * STAGE;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS_AS char*)mem;
    const int64_t a_step = A_KMAJ ? DBK * 2 : (int64_t)DBK * p.lda * 2;
    const int64_t b_step = B_KMAJ ? DBK * 2 : (int64_t)DBK * p.ldb * 2;
    const char* a_base = (const char*)(A_KMAJ ? p.A + (int64_t)m0 * p.lda : p.A);
    const char* b_base = (const char*)(B_KMAJ ? p.B + (int64_t)n0 * p.ldb : p.B);
    const int64_t a_bytes = (int64_t)(A_KMAJ ? p.M - m0 : p.K) * p.lda * 2;
    const int64_t b_bytes = (int64_t)(B_KMAJ ? p.N - n0 : p.K) * p.ldb * 2;
    auto issue = [&](int j, int st) {
        const int ks = ks0 + wave + 4 * j;
        const i32x4_t rb = rsrc_from(b_base, b_bytes, ks * b_step);
        const i32x4_t ra = rsrc_from(a_base, a_bytes, ks * a_step);
        const uint32_t l0 = lds0 + st * STAGE;
        const int left = p.K - ks * DBK;
        // K-major: rows past the matrix end read past the resource (zeros), chunks past K are masked
        auto offset = [&](int i, bool kmaj, int64_t ld, int col, int cols) -> uint32_t {
            const int r = kr + 8 * i;
            if (kmaj) {
                const int c = ((lane & 7) ^ kmaj_swz(r)) * 8;
                return c < left ? (uint32_t)((r * ld + c) * 2) : kMasked;
            }
            return col < cols ? (uint32_t)((r * ld + col) * 2) : kMasked;
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) lds_copy16(rb, l0 + i * 1024, offset(i, B_KMAJ, p.ldb, b_col, p.N));
        if constexpr (!A8) {
#pragma unroll
            for (int i = 0; i < XC; ++i) lds_copy16(ra, l0 + WB + i * 1024, offset(i, A_KMAJ, p.lda, a_col, p.M));
        }
    };
    // A from an 8-bit checkpoint: 4 pieces of 16 columns a lane, fetched a slab ahead
    static_assert(!A8 || (!A_KMAJ && ST == 2), "K outermost, one slab ahead");
    Codes16 codes[A8 ? 4 : 1];
    auto fetch_a8 = [&](int j) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            codes[A8 ? i : 0] = codes16_load(p, (int64_t)(ks0 + wave + 4 * j) * DBK + 16 * i + (lane >> 2), m0 + (lane & 3) * 16);
    };
    auto put_a8 = [&](int st) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 16 * i + (lane >> 2), c = (lane & 3) * 2, x = ((r >> 1) & 1) << 2;
            uint8_t* row = s_ab + (wave * ST + st) * STAGE + WB + r * 128;
            codes16_store(codes[A8 ? i : 0], row + ((c ^ x) << 4), row + (((c + 1) ^ x) << 4));
        }
    };
    // MFMA operand: index base + (lane & 31), k = 16 ks + 8 (lane >> 5) + [0, 8)
    auto frag = [&](const uint8_t* s, auto KM, int rows, int base, int ks) -> bf16x8_t {
        if constexpr (decltype(KM)::value) {
            // rows past the copied ones repeat them: their products are never stored
            const int r = (base + (lane & 31)) & (rows - 1);
            return __builtin_bit_cast(bf16x8_t, *(const uint4*)(s + kmaj_byte(r, 2 * ks + (lane >> 5))));
        } else {
            const int lg = lane & 15;
            const int c = base + 16 * ((lane >> 4) & 1) + 4 * (lg & 3);
            const int k0 = 16 * ks + 8 * (lane >> 5) + (lg >> 2), k1 = k0 + 4;
            const int o0 = k0 * 128 + (((c >> 3) ^ (((k0 >> 1) & 1) << 2)) << 4) + (c & 7) * 2;
            const int o1 = k1 * 128 + (((c >> 3) ^ (((k1 >> 1) & 1) << 2)) << 4) + (c & 7) * 2;
            const bf16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LDS_AS bf16x4_t*)(s + o0));
            const bf16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((LDS_AS bf16x4_t*)(s + o1));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };
    f32x16_t acc[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = (f32x16_t){};
    for (int j = 0; j < ST - 1 && j < mine; ++j) issue(j, j);
    if constexpr (A8) {
        if (mine > 0) {
            fetch_a8(0);
            put_a8(0);
        }
    }
    int st = 0;
    for (int j = 0; j < mine; ++j) {
        // slab j has landed; the reads of slab j - 1, whose stage is filled next, are done
        if (mine - 1 - j >= ST - 2)
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"((ST - 2) * CP) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : : : "memory");
        if (j + ST - 1 < mine) {
            if constexpr (A8) fetch_a8(j + 1);
            issue(j + ST - 1, (st + ST - 1) % ST);
        }
        const uint8_t* s = mem + st * STAGE;
        static_for<4>([&](auto KS) {
            constexpr int ks = KS;
            bf16x8_t fx[MT], fw[2];
#pragma unroll
            for (int i = 0; i < MT; ++i) fx[i] = frag(s + WB, std::bool_constant<A_KMAJ>{}, ROWS, 32 * i, ks);
#pragma unroll
            for (int u = 0; u < 2; ++u) fw[u] = frag(s, std::bool_constant<B_KMAJ>{}, 64, 32 * u, ks);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    acc[i][u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fw[u], fx[i], acc[i][u], 0, 0, 0);
        });
        if constexpr (A8) {
            if (j + 1 < mine) put_a8(st ^ 1);
        }
        st = st + 1 == ST ? 0 : st + 1;
    }
    // join of the 4 wavefronts: 32 rows at a time, wavefront w's 8 KiB at 8192 w, the
    // 16-byte chunks of a 256-byte row XOR-swizzled by the row
    const int h = lane >> 5, r = lane & 31;
    static_for<MT>([&](auto I) {
        __syncthreads();
        static_for<2>([&](auto J) {
            static_for<4>([&](auto Q) {
                const int ch = 8 * J + 2 * Q + h;
                *(float4*)(s_ab + wave * 8192 + r * 256 + ((ch ^ (r & 15)) << 4)) = make_float4(
                    acc[I][J][4 * Q], acc[I][J][4 * Q + 1], acc[I][J][4 * Q + 2], acc[I][J][4 * Q + 3]);
            });
        });
        __syncthreads();
        auto sum8 = [&](int row, int c8, float* v) {  // columns [8 c8, 8 c8 + 8) of the tile's row
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint8_t* at = s_ab + row * 256 + (((2 * c8 + q) ^ (row & 15)) << 4);
                const float4 a = *(const float4*)at, b = *(const float4*)(at + 8192);
                const float4 c = *(const float4*)(at + 16384), d = *(const float4*)(at + 24576);
                v[4 * q] = (a.x + b.x) + (c.x + d.x);
                v[4 * q + 1] = (a.y + b.y) + (c.y + d.y);
                v[4 * q + 2] = (a.z + b.z) + (c.z + d.z);
                v[4 * q + 3] = (a.w + b.w) + (c.w + d.w);
            }
        };
        float v[2][8];
        if (act > 1 || p.part) {
            const int row = tid >> 3, c8 = tid & 7, col = n0 + 8 * c8;
            const int64_t m = m0 + 32 * I + row;
            sum8(row, c8, v[0]);
            if (m < p.M && col < p.N) {
                if (p.part) {
                    float4* o = (float4*)(p.part + ((int64_t)split * p.M + m) * p.N + col);
                    o[0] = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
                    o[1] = make_float4(v[0][4], v[0][5], v[0][6], v[0][7]);
                } else if (act == 2) dense_finish8<2>(p, m, col / 8, v);
                else if (act == 3) dense_finish8<3>(p, m, col / 8, v);
                else if (act == 4) dense_finish8<4>(p, m, col / 8, v);
                else dense_finish8<5>(p, m, col / 8, v);
            }
        } else if (tid < 128) {
            const int row = tid >> 2, c8 = tid & 3;
            const int64_t m = m0 + 32 * I + row;
            sum8(row, c8, v[0]);
            sum8(row, c8 + 4, v[1]);
            if (m < p.M) {
                if (act == 0) dense_finish8<0>(p, m, n0 / 16 + c8, v);
                else dense_finish8<1>(p, m, n0 / 16 + c8, v);
            }
        }
    });
}

// ------------------------------------------------------------------ host side
static int tiles_left(const DensePlan& d) { return d.ntm * d.ntn - d.tail_first; }

size_t dense_part_bytes(int64_t M, int64_t N, int64_t K, DensePass pass) {
    const DensePlan d = dense_plan(M, N, K, pass);
    if (d.tail_splits > 1)
        return (size_t)tiles_left(d) * d.tail_splits * 65536 * sizeof(float);
    return d.splits > 1 ? (size_t)d.splits * M * N * sizeof(float) : 0;
}

template <bool A_KMAJ, bool B_KMAJ, int ACT>
static void dense_launch(const DensePlan& d, const DenseArgs& a, hipStream_t s) {
    const int tiles = d.ntm * d.ntn;
    const int total = d.tail_splits > 1 ? d.tail_first + (tiles - d.tail_first) * d.tail_splits : tiles * d.splits;
    if (d.kind == 's') {
        const unsigned grid = (unsigned)total;
        if constexpr (A_KMAJ) {
            if (a.M <= 8) return dense_small_kernel<true, B_KMAJ, 1, false><<<grid, 256, 0, s>>>(a, ACT);
            if (a.M <= 16) return dense_small_kernel<true, B_KMAJ, 2, false><<<grid, 256, 0, s>>>(a, ACT);
            if (a.M <= 32) return dense_small_kernel<true, B_KMAJ, 4, false><<<grid, 256, 0, s>>>(a, ACT);
        }
        if constexpr (!A_KMAJ) {
            if (a.a_q) return dense_small_kernel<false, B_KMAJ, 8, true><<<grid, 256, 0, s>>>(a, ACT);
        }
        return dense_small_kernel<A_KMAJ, B_KMAJ, 8, false><<<grid, 256, 0, s>>>(a, ACT);
    }
    // persistent: as many workgroups as the compute units hold, a multiple of 8; the
    // deep form runs one tile per workgroup
    const int most = d.kind == 'M' ? 2 * device_cus() : d.kind == 'L' ? device_cus() : total;
    const unsigned grid = (unsigned)((std::min(total, most) + 7) / 8 * 8);
    if (d.tail_splits > 1) dense_gemm_kernel<256, 256, 2, 4, 2, A_KMAJ, B_KMAJ, ACT, true><<<grid, 512, 0, s>>>(a);
    else if (d.kind == 'L') dense_gemm_kernel<256, 256, 2, 4, 2, A_KMAJ, B_KMAJ, ACT><<<grid, 512, 0, s>>>(a);
    else if (d.kind == 'D') dense_gemm_kernel<128, 128, 2, 2, 4, A_KMAJ, B_KMAJ, ACT><<<grid, 256, 0, s>>>(a);
    else if (d.kind == 'H') dense_gemm_kernel<256, 128, 4, 2, 3, A_KMAJ, B_KMAJ, ACT><<<grid, 512, 0, s>>>(a);
    else dense_gemm_kernel<128, 128, 2, 2, 2, A_KMAJ, B_KMAJ, ACT><<<grid, 256, 0, s>>>(a);
}

template <bool A_KMAJ, bool B_KMAJ, int ACT>
static int dense_run(DenseArgs a, void* ws, hipStream_t s) {
    const DensePlan d = dense_plan(a.M, a.N, a.K, !A_KMAJ ? kWgrad : B_KMAJ ? kDgrad : kForward);
    a.ntm = d.ntm;
    a.ntn = d.ntn;
    a.splits = d.splits;
    a.split_slabs = d.split_slabs;
    a.stream = (int64_t)a.M * a.N * (a.out_f32 ? 4 : 2) >= kDenseStreamBytes;
    a.tail_first = d.tail_first, a.tail_splits = d.tail_splits, a.tail_slabs = d.tail_slabs;
    if (d.splits == 1) {
        a.part = d.tail_splits > 1 ? (float*)ws : nullptr;
        dense_launch<A_KMAJ, B_KMAJ, ACT>(d, a, s);
        if (d.tail_splits > 1)
            dense_tail_join_kernel<ACT><<<(unsigned)(tiles_left(d) * (kGated<ACT> ? 16 : 32)), 256, 0, s>>>(a);
    } else {
        a.part = (float*)ws;
        dense_launch<A_KMAJ, B_KMAJ, 3>(d, a, s);
        const int64_t items = (int64_t)a.M * ((kGated<ACT> ? a.N / 2 : a.N) / 8);
        if (dense_join_wide(items, d.splits))
            dense_join_kernel<ACT, 8><<<(unsigned)((items + 31) / 32), 256, 0, s>>>(a);
        else
            dense_join_kernel<ACT, 1><<<(unsigned)((items + 255) / 256), 256, 0, s>>>(a);
    }
    return hipGetLastError() == hipSuccess ? 0 : -4;
}

int launch_linear_fwd(const uint16_t* x, const uint16_t* w, const uint16_t* bias, const uint16_t* res, int T,
                      int K, int N, int act, int y_f32, void* y, uint16_t* z, uint8_t* z_q, uint8_t* z_s,
                      void* ws, hipStream_t s) {
    DenseArgs a{};
    a.A = x, a.lda = K, a.B = w, a.ldb = N, a.M = T, a.N = N, a.K = K;
    a.bias = bias, a.res = res, a.out = y, a.out_f32 = y_f32, a.z = z, a.z_q = z_q, a.z_s = z_s;
    switch (act) {
        case 0: return dense_run<true, false, 0>(a, ws, s);
        case 1: return dense_run<true, false, 1>(a, ws, s);
        case 2: return dense_run<true, false, 2>(a, ws, s);
        case 3: return dense_run<true, false, 3>(a, ws, s);
        case 4: return dense_run<true, false, 4>(a, ws, s);
        default: return dense_run<true, false, 5>(a, ws, s);
    }
}

int launch_linear_dgrad(const uint16_t* dz, const uint16_t* w, const uint16_t* res, int T, int K, int N,
                        uint16_t* dx, void* ws, hipStream_t s) {
    DenseArgs a{};
    a.A = dz, a.lda = N, a.B = w, a.ldb = N, a.M = T, a.N = K, a.K = N;
    a.res = res, a.out = dx;
    return dense_run<true, true, 3>(a, ws, s);
}

// An 8-bit x is read as it is by the small kernel; larger products take a bf16 copy
// restored into the workspace first, because converting inside the tile loop costs
// more than the copy (16384 x 7168 x 4096: 892 us with the copy, 1260 converted in the
// loop, 876 from bf16; 200 x 1024 x 1024: 13.1, 9.9, 10.2).
static size_t dense_copy_bytes(int64_t T, int64_t K, int64_t N) {
    return K % 32 || dense_plan(K, N, T, kWgrad).kind == 's' ? 0 : (size_t)((T * K * 2 + 255) / 256 * 256);
}

size_t linear_wgrad_bytes(int T, int K, int N, bool x8) {
    return (x8 ? dense_copy_bytes(T, K, N) : 0) + dense_part_bytes(K, N, T, kWgrad);
}

int launch_linear_wgrad(const uint16_t* x, const uint8_t* x_q, const uint8_t* x_s, const uint16_t* dz, int T,
                        int K, int N, int dw_f32, int accumulate, void* dw, void* ws, hipStream_t s) {
    if (const size_t copy = x_q ? dense_copy_bytes(T, K, N) : 0) {
        if (launch_dequant_mxfp8(x_q, x_s, T, K, (uint16_t*)ws, s)) return -4;
        x = (const uint16_t*)ws;
        x_q = nullptr;
        ws = (char*)ws + copy;
    }
    DenseArgs a{};
    a.A = x, a.lda = K, a.a_q = x_q, a.a_s = x_s, a.B = dz, a.ldb = N, a.M = K, a.N = N, a.K = T;
    a.out = dw, a.out_f32 = dw_f32, a.accumulate = accumulate;
    return dense_run<false, false, 3>(a, ws, s);
}

}  // namespace moe
