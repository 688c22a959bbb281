/*
 * moe.h -- C ABI of libmoe.so: the dropless MoE expert MLP on one MI355X
 * (gfx950), run as a sync-free ragged grouped GEMM with a fused GLU epilogue.
 *
 * Sources (web pages, cited by title and section):
 *   [P1] "NVIDIA CuTe DSL 융합 커널은 MoE 학습의 CPU·메모리 병목을 지운다"
 *   [P2] "SonicMoE로 보는 GPU 커널 최적화"
 *   [P3] "Dropless MoE 학습과 NVIDIA Transformer Engine 소개"
 *
 * Conventions shared by every entry point
 *   - bf16 tensors are passed as uint16_t* raw bit patterns; all sizes are
 *     element counts; every matrix is row-major and densely packed.
 *   - Every pointer argument is a DEVICE pointer unless stated otherwise.
 *     The caller owns every buffer and keeps it alive until the stream work
 *     that uses it has completed. The library allocates nothing and keeps no
 *     pointer after a call returns. Its only mutable global state is two
 *     per-device caches filled on first use (the compute-unit count, and the
 *     device address of the static scratch of moe_route_counts_noalloc), so
 *     calls are reentrant and thread-safe, except that moe_route_counts_noalloc
 *     calls overlapping on one GPU share that scratch.
 *   - Every call only enqueues work on `stream` (a hipStream_t; NULL = the
 *     legacy default stream). No call synchronises, allocates or copies
 *     device-to-host, so every call may be recorded into a hipGraph. Shapes
 *     that depend on the routing (per-expert counts and offsets) are read by
 *     the kernels from device memory only [P1, core-idea section: per-expert
 *     counts tracked on the GPU so no host shape query is needed].
 *   - Host-checkable errors (NULL pointers, bad sizes, misaligned pointers,
 *     a too-small workspace or capacity) return a negative status before any
 *     launch. A launch failure returns MOE_ERR_LAUNCH. Data-dependent
 *     problems never trap: they set bits in a caller-owned device error word.
 *
 * Layout of the expert-major ragged buffer [P3, sections on ragged tensors,
 * dropless MoE, grouped GEMM (128-token alignment) and the dropless
 * boundary (one slot per (token, expert) pair, expert regions padded)]:
 *   pair p = t*k + j (token t, slot j) goes to expert e = topk_idx[t, j];
 *   expert e owns rows [offsets[e], offsets[e+1]), offsets[0] = 0,
 *   offsets[e+1] - offsets[e] = 128 * ceil(counts[e] / 128) (0 if empty);
 *   its pairs sit in rows offsets[e] + rank in ascending p, the remaining
 *   rows of its region are padding and every permuted tensor the library
 *   writes holds zeros there; rows >= offsets[E] are never read or written.
 *   M_cap = moe_capacity_rows(T, k, E) rows always suffice, so nothing is
 *   ever dropped [P3, dropless-boundary section: a worst-case buffer never
 *   drops].
 *
 * FC1 weight layout [P3, grouped-GEMM section: prefused FC1 weight of shape
 * (experts, embed_dim, 2*mlp_dim); P1, core-idea section: gate and input
 * columns interleaved so one tile holds both halves]: w1 is [E, d, 2n];
 * column block b (32 wide) of each row holds gate columns [2*32b, 2*32b+32)
 * = gate[32b, 32b+32) followed by up columns = up[32b, 32b+32).
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ALIGN 128          /* rows per expert-region alignment unit    */
#define MOE_MX_BLOCK 32        /* elements per MXFP8 scale block           */
#define MOE_GLU_INTERLEAVE 32  /* gate/up interleave granularity (columns) */
#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_WIDTH (1 << 20) /* largest d and FC1 width (2n, or n for sReLU) */

#define MOE_MAX_ROWS (1 << 30)  /* largest T of the dense entry points */

/* status codes */
#define MOE_OK 0
#define MOE_ERR_INVALID_ARG (-1)  /* NULL/negative/misaligned argument      */
#define MOE_ERR_UNSUPPORTED (-2)  /* valid but unsupported shape or option  */
#define MOE_ERR_WORKSPACE (-3)    /* workspace or M_cap too small           */
#define MOE_ERR_LAUNCH (-4)       /* a kernel launch reported an error      */

/* activation of the expert MLP */
#define MOE_ACT_SWIGLU 0       /* silu(gate) * up, silu(x) = x / (1 + e^-x) */
#define MOE_ACT_GEGLU 1        /* gelu(gate) * up, gelu(x) = x * Phi(x) (exact, erf form) */
#define MOE_ACT_SRELU 2        /* relu(h)^2, non-gated: FC1 has n columns, w1 [E, d, n],
                                  h and dh [M_cap, n], dw1 [E, d, n] [P1, problem and
                                  published-evidence sections: the sReLU family] */
/* further activations of the dense linear layer (non-gated) */
#define MOE_ACT_NONE 3         /* identity */
#define MOE_ACT_SILU 4         /* silu(z) */
#define MOE_ACT_GELU 5         /* gelu(z), exact */

/* passes of moe_linear_workspace_bytes (bits) */
#define MOE_LINEAR_FWD 0x1
#define MOE_LINEAR_BWD 0x2

/* stage bits of moe_grouped_mlp_fwd / moe_grouped_mlp_bwd */
#define MOE_STAGE_FC1 0x01     /* H = X_perm W1_e, A = GLU(H)               */
#define MOE_STAGE_FC2 0x02     /* Y = A W2_e                                */
#define MOE_STAGE_DGRAD2 0x04  /* dA' = dY_u W2_e^T + dGLU epilogue, dS     */
#define MOE_STAGE_WGRAD2 0x08  /* dW2_e = A'^T dY_u                          */
#define MOE_STAGE_DGRAD1 0x10  /* dX_perm = dH W1_e^T                        */
#define MOE_STAGE_WGRAD1 0x20  /* dW1_e = X_perm^T dH                        */
#define MOE_STAGES_FWD (MOE_STAGE_FC1 | MOE_STAGE_FC2)
#define MOE_STAGES_BWD (MOE_STAGE_DGRAD2 | MOE_STAGE_WGRAD2 | MOE_STAGE_DGRAD1 | MOE_STAGE_WGRAD1)
/* mode bit for moe_grouped_mlp_fwd / _bwd: the x_perm argument (and dy_u in
 * the backward) is the un-permuted [T, d] tensor, and the GEMMs read its rows
 * through src_of (row r = token src_of[r] / k; padding rows read zeros), so
 * no expert-major copy is written or read [P2, IO-hiding section: gather
 * fused into the GEMM's loads] */
#define MOE_GATHER_ROWS 0x100

/* bits of the device error word */
#define MOE_ERRBIT_NONFINITE_LOGIT 0x1

/* moe_quant_mxfp8 mode bits */
#define MOE_QUANT_ROWWISE 0x1
#define MOE_QUANT_COLWISE 0x2

typedef void* moe_stream_t; /* hipStream_t */

/* Human-readable name of a status code (static string, never NULL). */
const char* moe_status_str(int status);

/* Worst-case row count of the expert-major buffer for T tokens, top-k over E
 * experts: 128*ceil(T*k/128) + 128*E. Returns -1 for invalid arguments.
 * Host-only; touches no device. */
int64_t moe_capacity_rows(int T, int k, int E);

/* Device workspace (bytes) that moe_route_counts needs. Host-only. */
size_t moe_route_workspace_bytes(int T, int k, int E);

/* Device workspace (bytes) that moe_grouped_mlp_bwd needs (per-row router
 * gradient partials). Host-only. */
size_t moe_mlp_bwd_workspace_bytes(int n, int64_t M_cap);

/*
 * moe_route_counts -- softmax top-k routing plus the device-resident ragged
 * layout: per-expert counts, 128-aligned prefix offsets and both row maps.
 *   [P3, ragged-tensor section: a learned router sends each token to its
 *   top-K experts and the per-expert counts vary per batch; P1, core-idea
 *   section: counts stay in GPU memory; P3, grouped-GEMM section: 128-token
 *   alignment of expert regions.]
 * Routing: p = softmax over all E logits of a token (fp32); experts ranked by
 * raw logit, descending, ties to the lower expert index; slot j holds the
 * j-th best; topk_w[t, j] = p of that expert, renormalised over the k chosen
 * ones when renorm != 0.
 *   logits   [T, E] fp32 (in)
 *   topk_idx [T, k] int32 (out)    topk_w [T, k] fp32 (out)
 *   counts   [E] int32 (out)       offsets [E+1] int32 (out)
 *   row_of   [T*k] int32 (out): row of pair p in the expert-major buffer
 *   src_of   [M_cap] int32 (out): pair held by each row, -1 for padding and
 *            for rows >= offsets[E]
 *   err_word [1] int32 (in/out, device): MOE_ERRBIT_NONFINITE_LOGIT is OR-ed
 *            in when a logit is NaN or infinite (the routing of such a token
 *            is then unspecified but every output stays in range)
 *   workspace: >= moe_route_workspace_bytes(T, k, E) bytes, 16-byte aligned
 * Requires 1 <= k <= E <= MOE_MAX_EXPERTS, T >= 1, M_cap >= capacity rows.
 */
int moe_route_counts(const float* logits, int T, int E, int k, int renorm,
                     int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* offsets,
                     int32_t* row_of, int32_t* src_of, int64_t M_cap, int32_t* err_word,
                     void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* Bytes of the static device scratch behind moe_route_counts_noalloc (per GPU). */
#define MOE_ROUTE_STATIC_SCRATCH_BYTES (8u << 20)

/*
 * moe_route_counts_noalloc -- moe_route_counts with no workspace argument, for
 *   callers that cannot allocate device memory: code under hipGraph capture
 *   that may not call hipMalloc, tight serving loops, harnesses that forbid
 *   allocation. Same arguments (minus the workspace), the same kernels and
 *   bit-identical outputs. The layout scratch is a device array of
 *   MOE_ROUTE_STATIC_SCRATCH_BYTES that the library reserves statically; each
 *   GPU holds its own copy until the process ends, and its address is looked
 *   up once per device on the first call with that device current. The call
 *   allocates nothing (no hipMalloc/hipFree, no allocating library routine).
 *   Returns MOE_ERR_WORKSPACE, before launching anything, when
 *   moe_route_workspace_bytes(T, k, E) exceeds that size (at most 8 bytes per
 *   expert per 1024 routed pairs: e.g. T*k = 2^20 pairs with E = 1024 experts fit).
 *   Every call on one GPU shares the array and leaves its contents behind
 *   (nothing in it needs clearing between calls), so calls that overlap on a
 *   GPU (concurrent streams or host threads) race: the caller serialises them.
 */
int moe_route_counts_noalloc(const float* logits, int T, int E, int k, int renorm,
                             int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* offsets,
                             int32_t* row_of, int32_t* src_of, int64_t M_cap, int32_t* err_word,
                             moe_stream_t stream);

/*
 * moe_route_bwd -- router backward: gradient of the loss w.r.t. the router
 *   logits, given ds = dL/dtopk_w from moe_grouped_mlp_bwd, for the experts
 *   the forward chose (topk_idx). Without renormalisation
 *     dlogits[t, e] = p_e (g_e - sum_j p_{e_j} ds[t, j]),
 *   p = softmax(logits[t]) over all E, g_e = ds[t, j] if e = e_j else 0;
 *   with renorm != 0 (weights renormalised over the chosen k)
 *     dlogits[t, e_j] = w_j (ds[t, j] - sum_i w_i ds[t, i]), 0 elsewhere.
 *   Non-finite logits have probability 0 and gradient 0.
 *   [P2, backward-rewrite section: dS is the router-score gradient and flows
 *   on through the router.]
 *   logits [T, E] fp32, topk_idx [T, k] int32 (as written by
 *   moe_route_counts), ds [T, k] fp32 (in); dlogits [T, E] fp32 (out).
 * Requires 0 < k <= E <= MOE_MAX_EXPERTS, T > 0; else MOE_ERR_INVALID_ARG.
 */
int moe_route_bwd(const float* logits, const int32_t* topk_idx, const float* ds, int T, int E,
                  int k, int renorm, float* dlogits, moe_stream_t stream);

/*
 * moe_permute -- gather token rows into the expert-major buffer
 *   x_perm[row_of[t*k + j]] = x[t] for every token t and slot j, and
 *   x_perm[r] = 0 for the padding rows of every expert region (the rows
 *   r < offsets[E] with src_of[r] < 0). Each token row is read once and
 *   written to its k rows.
 *   [P2, SonicMoE section: the gather sub-kernel; P3, EP section: dispatch
 *   permutes tokens expert-major.] Used for activations (forward) and for the
 *   upstream gradient dO (backward; no weighting).
 *   x [T, d] bf16 (in); row_of [T*k], src_of [M_cap], offsets [E+1] (in, as
 *   written by moe_route_counts: row_of and src_of are inverse maps);
 *   x_perm [M_cap, d] bf16 (out; rows >= offsets[E] untouched).
 * Requires d % 8 == 0; x and x_perm 16-byte aligned.
 */
int moe_permute(const uint16_t* x, const int32_t* row_of, const int32_t* src_of,
                const int32_t* offsets, int T, int k, int E, int d, int64_t M_cap,
                uint16_t* x_perm, moe_stream_t stream);

/*
 * moe_combine -- weighted un-permute: out[t] = sum over j ascending of
 *   w[t, j] * y[row_of[t*k + j]], accumulated in fp32, rounded once to bf16.
 *   w == NULL means unit weights (the backward's dX = sum_j dX_perm rows).
 *   [P2, SonicMoE section: scatter + expert aggregation sub-kernels; P3, EP
 *   section: combine restores token order and accumulates per token.]
 *   y [M_cap, d] bf16, row_of [T*k], w [T, k] fp32 or NULL (in),
 *   out [T, d] bf16 (out). Requires d % 8 == 0, 16-byte aligned y and out.
 */
int moe_combine(const uint16_t* y, const int32_t* row_of, const float* w,
                int T, int k, int d, uint16_t* out, moe_stream_t stream);

/* MXFP8 side of the forward (all device pointers). E4M3 codes (OCP, bias 7,
 * round to nearest-even), E8M0 block scales (code = exponent + 127) over 32
 * elements: the shared exponent is the smallest e with amax <= 448 * 2^e, so
 * no element saturates; a zero block takes code 0. */
typedef struct moe_mx_fwd {
    uint8_t* a_q;          /* [M_cap, n]    row-wise codes of A (out)            */
    uint8_t* a_s;          /* [M_cap, n/32] row-wise scales of A (out)           */
    uint8_t* at_q;         /* [n, M_cap]    transposed (column-wise) codes, or NULL */
    uint8_t* at_s;         /* [n, M_cap/32] transposed scales, or NULL           */
    const uint8_t* w2t_q;  /* [E, d, n]     W2_e quantized along n, transposed (in) */
    const uint8_t* w2t_s;  /* [E, d, n/32]  its scales (in)                      */
    const uint8_t* x_q;    /* [M_cap, d]    X_perm row-wise codes (in), or NULL: FC1 in bf16 */
    const uint8_t* x_s;    /* [M_cap, d/32] its scales (in)                      */
    const uint8_t* w1t_q;  /* [E, 2n, d]    W1_e quantized along d, transposed (in) */
    const uint8_t* w1t_s;  /* [E, 2n, d/32] its scales (in)                      */
    uint8_t* y_q;          /* [M_cap, d]    row-wise codes of Y (out), or NULL    */
    uint8_t* y_s;          /* [M_cap, d/32] its scales (out)                     */
    uint8_t* yt_q;         /* [d, M_cap]    transposed (column-wise) codes of Y (out), or NULL */
    uint8_t* yt_s;         /* [d, M_cap/32] its scales (out)                     */
} moe_mx_fwd;

/*
 * moe_grouped_mlp_fwd -- grouped FC1 + GLU epilogue, then grouped FC2,
 * one launch each over all experts, tiles scheduled from device offsets;
 * empty experts take no tiles.
 *   [P1, problem and core-idea sections: the GLU activation fused into the
 *   FC1 GEMM epilogue over interleaved weights; P3, grouped-GEMM section: one
 *   call for all experts computing only the real rows.]
 *   FC1: H = X_perm[R_e] W1_e (fp32 accumulate); A = bf16(f(g) * u) from
 *        the fp32 accumulators, f = silu (act = MOE_ACT_SWIGLU) or exact
 *        gelu (act = MOE_ACT_GEGLU) [P1, problem section: SwiGLU and GeGLU
 *        epilogues]; H is stored (bf16) when h != NULL.
 *   FC2: Y = bf16(A[R_e] W2_e). With mx != NULL:
 *        - a_q != NULL: the FC1 epilogue also writes the MXFP8 row-wise (and,
 *          if at_q != NULL, transposed) copy of the bf16 A [P1, core-idea
 *          section: MXFP8 and transposed output fused in the GEMM];
 *        - w2t_q != NULL: FC2 runs on MX-scaled MFMA from a_q/a_s and
 *          w2t_q/w2t_s instead of a and w2 [P3, three-components section:
 *          MXFP8 grouped GEMM]; otherwise FC2 stays bf16 from a and w2;
 *        - y_q != NULL: the FC2 epilogue also writes the row-wise MXFP8 copy
 *          of the bf16 Y (blocks of 32 along d; the "GroupGemm + Quantize"
 *          fused kernel [P3, next-steps section], for an FP8 combine or
 *          all-to-all), and, if yt_q != NULL, its column-wise copy stored
 *          transposed (blocks of 32 rows of an expert region, as at_q); y may
 *          then be NULL;
 *        - x_q != NULL: FC1 also runs on MX-scaled MFMA, from x_q/x_s and
 *          w1t_q/w1t_s instead of x_perm and w1 (then a_q is required,
 *          d % 128 == 0 and no MOE_GATHER_ROWS).
 *   x_perm [M_cap, d], w1 [E, d, 2n], w2 [E, n, d] (bf16, in);
 *   offsets [E+1] (in); h [M_cap, 2n] (out, nullable), a [M_cap, n] (out;
 *   nullable when A's MXFP8 copy is written and FC2 reads only that copy),
 *   y [M_cap, d] (out; needed with MOE_STAGE_FC2 unless y_q is given).
 *   stages: MOE_STAGE_FC1 and/or MOE_STAGE_FC2 (FC2 alone reads a), plus
 *   optionally MOE_GATHER_ROWS: x_perm is then x [T, d] and FC1 reads its
 *   rows through src_of [M_cap] (T, k: the routing shape; both are ignored
 *   without the bit; T * d * 2 < 2^31).
 * With act = MOE_ACT_SRELU the MLP is non-gated: FC1 = X_perm[R_e] W1_e with
 * w1 [E, d, n], A = bf16(relu(H)^2), h [M_cap, n]; no MXFP8 form (mx must be
 * NULL).
 * Requires d % 64 == 0, n % 64 == 0, act MOE_ACT_SWIGLU, MOE_ACT_GEGLU or MOE_ACT_SRELU,
 * M_cap % 128 == 0, M_cap < 2^31, d and the FC1 width (2n; n for sReLU) at
 * most MOE_MAX_WIDTH; no limit on the size of any tensor (every GEMM tile
 * and K slab is addressed from its own 64-bit base). With MOE_GATHER_ROWS
 * the un-permuted x is addressed as a whole with 32-bit byte offsets:
 * T * d * 2 < 2^31. With mx != NULL: n % 128 == 0 (the MX FC2 reads whole
 * 128-byte K slabs of A's codes), and with mx->x_q also d % 128 == 0, so the
 * MXFP8 form needs d, n multiples of 128 (a 2880-wide model is refused).
 * 16-byte aligned pointers. Otherwise MOE_ERR_UNSUPPORTED.
 */
int moe_grouped_mlp_fwd(const uint16_t* x_perm, const uint16_t* w1, const uint16_t* w2,
                        const int32_t* offsets, const int32_t* src_of, int T, int k, int E, int d,
                        int n, int64_t M_cap, int act, unsigned stages, uint16_t* h, uint16_t* a,
                        uint16_t* y, const moe_mx_fwd* mx, moe_stream_t stream);

/* MXFP8 side of the backward (all device pointers; codes and scales as in
 * moe_mx_fwd). DGRAD2 writes the first six, the others are inputs the caller
 * quantizes with moe_quant_mxfp8 (column-wise dY_u and X_perm, row-wise W1). */
typedef struct moe_mx_bwd {
    uint8_t* dh_q;         /* [M_cap, 2n]     row-wise codes of dH (DGRAD2 out, DGRAD1 in) */
    uint8_t* dh_s;         /* [M_cap, 2n/32]  its scales                        */
    uint8_t* dht_q;        /* [2n, M_cap]     column-wise codes of dH, transposed (DGRAD2 out, WGRAD1 in) */
    uint8_t* dht_s;        /* [2n, M_cap/32]  its scales                        */
    uint8_t* awt_q;        /* [n, M_cap]      column-wise codes of A', transposed (DGRAD2 out, WGRAD2 in) */
    uint8_t* awt_s;        /* [n, M_cap/32]   its scales                        */
    const uint8_t* dyt_q;  /* [d, M_cap]      column-wise codes of dY_u, transposed (WGRAD2 in) */
    const uint8_t* dyt_s;  /* [d, M_cap/32]                                     */
    const uint8_t* xt_q;   /* [d, M_cap]      column-wise codes of X_perm, transposed (WGRAD1 in) */
    const uint8_t* xt_s;   /* [d, M_cap/32]                                     */
    const uint8_t* w1_q;   /* [E, d, 2n]      W1_e row-wise along 2n (DGRAD1 in) */
    const uint8_t* w1_s;   /* [E, d, 2n/32]                                     */
    const uint8_t* dy_q;   /* [M_cap, d]      dY_u row-wise codes (DGRAD2 in), or NULL: DGRAD2 in bf16 */
    const uint8_t* dy_s;   /* [M_cap, d/32]                                     */
    const uint8_t* w2_q;   /* [E, n, d]       W2_e row-wise along d (DGRAD2 in) */
    const uint8_t* w2_s;   /* [E, n, d/32]                                      */
    uint8_t* dx_q;         /* [M_cap, d]      row-wise codes of dX_perm (DGRAD1 out), or NULL */
    uint8_t* dx_s;         /* [M_cap, d/32]                                     */
    uint8_t* dxt_q;        /* [d, M_cap]      column-wise codes of dX_perm, transposed (DGRAD1 out), or NULL */
    uint8_t* dxt_s;        /* [d, M_cap/32]                                     */
} moe_mx_bwd;

/*
 * moe_grouped_mlp_bwd -- backward of the expert MLP for fixed routing.
 *   [P2, backward-rewrite section: dS_{t,e} = <dO_t, Y> = <dO_t W2^T, A>;
 *   GEMM-overlapping section: the dH kernel reloads H in its epilogue and
 *   stores dH, dS and A'; P1, published-evidence section: dSwiGLU and dGeGLU
 *   fused into the dgrad GEMM.]
 *   DGRAD2: dA' = dY_u[R_e] W2_e^T (fp32); epilogue with a = f(g) u from
 *           the stored H (f the gate activation selected by act) and
 *           w = topk_w of the row's pair (0 for padding):
 *           dS partials += dA' . a per row; dA = w dA';
 *           dg = dA u f'(g) (silu' = s (1 + g (1 - s)), s = sigmoid(g);
 *           gelu' = Phi(g) + g phi(g)); du = dA f(g);
 *           dH = bf16 interleaved (dg, du); A' = bf16(w a);
 *           then ds[t, j] = sum of the row's partials in a fixed order.
 *   WGRAD2: dW2_e = A'[R_e]^T dY_u[R_e] (fp32; exactly 0 for empty experts).
 *   DGRAD1: dX_perm[R_e] = bf16(dH[R_e] W1_e^T).
 *   WGRAD1: dW1_e = X_perm[R_e]^T dH[R_e] (fp32, interleaved like w1).
 *   Non-gated act = MOE_ACT_SRELU: dH = bf16(w dA' * 2 relu(h)), A' = w relu(h)^2,
 *   dS partials += dA' . relu(h)^2; h, dh [M_cap, n], w1 and dw1 [E, d, n].
 *   dy_u = moe_permute of dO (unweighted). Stages run in the order above.
 *   With MOE_GATHER_ROWS in stages, x_perm is x [T, d] and dy_u is dO [T, d]
 *   (un-permuted) and every GEMM reads their rows through src_of.
 *   x_perm, dy_u [M_cap, d]; w1 [E, d, 2n]; w2 [E, n, d]; h [M_cap, 2n]
 *   (bf16, in); topk_w [T, k] fp32, src_of [M_cap], row_of [T*k],
 *   offsets [E+1] (in); dh [M_cap, 2n], a_w [M_cap, n], dx_perm [M_cap, d]
 *   (bf16, out); ds [T, k] fp32 (out); dw1 [E, d, 2n], dw2 [E, n, d]
 *   (fp32, out). Outputs of stages not requested may be NULL.
 *   workspace: >= moe_mlp_bwd_workspace_bytes(n, M_cap) bytes.
 *   With mx != NULL [P1, core-idea and published-evidence sections:
 *   GroupGemm + dActivation + Quantize/Transpose; P3, three-components
 *   section: MXFP8 grouped GEMM]: DGRAD2 stays bf16 and its epilogue also
 *   writes the MXFP8 copies of the bf16 dH (row-wise, and column-wise
 *   transposed) and of A' (column-wise transposed); the other three GEMMs
 *   run on MX-scaled MFMA: DGRAD1 from dh_q x w1_q (with dx_q != NULL its
 *   epilogue also writes the row-wise MXFP8 copy of the bf16 dX_perm, the
 *   "GroupGemm + Quantize" kernel [P3, next-steps section], with dxt_q !=
 *   NULL also its column-wise copy stored transposed, and dx_perm may then
 *   be NULL), WGRAD2 from awt_q x
 *   dyt_q, WGRAD1 from xt_q x dht_q (K = the expert's row region). Only the
 *   rows of expert regions are written in the transposed copies; dh and
 *   a_w may then be NULL (their bf16 stores are skipped; no stage reads
 *   them). With
 *   dy_q != NULL DGRAD2 also runs on MX-scaled MFMA (dy_q x w2_q, then d %
 *   128 == 0 and no MOE_GATHER_ROWS), its dGLU epilogue taking that product
 *   as dA' and dS on the rewritten side as always.
 * Requires the shape constraints of moe_grouped_mlp_fwd; with mx != NULL also
 * M_cap < 2^23 (the MX wgrads address 256 rows of the transposed [rows,
 * M_cap] copies with 32-bit byte offsets).
 */
int moe_grouped_mlp_bwd(const uint16_t* x_perm, const uint16_t* w1, const uint16_t* w2,
                        const uint16_t* h, const uint16_t* dy_u, const float* topk_w,
                        const int32_t* src_of, const int32_t* row_of, const int32_t* offsets,
                        int T, int k, int E, int d, int n, int64_t M_cap, int act,
                        unsigned stages, uint16_t* dh, uint16_t* a_w, float* ds,
                        uint16_t* dx_perm, float* dw1, float* dw2,
                        void* workspace, size_t workspace_bytes, const moe_mx_bwd* mx,
                        moe_stream_t stream);

/*
 * moe_quant_mxfp8 -- standalone MXFP8 quantization of `batch` bf16 matrices
 * src [batch, R, C] [P3, three-components section: group-aware MXFP8
 * quantization; P1, problem section: the BF16 -> MXFP8 pass plus its
 * transposed copy].
 *   MOE_QUANT_ROWWISE: blocks of 32 consecutive columns;
 *     q_row [batch, R, C] codes, s_row [batch, R, C/32] scales.
 *   MOE_QUANT_COLWISE: blocks of 32 consecutive rows, stored transposed;
 *     q_col [batch, C, R] codes, s_col [batch, C, R/32] scales.
 *   Row-wise needs C % 32 == 0, column-wise R % 32 == 0. On the expert-major
 *   buffer every 32-row block lies inside one expert region (regions are
 *   128-row aligned), which is what makes the quantization group-aware.
 */
int moe_quant_mxfp8(const uint16_t* src, int batch, int64_t R, int C, int mode,
                    uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col,
                    moe_stream_t stream);

/*
 * moe_permute_quant_mxfp8 -- the expert-major permutation of x [T, d] fused
 * with its MXFP8 quantization: row r of the permuted matrix is
 * x[src_of[r] / k] (zeros where src_of[r] < 0), and it is quantized as
 * moe_quant_mxfp8 would quantize X_perm [M_cap, d], without the bf16 copy
 * ever being written [P1, problem section: the BF16 -> MXFP8 pass and its
 * transposed copy; P3, three-components section: group-aware MXFP8
 * quantization on the expert-major buffer].
 *   x [T, d] bf16, src_of [M_cap] (in, from moe_route_counts); mode, q_row
 *   [M_cap, d] + s_row [M_cap, d/32], q_col [d, M_cap] + s_col [d, M_cap/32]
 *   as in moe_quant_mxfp8 (out, every row of [0, M_cap)).
 * Requires d % 32 == 0, M_cap % 128 == 0, M_cap >= moe_capacity_rows(T, k, E),
 * 16-byte aligned x and code buffers.
 */
int moe_permute_quant_mxfp8(const uint16_t* x, const int32_t* src_of, int T, int k, int E, int d,
                            int64_t M_cap, int mode, uint8_t* q_row, uint8_t* s_row,
                            uint8_t* q_col, uint8_t* s_col, moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * The dense half of a mixture-of-experts layer: the router projection and the
 * shared expert that every token passes, their 8-bit activation checkpoints,
 * and the router's losses.
 *
 * A linear layer is z = x W + b, y = f(z) + r with x [T, K], W [K, N], z [T, N]
 * and y, r [T, NO]: NO = N, or N / 2 for the gated activations, whose columns
 * are interleaved as in w1 above (32 gate columns, then their 32 up columns).
 * K and N are multiples of 8 (N of 64 when gated) up to MOE_MAX_WIDTH; T is any
 * row count from 1 to MOE_MAX_ROWS. Pointers to tensors of 16-bit values or codes, and the
 * workspace, are 16-byte aligned. Outputs must not overlap inputs, except that
 * a residual may be the output itself.
 *
 * An 8-bit checkpoint of a [T, N] activation is its row-wise MXFP8 copy: codes
 * [T, N] and scales [T, N / 32], as moe_quant_mxfp8 writes it (N % 32 == 0): 33
 * bytes for 32 values. A rounding of one step moves a value by at most 2^-4 of
 * itself (2^-10 * 2^e below the block's normal range). It is meant for finite
 * values.
 * ------------------------------------------------------------------------- */

/* Device workspace (bytes) of a linear layer's calls: MOE_LINEAR_FWD for
 * moe_linear_fwd, MOE_LINEAR_BWD for moe_act_bwd, moe_linear_dgrad and
 * moe_linear_wgrad (which may share it, one after the other on a stream). 0 for
 * invalid shapes, and where none is needed. A workspace holds nothing between
 * calls; calls that may overlap in time (two streams, two graphs replayed side
 * by side) need one each. Host-only. */
size_t moe_linear_workspace_bytes(int T, int K, int N, int pass);

/*
 * moe_linear_fwd -- y = f(x W + b) + r in one matrix product with its epilogue.
 *   The sum over K and the epilogue are fp32; y is rounded once, to bf16, or is
 *   fp32 when y_f32 != 0 (router logits).
 *   x [T, K], w [K, N], bias [N] or NULL, residual [T, NO] or NULL (bf16, in);
 *   y [T, NO] (out). For the backward, optionally z: as bf16 (z [T, N]) and / or
 *   as an 8-bit checkpoint of its bf16 value (z_q [T, N], z_s [T, N / 32], both
 *   or neither). act: any MOE_ACT_*; with MOE_ACT_NONE there is no z to keep.
 *   Few rows (single tokens, decode batches) cut K over the chip and join the
 *   parts in a second launch, in a fixed order.
 *   workspace: moe_linear_workspace_bytes(T, K, N, MOE_LINEAR_FWD) bytes.
 */
int moe_linear_fwd(const uint16_t* x, const uint16_t* w, const uint16_t* bias, const uint16_t* residual, int T,
                   int K, int N, int act, int y_f32, void* y, uint16_t* z, uint8_t* z_q, uint8_t* z_s,
                   void* workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * moe_act_bwd -- through the activation: dz = dy f'(z) (gated: dg = dy u f'(g),
 *   du = dy f(g), interleaved like z), dbias = sum over t of dz, a = f(z).
 *   dy [T, NO] bf16 (NULL when only a is asked for); z [T, N] bf16, or z_q and
 *   z_s, its 8-bit checkpoint (neither with MOE_ACT_NONE, where dz = dy).
 *   dz [T, N] bf16, a [T, NO] bf16, dbias [N] fp32 (out; each NULL when not
 *   wanted): dbias sums the fp32 values of dz before their rounding to bf16; a
 *   is recomputed for the next layer's weight gradient.
 *   workspace: moe_linear_workspace_bytes(T, K, N, MOE_LINEAR_BWD) bytes when
 *   dbias is asked for.
 */
int moe_act_bwd(const uint16_t* dy, const uint16_t* z, const uint8_t* z_q, const uint8_t* z_s, int T, int N,
                int act, uint16_t* dz, uint16_t* a, float* dbias, void* workspace, size_t workspace_bytes,
                moe_stream_t stream);

/*
 * moe_linear_dgrad -- dx = dz W^T + r: dz [T, N], w [K, N], residual [T, K] or
 *   NULL (a gradient that reaches x by another way; may be dx itself), dx [T, K]
 *   (bf16, fp32 sums, one rounding).
 */
int moe_linear_dgrad(const uint16_t* dz, const uint16_t* w, const uint16_t* residual, int T, int K, int N,
                     uint16_t* dx, void* workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * moe_linear_wgrad -- dw = x^T dz, or dw += x^T dz when accumulate != 0 (fp32
 *   only): x [T, K] bf16, or x_q and x_s, its 8-bit checkpoint; dz [T, N] bf16;
 *   dw [K, N] fp32 when dw_f32 != 0, else bf16.
 */
int moe_linear_wgrad(const uint16_t* x, const uint8_t* x_q, const uint8_t* x_s, const uint16_t* dz, int T, int K,
                     int N, int dw_f32, int accumulate, void* dw, void* workspace, size_t workspace_bytes,
                     moe_stream_t stream);

/*
 * moe_dequant_mxfp8 -- restores an 8-bit checkpoint: out [R, C] bf16 from codes q
 *   [R, C] and scales s [R, C / 32] (row-wise, as moe_quant_mxfp8 writes them).
 *   Exact wherever code * scale is a bf16 number (all but values below bf16's
 *   smallest normal, which round to nearest). Scale 255 and codes 0x7f, 0xff are
 *   NaN. Requires C % 32 == 0.
 */
int moe_dequant_mxfp8(const uint8_t* q, const uint8_t* s, int64_t R, int C, uint16_t* out, moe_stream_t stream);

/* Device workspace (bytes) of moe_balance_loss. Host-only. */
size_t moe_balance_workspace_bytes(int T, int E, int S);

/*
 * moe_balance_loss -- the router's load-balance and z losses with the per-expert
 *   counts, per sequence. With p = softmax(logits[t]) and n_s the live tokens of
 *   sequence s:
 *     f_se = E counts[s, e] / (k n_s),  P_se = mean of p_e over the live tokens,
 *     B = mean over the sequences with a live token of sum_e f_se P_se,
 *     Z = mean over all live tokens of (log sum_e exp logits[t, e])^2,
 *     loss[0] = balance_coef B + z_coef Z, loss[1] = B, loss[2] = Z
 *   (a term whose coefficient is 0 stays out of loss[0], also where it is infinite).
 *   A token is live unless valid[t] == 0, it lies outside [seq_offsets[0],
 *   seq_offsets[S]), or it has no finite logit. Non-finite logits have
 *   probability 0, as in the router. Without a live token every loss is 0.
 *   logits [T, E] fp32, topk_idx [T, k] int32 (from moe_route_counts; entries
 *   outside [0, E) are not counted), valid [T] bytes or NULL (all valid),
 *   seq_offsets [S + 1] int32 ascending, device, or NULL with S = 1 (in);
 *   loss [3] fp32, counts [S, E] int32, prob [S, E] fp32 (P; 0 for a sequence
 *   without live tokens), tokens [S + 2] int32 (n_s, then the number of sequences
 *   with a live token, then all live tokens) (out).
 *   Sums are joined in a fixed order: the same inputs give the same bits.
 *   workspace: moe_balance_workspace_bytes(T, E, S) bytes.
 * Requires 1 <= k <= E <= MOE_MAX_EXPERTS, 1 <= S <= T <= MOE_MAX_ROWS.
 */
int moe_balance_loss(const float* logits, const int32_t* topk_idx, const uint8_t* valid,
                     const int32_t* seq_offsets, int T, int E, int k, int S, float balance_coef, float z_coef,
                     float* loss, int32_t* counts, float* prob, int32_t* tokens, void* workspace,
                     size_t workspace_bytes, moe_stream_t stream);

/*
 * moe_balance_loss_bwd -- gradient of loss[0] w.r.t. the logits (the counts have
 *   none), times the upstream gradient grad [1] fp32 (device; NULL: 1):
 *     g (balance_coef / (S' n_s) p_e (f_se - sum_j f_sj p_j) + z_coef 2 lse_t p_e / n)
 *   for live tokens, 0 for the others. counts and tokens are moe_balance_loss's
 *   outputs; logits, valid, seq_offsets and the sizes those of its call.
 *   dlogits [T, E] fp32 (out), or added to it when accumulate != 0 (the gradient
 *   that moe_route_bwd wrote); dlogits_bf16 [T, E] or NULL: the result rounded,
 *   for the projection's gradient products.
 */
int moe_balance_loss_bwd(const float* logits, const int32_t* counts, const int32_t* tokens, const uint8_t* valid,
                         const int32_t* seq_offsets, int T, int E, int k, int S, float balance_coef,
                         float z_coef, const float* grad, int accumulate, float* dlogits, uint16_t* dlogits_bf16,
                         moe_stream_t stream);

/* ---------------------------------------------------------------------------
 * Around a MoE block: the router with scores, a balance bias and groups; 4-bit
 * blocks and the experts' products with them; the norms before and after.
 * ------------------------------------------------------------------------- */

#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1
#define MOE_MAX_TOPK 64       /* largest k of moe_route_scores      */
#define MOE_MAX_GROUPS 64     /* largest number of expert groups    */

/* How tokens choose experts. */
typedef struct moe_routing {
    int score;        /* MOE_SCORE_*: s = softmax over all E, or sigmoid, of the logits           */
    int groups;       /* the E experts as so many groups of neighbours (a divisor of E); 1: none */
    int topk_groups;  /* groups that a token keeps                                              */
    int group_top;    /* a group is worth its best choice value (1) or the sum of its two best (2) */
    int renorm;       /* weights divided by their sum over the chosen k                        */
    float scale;      /* factor of all weights                                                 */
} moe_routing;

/* Device workspace (bytes) of moe_route_scores. Host-only. */
size_t moe_route_scores_workspace_bytes(int T, int k, int E);

/*
 * moe_route_scores -- moe_route_counts with a choice of scores: with s the
 *   scores of a token's logits and b a bias that takes part in the choice alone,
 *   c_e = s_e + b_e; the topk_groups groups of largest value are kept; slot j
 *   holds the expert of j-th largest c in them, and
 *   topk_w[t, j] = scale s_{e_j} (/ sum_i s_{e_i} with renorm).
 *   The order is that of the exact values (formed in 64 bits where they lie
 *   near), ties to the lower index; without a bias experts are ordered by their
 *   logits. An expert whose logit or bias is not finite (a bias of -inf takes
 *   one out of service) is chosen only when its kept groups hold too few others,
 *   lowest index first, and then weighs 0; a non-finite logit sets
 *   MOE_ERRBIT_NONFINITE_LOGIT, has no part in the softmax and none in a
 *   group's value.
 *   logits [T, E] fp32, bias [E] fp32 or NULL (in); the outputs, err_word and
 *   M_cap as of moe_route_counts.
 *   workspace: moe_route_scores_workspace_bytes(T, k, E) bytes, 16-byte aligned.
 * Requires 1 <= k <= E <= MOE_MAX_EXPERTS, k <= MOE_MAX_TOPK, at most the experts
 * of topk_groups groups, groups <= MOE_MAX_GROUPS.
 */
int moe_route_scores(const float* logits, const float* bias, const moe_routing* how, int T, int E, int k,
                     int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* offsets, int32_t* row_of,
                     int32_t* src_of, int64_t M_cap, int32_t* err_word, void* workspace, size_t workspace_bytes,
                     moe_stream_t stream);

/*
 * moe_route_scores_bwd -- gradient w.r.t. the logits given ds = dL/dtopk_w, for
 *   the experts chosen (topk_idx as moe_route_scores wrote it; the choice itself
 *   and the bias have none). An expert that weighs 0 for want of a finite logit
 *   or bias has none either, and its ds, finite or not, has no part in the others'.
 *   dlogits [T, E] fp32 (out, every element).
 */
int moe_route_scores_bwd(const float* logits, const float* bias, const moe_routing* how, const int32_t* topk_idx,
                         const float* ds, int T, int E, int k, float* dlogits, moe_stream_t stream);

/*
 * moe_quant_mxfp4 -- MXFP4 quantization of `batch` bf16 matrices src [batch, R, C]:
 *   blocks of 32 values share the smallest E8M0 scale 2^e with amax <= 6 * 2^e, so
 *   that none is clipped, and are E2M1 codes, rounded to nearest-even, two a byte
 *   (the first in the low half). A value moves by at most a quarter of itself
 *   while it lies in its block's normal range, by at most 2^(e-2) below it. A
 *   block with a NaN or an infinity takes scale 255 and is NaN as a whole.
 *   MOE_QUANT_ROWWISE: blocks along the columns; q_row [batch, R, C / 2], s_row
 *     [batch, R, C / 32]. Needs C % 32 == 0.
 *   MOE_QUANT_COLWISE: blocks along the rows, stored transposed; q_col
 *     [batch, C, R / 2], s_col [batch, C, R / 32]: weights [E, K, N] as
 *     moe_grouped_linear_mxfp4 reads them. Needs R % 32 == 0, C % 8 == 0, C < 2^30.
 *   src and the codes 16-byte aligned.
 */
int moe_quant_mxfp4(const uint16_t* src, int batch, int64_t R, int C, int mode, uint8_t* q_row, uint8_t* s_row,
                    uint8_t* q_col, uint8_t* s_col, moe_stream_t stream);

/* moe_dequant_mxfp4 -- bf16 values [R, C] of row-wise codes q [R, C / 2] and scales
 *   s [R, C / 32]; exact wherever code * scale is a bf16 number (all but a magnitude of 2^128, to
 *   which bf16's very largest round: an infinity). Requires C % 32 == 0. */
int moe_dequant_mxfp4(const uint8_t* q, const uint8_t* s, int64_t R, int C, uint16_t* out, moe_stream_t stream);

/* forms of the rows that the 4-bit product reads */
#define MOE_X_BF16 0
#define MOE_X_MXFP8 1   /* codes [rows, K], scales [rows, K / 32], as moe_quant_mxfp8 writes row-wise */
#define MOE_X_MXFP4 2   /* codes [rows, K / 2], scales [rows, K / 32], as moe_quant_mxfp4 does      */

/* Device workspace (bytes) of moe_grouped_linear_mxfp4: 0, none is needed (any pointer, or NULL). Host-only. */
size_t moe_grouped_linear_mxfp4_workspace_bytes(int T, int k, int E, int K, int N);

/*
 * moe_grouped_linear_mxfp4 -- one product of all experts with 4-bit weights:
 *   y[r] = f(x_r W_e) for the counts[e] rows r from offsets[e] of every expert e,
 *   with W_e [K, N] given transposed as MXFP4: w_q [E, N, K / 2], w_s [E, N, K / 32]
 *   (moe_quant_mxfp4 of w [E, K, N], column-wise). x_r is row r of x [M_cap, K]
 *   (the experts' buffer), or with src_of != NULL row src_of[r] / k of x [T, K]:
 *   tokens are read, and quantized, once, and not copied k times.
 *   act: any MOE_ACT_*; the gated ones take N as 32 gate and 32 up columns in turn
 *   and give y [M_cap, N / 2], the others y [M_cap, N] (bf16). Sums and f are fp32,
 *   y is rounded once; with MXFP8 rows the matrix cores add the products of 8
 *   consecutive k first, each cut off at 2^-13 of 2^(largest sum of two operands'
 *   exponents among them). Rows past an
 *   expert's counts[e] are neither read nor written, of x and y alike.
 *   T, k: the routing's sizes (the host does not know the counts).
 *   workspace: moe_grouped_linear_mxfp4_workspace_bytes(T, k, E, K, N) bytes.
 * Requires K % 32 == 0, N % 8 == 0 (64 when gated), both at most MOE_MAX_WIDTH,
 * M_cap >= moe_capacity_rows(T, k, E), 16-byte aligned x, w_q and y; gathered
 * rows within 2^31 bytes.
 */
int moe_grouped_linear_mxfp4(const void* x, const uint8_t* x_s, int x_fmt, const int32_t* src_of, int T, int k,
                             const uint8_t* w_q, const uint8_t* w_s, const int32_t* offsets, const int32_t* counts,
                             int E, int K, int N, int64_t M_cap, int act, uint16_t* y, void* workspace,
                             size_t workspace_bytes, moe_stream_t stream);

#define MOE_MAX_NORM_WIDTH 16384 /* largest d of the norms */
#define MOE_GATE_LINEAR 0        /* the gate's values as they are */
#define MOE_GATE_SIGMOID 1       /* their logistic sigmoid        */

/* Device workspace (bytes) of moe_norm_bwd and moe_post_norm_bwd where dw is asked
 * for. Host-only. */
size_t moe_norm_workspace_bytes(int T, int d);

/*
 * moe_norm_fwd -- the norm before a block, with the residual sum: total = x +
 *   residual, rounded to bf16 (both NULL: x itself is normalised), rstd = 1 /
 *   sqrt(mean(total^2) + eps), y = total rstd w.
 *   x, residual, total, y [T, d], w [d] bf16; rstd [T] fp32, or NULL. total may be
 *   x or residual, and y may be x where there is no residual.
 *   Sums are fp32, y is rounded once; the squares' mean must lie within fp32.
 * Requires d % 8 == 0, d <= MOE_MAX_NORM_WIDTH, eps > 0, 16-byte aligned bf16
 * tensors, as the three entry points below.
 */
int moe_norm_fwd(const uint16_t* x, const uint16_t* residual, const uint16_t* w, int T, int d, float eps,
                 uint16_t* total, uint16_t* y, float* rstd, moe_stream_t stream);

/*
 * moe_norm_bwd -- dx = rstd (g - h mean(g h)) + dres with h = x rstd, g = dy w; dw =
 *   sum over t of dy h. x is what was normalised (total, where there was one), so
 *   dx is the gradient of x and of the residual alike; dres [T, d] or NULL is the
 *   gradient that reaches it by the residual stream. dx bf16 (may be dy or dres),
 *   dw [d] fp32 or NULL, summed in a fixed order.
 */
int moe_norm_bwd(const uint16_t* dy, const uint16_t* x, const uint16_t* w, const float* rstd, const uint16_t* dres,
                 int T, int d, uint16_t* dx, float* dw, void* workspace, size_t workspace_bytes,
                 moe_stream_t stream);

/*
 * moe_post_norm_fwd -- after a block: out = x + scale f(gate) (y rstd w).
 *   With row_of != NULL y holds the experts' rows and the block's output is their
 *   weighted sum, rounded to bf16 as moe_combine gives it (topk_w NULL: unit
 *   weights); it is stored in total [T, d] when that is not NULL. Else y is [T, d].
 *   gate: NULL (gate_cols 0), one a token [T] (1), or one a channel [T, d] (d); f
 *   is the identity or the sigmoid (gate_act). x [T, d]: the residual stream; out
 *   may be x. rstd [T] fp32 or NULL.
 */
int moe_post_norm_fwd(const uint16_t* y, const int32_t* row_of, const float* topk_w, int k, const uint16_t* x,
                      const uint16_t* w, const uint16_t* gate, int gate_cols, int gate_act, float scale, float eps,
                      int T, int d, uint16_t* total, uint16_t* out, float* rstd, moe_stream_t stream);

/*
 * moe_post_norm_bwd -- gradients of y [T, d] (the block's output: total, where the
 *   rows were combined; moe_grouped_mlp_bwd takes dy from there), of the gate
 *   (bf16 [T, d], or fp32 [T] for one a token; NULL: not wanted) and of w (fp32,
 *   or NULL). The gradient of x is dout itself. dy may be dout.
 */
int moe_post_norm_bwd(const uint16_t* dout, const uint16_t* y, const uint16_t* w, const float* rstd,
                      const uint16_t* gate, int gate_cols, int gate_act, float scale, int T, int d, uint16_t* dy,
                      void* dgate, float* dw, void* workspace, size_t workspace_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
