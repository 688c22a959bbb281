// Internal launcher declarations of the operators around a MoE block: the router with scores,
// bias and groups, 4-bit blocks and the experts' products with them, and the norms.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// ---- router
constexpr int kRouteMaxTopk = 64, kRouteMaxGroups = 64;

struct RouteCall {
    const float *logits, *bias;  // bias nullable
    int T, E, k, sigmoid, groups, kept, top, renorm;
    float scale;
    int32_t* topk_idx;
    float* topk_w;
    int32_t *counts, *offsets, *row_of, *src_of;
    int64_t M_cap;
    int32_t* err_word;  // nullable
    void* ws;
};
size_t route_scores_workspace_bytes(int T, int k, int E);
int launch_route_scores(const RouteCall& c, hipStream_t s);
int launch_route_scores_bwd(const float* logits, const float* bias, const int32_t* topk_idx, const float* ds, int T,
                            int E, int k, int sigmoid, int renorm, float scale, float* dlogits, hipStream_t s);

// ---- 4-bit blocks (MXFP4: E2M1 codes, two a byte, the first in the low half; E8M0 scales over 32)
int launch_quant_mxfp4(const uint16_t* src, int batch, int64_t R, int C, int mode, uint8_t* q_row, uint8_t* s_row,
                       uint8_t* q_col, uint8_t* s_col, hipStream_t s);
int launch_dequant_mxfp4(const uint8_t* q, const uint8_t* sc, int64_t R, int C, uint16_t* out, hipStream_t s);

// ---- the experts' product with 4-bit weights
struct Experts4Call {
    const void* x;
    const uint8_t* x_s;
    int fmt;                // of x: 0 bf16, 1 MXFP8, 2 MXFP4
    const int32_t* src_of;  // nullable
    int T, k;
    const uint8_t *w_q, *w_s;
    const int32_t *offsets, *counts;
    int E, N, K;
    int64_t M_cap;
    int act;
    uint16_t* y;
};
int launch_experts4(const Experts4Call& c, hipStream_t s);

// ---- norms
constexpr int kNormMaxWidth = 16384;

struct NormFwd {
    const uint16_t *x, *res, *w;  // res nullable
    int T, d;
    float eps;
    uint16_t *total, *y;  // total nullable
    float* rstd;          // nullable
};
struct NormBwd {
    const uint16_t *dy, *x, *w;
    const float* rstd;
    const uint16_t* dres;  // nullable
    int T, d;
    uint16_t* dx;
    float* dw;  // nullable
};
struct PostNormFwd {
    const uint16_t* y;      // [T, d], or the experts' rows with row_of
    const int32_t* row_of;  // nullable
    const float* topk_w;    // nullable
    int k;
    const uint16_t *x, *w, *gate;  // gate nullable
    int gate_cols, sigmoid;
    float scale, eps;
    int T, d;
    uint16_t *total, *out;  // total nullable
    float* rstd;            // nullable
};
struct PostNormBwd {
    const uint16_t *dout, *y, *w;
    const float* rstd;
    const uint16_t* gate;
    int gate_cols, sigmoid;
    float scale;
    int T, d;
    uint16_t* dy;
    void* dgate;  // bf16 [T, d] or fp32 [T]; nullable
    float* dw;    // nullable
};
size_t norm_workspace_bytes(int T, int d);
int launch_norm_fwd(const NormFwd& p, hipStream_t s);
int launch_norm_bwd(const NormBwd& p, void* ws, hipStream_t s);
int launch_post_norm_fwd(const PostNormFwd& p, hipStream_t s);
int launch_post_norm_bwd(const PostNormBwd& p, void* ws, hipStream_t s);

}  // namespace moe
