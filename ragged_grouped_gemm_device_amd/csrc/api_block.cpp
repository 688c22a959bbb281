// extern "C" entry points of the operators around a MoE block (router with scores, bias and groups;
// 4-bit blocks and the experts' products with them; norms): host-side validation, then kernel launches
// on the caller's stream, as in api.cpp.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <cmath>
#include <initializer_list>

#include "../../include/moe.h"
#include "block_launch.hpp"

namespace {

inline hipStream_t S(moe_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

// every given (non-NULL) pointer is 16-byte aligned
bool aligned(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
    return true;
}

int status(int rc) { return rc ? MOE_ERR_LAUNCH : MOE_OK; }

int check_routing(const moe_routing* how, int T, int E, int k) {
    if (!how || T <= 0 || E <= 0 || k <= 0 || k > E || E > MOE_MAX_EXPERTS) return MOE_ERR_INVALID_ARG;
    if (how->score != MOE_SCORE_SOFTMAX && how->score != MOE_SCORE_SIGMOID) return MOE_ERR_UNSUPPORTED;
    if (how->groups <= 0 || E % how->groups || how->topk_groups <= 0 || how->topk_groups > how->groups)
        return MOE_ERR_INVALID_ARG;
    if (how->group_top != 1 && how->group_top != 2) return MOE_ERR_INVALID_ARG;
    if (k > how->topk_groups * (E / how->groups)) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(how->scale)) return MOE_ERR_INVALID_ARG;
    if (k > MOE_MAX_TOPK || how->groups > MOE_MAX_GROUPS) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int check_norm(int T, int d) {
    if (T <= 0 || d <= 0) return MOE_ERR_INVALID_ARG;
    if (T > MOE_MAX_ROWS || d % 8 || d > MOE_MAX_NORM_WIDTH) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// the gate of a post norm: none, one a token, or one a channel
int check_gate(const uint16_t* gate, int gate_cols, int gate_act, int d) {
    if (!gate != (gate_cols == 0) || (gate_cols != 0 && gate_cols != 1 && gate_cols != d)) return MOE_ERR_INVALID_ARG;
    if (gate_act != MOE_GATE_LINEAR && gate_act != MOE_GATE_SIGMOID) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool has_space(const void* ws, size_t bytes, size_t need) {
    return need == 0 || (ws && bytes >= need && aligned({ws}));
}

}  // namespace

extern "C" {

size_t moe_route_scores_workspace_bytes(int T, int k, int E) {
    if (moe_capacity_rows(T, k, E) < 0) return 0;
    return moe::route_scores_workspace_bytes(T, k, E);
}

int moe_route_scores(const float* logits, const float* bias, const moe_routing* how, int T, int E, int k,
                     int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* offsets, int32_t* row_of,
                     int32_t* src_of, int64_t M_cap, int32_t* err_word, void* workspace, size_t workspace_bytes,
                     moe_stream_t stream) {
    const int rc = check_routing(how, T, E, k);
    if (rc != MOE_OK) return rc;
    if (!logits || !topk_idx || !topk_w || !counts || !offsets || !row_of || !src_of) return MOE_ERR_INVALID_ARG;
    if (M_cap < moe_capacity_rows(T, k, E) || M_cap > INT32_MAX) return MOE_ERR_WORKSPACE;
    if (!has_space(workspace, workspace_bytes, moe::route_scores_workspace_bytes(T, k, E))) return MOE_ERR_WORKSPACE;
    moe::RouteCall c{};
    c.logits = logits, c.bias = bias, c.T = T, c.E = E, c.k = k;
    c.sigmoid = how->score == MOE_SCORE_SIGMOID, c.groups = how->groups, c.kept = how->topk_groups;
    c.top = how->group_top, c.renorm = how->renorm != 0, c.scale = how->scale;
    c.topk_idx = topk_idx, c.topk_w = topk_w, c.counts = counts, c.offsets = offsets, c.row_of = row_of;
    c.src_of = src_of, c.M_cap = M_cap, c.err_word = err_word, c.ws = workspace;
    return status(moe::launch_route_scores(c, S(stream)));
}

int moe_route_scores_bwd(const float* logits, const float* bias, const moe_routing* how, const int32_t* topk_idx,
                         const float* ds, int T, int E, int k, float* dlogits, moe_stream_t stream) {
    const int rc = check_routing(how, T, E, k);
    if (rc != MOE_OK) return rc;
    if (!logits || !topk_idx || !ds || !dlogits) return MOE_ERR_INVALID_ARG;
    if (T > MOE_MAX_ROWS) return MOE_ERR_UNSUPPORTED;
    return status(moe::launch_route_scores_bwd(logits, bias, topk_idx, ds, T, E, k, how->score == MOE_SCORE_SIGMOID,
                                               how->renorm != 0, how->scale, dlogits, S(stream)));
}

int moe_quant_mxfp4(const uint16_t* src, int batch, int64_t R, int C, int mode, uint8_t* q_row, uint8_t* s_row,
                    uint8_t* q_col, uint8_t* s_col, moe_stream_t stream) {
    if (!src || batch <= 0 || R <= 0 || C <= 0) return MOE_ERR_INVALID_ARG;
    if (mode <= 0 || (mode & ~(MOE_QUANT_ROWWISE | MOE_QUANT_COLWISE))) return MOE_ERR_INVALID_ARG;
    if ((mode & MOE_QUANT_ROWWISE) && (!q_row || !s_row)) return MOE_ERR_INVALID_ARG;
    if ((mode & MOE_QUANT_COLWISE) && (!q_col || !s_col)) return MOE_ERR_INVALID_ARG;
    if (!aligned({src, q_row, q_col})) return MOE_ERR_INVALID_ARG;
    if (C % 8 || ((mode & MOE_QUANT_ROWWISE) && C % MOE_MX_BLOCK)) return MOE_ERR_UNSUPPORTED;
    // a launch holds 65535 workgroups of 256 rows, and below 2^32 threads, four a column
    if ((mode & MOE_QUANT_COLWISE) && (R % MOE_MX_BLOCK || (R + 255) / 256 > 65535 || C >= 1 << 30)) return MOE_ERR_UNSUPPORTED;
    if (R > ((int64_t)1 << 40) / C / batch || batch > 65535) return MOE_ERR_UNSUPPORTED;
    return status(moe::launch_quant_mxfp4(src, batch, R, C, mode, q_row, s_row, q_col, s_col, S(stream)));
}

int moe_dequant_mxfp4(const uint8_t* q, const uint8_t* s, int64_t R, int C, uint16_t* out, moe_stream_t stream) {
    if (R <= 0 || C <= 0 || !q || !s || !out || !aligned({q, out})) return MOE_ERR_INVALID_ARG;
    if (C % MOE_MX_BLOCK || R > ((int64_t)1 << 40) / C) return MOE_ERR_UNSUPPORTED;
    return status(moe::launch_dequant_mxfp4(q, s, R, C, out, S(stream)));
}

size_t moe_grouped_linear_mxfp4_workspace_bytes(int T, int k, int E, int K, int N) {
    return 0;
}

int moe_grouped_linear_mxfp4(const void* x, const uint8_t* x_s, int x_fmt, const int32_t* src_of, int T, int k,
                             const uint8_t* w_q, const uint8_t* w_s, const int32_t* offsets, const int32_t* counts,
                             int E, int K, int N, int64_t M_cap, int act, uint16_t* y, void* workspace,
                             size_t workspace_bytes, moe_stream_t stream) {
    const int64_t cap = moe_capacity_rows(T, k, E);
    if (cap < 0 || K <= 0 || N <= 0) return MOE_ERR_INVALID_ARG;
    if (!x || !w_q || !w_s || !offsets || !counts || !y || !aligned({x, w_q, y})) return MOE_ERR_INVALID_ARG;
    if (x_fmt != MOE_X_BF16 && x_fmt != MOE_X_MXFP8 && x_fmt != MOE_X_MXFP4) return MOE_ERR_UNSUPPORTED;
    if (!x_s != (x_fmt == MOE_X_BF16)) return MOE_ERR_INVALID_ARG;
    if (act < MOE_ACT_SWIGLU || act > MOE_ACT_GELU) return MOE_ERR_UNSUPPORTED;
    const bool gated = act == MOE_ACT_SWIGLU || act == MOE_ACT_GEGLU;
    if (K % MOE_MX_BLOCK || N % (gated ? 2 * MOE_GLU_INTERLEAVE : 8)) return MOE_ERR_UNSUPPORTED;
    if (K > MOE_MAX_WIDTH || N > MOE_MAX_WIDTH) return MOE_ERR_UNSUPPORTED;
    if (M_cap < cap || M_cap > INT32_MAX) return MOE_ERR_WORKSPACE;
    // gathered rows are addressed from x with 32-bit byte offsets
    const int64_t row = x_fmt == MOE_X_BF16 ? 2 * (int64_t)K : x_fmt == MOE_X_MXFP8 ? K : K / 2;
    if (src_of && T * row > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    // tiles are counted in 32 bits
    if ((cap / 64 + E) * ((N + 63) / 64) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    return status(moe::launch_experts4({x, x_s, x_fmt, src_of, T, k, w_q, w_s, offsets, counts, E, N, K, M_cap, act, y},
                                       S(stream)));
}

size_t moe_norm_workspace_bytes(int T, int d) {
    return check_norm(T, d) == MOE_OK ? moe::norm_workspace_bytes(T, d) : 0;
}

int moe_norm_fwd(const uint16_t* x, const uint16_t* residual, const uint16_t* w, int T, int d, float eps,
                 uint16_t* total, uint16_t* y, float* rstd, moe_stream_t stream) {
    const int rc = check_norm(T, d);
    if (rc != MOE_OK) return rc;
    if (!x || !w || !y || !aligned({x, residual, w, total, y}) || !(eps > 0.f)) return MOE_ERR_INVALID_ARG;
    if (!residual != !total) return MOE_ERR_INVALID_ARG;
    return status(moe::launch_norm_fwd({x, residual, w, T, d, eps, total, y, rstd}, S(stream)));
}

int moe_norm_bwd(const uint16_t* dy, const uint16_t* x, const uint16_t* w, const float* rstd, const uint16_t* dres,
                 int T, int d, uint16_t* dx, float* dw, void* workspace, size_t workspace_bytes,
                 moe_stream_t stream) {
    const int rc = check_norm(T, d);
    if (rc != MOE_OK) return rc;
    if (!dy || !x || !w || !rstd || !dx || !aligned({dy, x, w, dres, dx, dw})) return MOE_ERR_INVALID_ARG;
    if (dw && !has_space(workspace, workspace_bytes, moe::norm_workspace_bytes(T, d))) return MOE_ERR_WORKSPACE;
    return status(moe::launch_norm_bwd({dy, x, w, rstd, dres, T, d, dx, dw}, workspace, S(stream)));
}

int moe_post_norm_fwd(const uint16_t* y, const int32_t* row_of, const float* topk_w, int k, const uint16_t* x,
                      const uint16_t* w, const uint16_t* gate, int gate_cols, int gate_act, float scale, float eps,
                      int T, int d, uint16_t* total, uint16_t* out, float* rstd, moe_stream_t stream) {
    int rc = check_norm(T, d);
    if (rc == MOE_OK) rc = check_gate(gate, gate_cols, gate_act, d);
    if (rc != MOE_OK) return rc;
    if (!y || !x || !w || !out || !aligned({y, x, w, gate_cols > 1 ? gate : nullptr, total, out}))
        return MOE_ERR_INVALID_ARG;
    if (!(eps > 0.f) || !std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
    if (row_of ? k <= 0 || k > MOE_MAX_EXPERTS : topk_w || total) return MOE_ERR_INVALID_ARG;
    return status(moe::launch_post_norm_fwd({y, row_of, topk_w, k, x, w, gate, gate_cols, gate_act == MOE_GATE_SIGMOID,
                                             scale, eps, T, d, total, out, rstd}, S(stream)));
}

int moe_post_norm_bwd(const uint16_t* dout, const uint16_t* y, const uint16_t* w, const float* rstd,
                      const uint16_t* gate, int gate_cols, int gate_act, float scale, int T, int d, uint16_t* dy,
                      void* dgate, float* dw, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    int rc = check_norm(T, d);
    if (rc == MOE_OK) rc = check_gate(gate, gate_cols, gate_act, d);
    if (rc != MOE_OK) return rc;
    if (!dout || !y || !w || !rstd || !dy || (dgate && !gate)) return MOE_ERR_INVALID_ARG;
    if (!aligned({dout, y, w, gate_cols > 1 ? gate : nullptr, gate_cols > 1 ? dgate : nullptr, dy, dw}))
        return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
    if (dw && !has_space(workspace, workspace_bytes, moe::norm_workspace_bytes(T, d))) return MOE_ERR_WORKSPACE;
    return status(moe::launch_post_norm_bwd({dout, y, w, rstd, gate, gate_cols, gate_act == MOE_GATE_SIGMOID, scale, T,
                                             d, dy, dgate, dw}, workspace, S(stream)));
}

}  // extern "C"
