// extern "C" entry points of the dense half of the layer (linear layer, 8-bit
// checkpoints, router losses): host-side validation, then kernel launches on the
// caller's stream, as in api.cpp.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "../../include/moe.h"
#include "dense_launch.hpp"

namespace {

inline hipStream_t S(moe_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

// every given (non-NULL) pointer is 16-byte aligned
bool aligned(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
    return true;
}

bool gated(int act) { return act == MOE_ACT_SWIGLU || act == MOE_ACT_GEGLU; }

int check_linear(int T, int K, int N, int act) {
    if (T <= 0 || K <= 0 || N <= 0) return MOE_ERR_INVALID_ARG;
    if (T > MOE_MAX_ROWS) return MOE_ERR_UNSUPPORTED;  // row numbers past a tile's end stay 32-bit
    if (act < MOE_ACT_SWIGLU || act > MOE_ACT_GELU) return MOE_ERR_UNSUPPORTED;
    if (K % 8 || N % 8 || (gated(act) && N % (2 * MOE_GLU_INTERLEAVE))) return MOE_ERR_UNSUPPORTED;
    if (K > MOE_MAX_WIDTH || N > MOE_MAX_WIDTH) return MOE_ERR_UNSUPPORTED;
    // tiles of any of the three products are counted in 32 bits
    const int64_t wide = (std::max(K, N) + 127) / 128;
    if (((int64_t)T + 127) / 128 * wide >= (int64_t)1 << 30) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// an 8-bit checkpoint is given whole, and its rows are whole blocks
int check_mx(const uint8_t* q, const uint8_t* s, int C) {
    if (!q != !s) return MOE_ERR_INVALID_ARG;
    if (q && C % MOE_MX_BLOCK) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool has_space(const void* ws, size_t bytes, size_t need) {
    return need == 0 || (ws && bytes >= need && aligned({ws}));
}

int status(int rc) { return rc ? MOE_ERR_LAUNCH : MOE_OK; }

}  // namespace

extern "C" {

size_t moe_linear_workspace_bytes(int T, int K, int N, int pass) {
    if (check_linear(T, K, N, MOE_ACT_NONE) != MOE_OK) return 0;
    const size_t fwd = moe::dense_part_bytes(T, N, K, moe::kForward);
    const size_t bwd = std::max({moe::dense_part_bytes(T, K, N, moe::kDgrad), moe::linear_wgrad_bytes(T, K, N, true),
                                 moe::act_part_bytes(T, N)});
    return std::max(pass & MOE_LINEAR_FWD ? fwd : 0, pass & MOE_LINEAR_BWD ? bwd : 0);
}

int moe_linear_fwd(const uint16_t* x, const uint16_t* w, const uint16_t* bias, const uint16_t* residual, int T,
                   int K, int N, int act, int y_f32, void* y, uint16_t* z, uint8_t* z_q, uint8_t* z_s,
                   void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    int rc = check_linear(T, K, N, act);
    if (rc == MOE_OK) rc = check_mx(z_q, z_s, N);
    if (rc != MOE_OK) return rc;
    if (!x || !w || !y || !aligned({x, w, bias, residual, y, z, z_q})) return MOE_ERR_INVALID_ARG;
    if (act == MOE_ACT_NONE && (z || z_q)) return MOE_ERR_INVALID_ARG;
    if (!has_space(workspace, workspace_bytes, moe::dense_part_bytes(T, N, K, moe::kForward))) return MOE_ERR_WORKSPACE;
    return status(moe::launch_linear_fwd(x, w, bias, residual, T, K, N, act, y_f32, y, z, z_q, z_s, workspace,
                                         S(stream)));
}

int moe_act_bwd(const uint16_t* dy, const uint16_t* z, const uint8_t* z_q, const uint8_t* z_s, int T, int N,
                int act, uint16_t* dz, uint16_t* a, float* dbias, void* workspace, size_t workspace_bytes,
                moe_stream_t stream) {
    int rc = check_linear(T, 8, N, act);
    if (rc == MOE_OK) rc = check_mx(z_q, z_s, N);
    if (rc != MOE_OK) return rc;
    if (!aligned({dy, z, z_q, dz, a})) return MOE_ERR_INVALID_ARG;
    if (!dz && !a && !dbias) return MOE_ERR_INVALID_ARG;
    if ((dz || dbias) && !dy) return MOE_ERR_INVALID_ARG;
    if (act == MOE_ACT_NONE ? (a || z || z_q) : (!z == !z_q)) return MOE_ERR_INVALID_ARG;
    if (dbias && !has_space(workspace, workspace_bytes, moe::act_part_bytes(T, N))) return MOE_ERR_WORKSPACE;
    return status(moe::launch_act_bwd(dy, z, z_q, z_s, T, N, act, dz, a, dbias, workspace, S(stream)));
}

int moe_linear_dgrad(const uint16_t* dz, const uint16_t* w, const uint16_t* residual, int T, int K, int N,
                     uint16_t* dx, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    const int rc = check_linear(T, K, N, MOE_ACT_NONE);
    if (rc != MOE_OK) return rc;
    if (!dz || !w || !dx || !aligned({dz, w, residual, dx})) return MOE_ERR_INVALID_ARG;
    if (!has_space(workspace, workspace_bytes, moe::dense_part_bytes(T, K, N, moe::kDgrad))) return MOE_ERR_WORKSPACE;
    return status(moe::launch_linear_dgrad(dz, w, residual, T, K, N, dx, workspace, S(stream)));
}

int moe_linear_wgrad(const uint16_t* x, const uint8_t* x_q, const uint8_t* x_s, const uint16_t* dz, int T, int K,
                     int N, int dw_f32, int accumulate, void* dw, void* workspace, size_t workspace_bytes,
                     moe_stream_t stream) {
    int rc = check_linear(T, K, N, MOE_ACT_NONE);
    if (rc == MOE_OK) rc = check_mx(x_q, x_s, K);
    if (rc != MOE_OK) return rc;
    if (!x == !x_q || !dz || !dw || !aligned({x, x_q, dz, dw})) return MOE_ERR_INVALID_ARG;
    if (accumulate && !dw_f32) return MOE_ERR_UNSUPPORTED;
    if (!has_space(workspace, workspace_bytes, moe::linear_wgrad_bytes(T, K, N, x_q != nullptr)))
        return MOE_ERR_WORKSPACE;
    return status(moe::launch_linear_wgrad(x, x_q, x_s, dz, T, K, N, dw_f32, accumulate, dw, workspace, S(stream)));
}

int moe_dequant_mxfp8(const uint8_t* q, const uint8_t* s, int64_t R, int C, uint16_t* out, moe_stream_t stream) {
    if (R <= 0 || C <= 0 || !q || !s || !out || !aligned({q, out})) return MOE_ERR_INVALID_ARG;
    if (C % MOE_MX_BLOCK) return MOE_ERR_UNSUPPORTED;
    return status(moe::launch_dequant_mxfp8(q, s, R, C, out, S(stream)));
}

static int check_balance(int T, int E, int k, int S) {
    if (T <= 0 || E <= 0 || E > MOE_MAX_EXPERTS || k <= 0 || k > E || S <= 0 || S > T) return MOE_ERR_INVALID_ARG;
    if (T > MOE_MAX_ROWS || (int64_t)S * ((E + 31) / 32) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

size_t moe_balance_workspace_bytes(int T, int E, int S) {
    return check_balance(T, E, 1, S) == MOE_OK ? moe::balance_workspace_bytes(T, E, S) : 0;
}

int moe_balance_loss(const float* logits, const int32_t* topk_idx, const uint8_t* valid,
                     const int32_t* seq_offsets, int T, int E, int k, int S_, float balance_coef, float z_coef,
                     float* loss, int32_t* counts, float* prob, int32_t* tokens, void* workspace,
                     size_t workspace_bytes, moe_stream_t stream) {
    const int rc = check_balance(T, E, k, S_);
    if (rc != MOE_OK) return rc;
    if (!logits || !topk_idx || !loss || !counts || !prob || !tokens) return MOE_ERR_INVALID_ARG;
    if (!seq_offsets && S_ != 1) return MOE_ERR_INVALID_ARG;
    if (!has_space(workspace, workspace_bytes, moe::balance_workspace_bytes(T, E, S_))) return MOE_ERR_WORKSPACE;
    return status(moe::launch_balance_loss(logits, topk_idx, valid, seq_offsets, T, E, k, S_, balance_coef, z_coef,
                                           loss, counts, prob, tokens, workspace, S(stream)));
}

int moe_balance_loss_bwd(const float* logits, const int32_t* counts, const int32_t* tokens, const uint8_t* valid,
                         const int32_t* seq_offsets, int T, int E, int k, int S_, float balance_coef,
                         float z_coef, const float* grad, int accumulate, float* dlogits, uint16_t* dlogits_bf16,
                         moe_stream_t stream) {
    const int rc = check_balance(T, E, k, S_);
    if (rc != MOE_OK) return rc;
    if (!logits || !counts || !tokens || !dlogits) return MOE_ERR_INVALID_ARG;
    if (!seq_offsets && S_ != 1) return MOE_ERR_INVALID_ARG;
    return status(moe::launch_balance_loss_bwd(logits, counts, tokens, valid, seq_offsets, T, E, k, S_, balance_coef,
                                               z_coef, grad, accumulate, dlogits, dlogits_bf16, S(stream)));
}

}  // extern "C"
