// Internal launcher declarations of the dense half of the layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dense_plan.hpp"

namespace moe {

// Outputs of at least this size are stored past the caches by the streaming passes:
// a quarter of the 256 MB last-level cache, so smaller ones stay there for their reader.
constexpr int64_t kDenseStreamBytes = (int64_t)64 << 20;

// Dense linear layer (act: the MOE_ACT_* codes; N: columns of W, 2n when gated)
size_t dense_part_bytes(int64_t M, int64_t N, int64_t K, DensePass pass);
int launch_linear_fwd(const uint16_t* x, const uint16_t* w, const uint16_t* bias, const uint16_t* res, int T,
                      int K, int N, int act, int y_f32, void* y, uint16_t* z, uint8_t* z_q, uint8_t* z_s,
                      void* ws, hipStream_t s);
int launch_linear_dgrad(const uint16_t* dz, const uint16_t* w, const uint16_t* res, int T, int K, int N,
                        uint16_t* dx, void* ws, hipStream_t s);
int launch_linear_wgrad(const uint16_t* x, const uint8_t* x_q, const uint8_t* x_s, const uint16_t* dz, int T,
                        int K, int N, int dw_f32, int accumulate, void* dw, void* ws, hipStream_t s);
size_t linear_wgrad_bytes(int T, int K, int N, bool x8);
size_t act_part_bytes(int T, int N);
int launch_act_bwd(const uint16_t* dy, const uint16_t* z, const uint8_t* z_q, const uint8_t* z_s, int T, int N,
                   int act, uint16_t* dz, uint16_t* a, float* dbias, void* ws, hipStream_t s);
int launch_dequant_mxfp8(const uint8_t* q, const uint8_t* sc, int64_t R, int C, uint16_t* out, hipStream_t s);

// Router losses
size_t balance_workspace_bytes(int T, int E, int S);
int launch_balance_loss(const float* logits, const int32_t* topk_idx, const uint8_t* valid, const int32_t* seq,
                        int T, int E, int k, int S, float cb, float cz, float* loss, int32_t* counts,
                        float* prob, int32_t* tokens, void* ws, hipStream_t s);
int launch_balance_loss_bwd(const float* logits, const int32_t* counts, const int32_t* tokens,
                            const uint8_t* valid, const int32_t* seq, int T, int E, int k, int S, float cb,
                            float cz, const float* grad, int accumulate, float* dlogits, uint16_t* dlogits16,
                            hipStream_t s);

}  // namespace moe
