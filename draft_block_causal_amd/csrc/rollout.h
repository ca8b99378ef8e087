// Host-side launchers of the 8-bit roll-out and policy-training kernels
// (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "policy_plan.h"

namespace domino {

// Rows in 8 bits with one scale a row (quantize.hip); dtype 0 = f32, 1 = bf16;
// cols % 32 == 0, cols <= 8192.
hipError_t launch_quantize_rows(int rows, int cols, int dtype, const void* x, int8_t* q, float* scale, hipStream_t s);

// C[m][n] = a_scale[m] w_scale[n] sum_k A[m][k] W[n][k] (gemm_i8.hip): int8
// operands, K % 32 == 0, K <= 8192, rows contiguous, exact int32 sums.
hipError_t launch_gemm_i8(const int8_t* A, const float* a_scale, int M, const int8_t* W, const float* w_scale, int N,
                          int K, float* C, int num_cu, hipStream_t s);

// Drafted-token log-probabilities and the clipped policy loss (policy.hip);
// the workspace follows policy_plan(B, K, V).
hipError_t launch_token_logprobs(int B, int K, int V, const float* logits, const int32_t* tokens, const float* weights,
                                 double temperature, float* logp, float* entropy, const PolicyPlan& plan,
                                 void* workspace, int num_cu, hipStream_t s);
hipError_t launch_policy_loss(const PolicyArgs& a, const PolicyPlan& plan, void* workspace, int num_cu,
                              hipStream_t s);

}  // namespace domino
