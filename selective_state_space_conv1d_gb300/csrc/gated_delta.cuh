// gated_delta.cuh - the gates and the argument block shared by the kernels of
// the gated delta rule:
//
//   alpha_t = exp(-exp(A_log) softplus(a_t + dt_bias)),  beta_t = sigmoid(b_t)
//   S_t = alpha_t S_{t-1} + beta_t (v_t - alpha_t S_{t-1} k_t) k_t^T
//   y_t = scale S_t q_t                                   S in R^{dv x dk}
//
// The decays multiply over thousands of tokens, so an error of the gate's
// exponent is an error of the state: softplus and the exponentials are the
// accurate functions here (a few per token and head, against 7 dk dv flops).
// The selective scan's two-MUFU softplus has an absolute error near 1e-7, which
// exp(A_log) (up to 16 and more) would bring to 2e-6 of the state.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "device_math.cuh"
#include "launch.h"

namespace mamba {

// log(alpha), <= 0; -inf for a = +inf (alpha = 0: the state is dropped)
__device__ __forceinline__ float gdr_log_alpha(float a, float dt_bias, float neg_A) {
  const float v = a + dt_bias;
  return neg_A * (fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))));
}

__device__ __forceinline__ float gdr_beta(float b) { return 1.0f / (1.0f + expf(-b)); }

}  // namespace mamba
