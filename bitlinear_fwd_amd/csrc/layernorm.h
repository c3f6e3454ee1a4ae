// Layer normalisation launchers (layernorm.hip); arguments validated by the C ABI.
#pragma once
#include "bl_internal.h"

namespace bl {

hipError_t launch_layernorm(const void* X, int bf16, int64_t M, int64_t K, const float* weight, const float* bias,
                            float eps, void* Y, float* mean, float* rstd, hipStream_t s);

// Launch plan of the backward pass: how many partial rows of the weight and bias gradients the
// first launch writes, and the bytes they take.
struct LnBwdPlan {
  int rows = 0;         // rows of a workgroup at once (0: the long-row form)
  int threads = 0;      // that share a row
  int groups = 0;       // of 8 elements per thread
  int64_t wgs = 0;      // workgroups of the first launch
  int64_t parts = 0;    // partial rows
  int64_t ws_bytes = 0;
};
LnBwdPlan plan_layernorm_backward(int64_t M, int64_t K);
hipError_t launch_layernorm_backward(const void* dY, const void* X, int bf16, int64_t M, int64_t K,
                                     const float* weight, const float* mean, const float* rstd, void* dX, float* dW,
                                     float* dB, float* workspace, hipStream_t s);

}  // namespace bl
