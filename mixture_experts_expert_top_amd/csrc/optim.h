// Launchers of the optimizer's kernels (optim.hip) for the C-ABI layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// values of an 8-bit moment that share one scale
constexpr int kStateBlock = MOE_ADAMW_BLOCK;
// largest tensor: its chunks fit one launch
constexpr int64_t kMaxTensor = int64_t{1} << 34;

size_t grad_norm_workspace();
hipError_t launch_grad_norm(const moe_grad* grads, int count, float* norm,
                            void* ws, hipStream_t s);

struct AdamwHyper {
  float b1, c1, b2, c2;        // beta and 1 - beta, each rounded once
  double log_b1, log_b2;       // natural logarithms (-inf for beta 0)
  float eps;
  float max_norm;
  const int64_t* step;
  const float* lr;
  const float* norm;           // may be null
};
hipError_t launch_adamw(bool bits8, const moe_adamw_tensor* t, int count,
                        const AdamwHyper& h, hipStream_t s);

}  // namespace moe
