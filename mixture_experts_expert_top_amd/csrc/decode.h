// Launcher of the whole expert layer for few tokens (decode.hip) for the
// C-ABI layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// tokens of a call: a wave has a lane for each
constexpr int kFewTokens = 64;
// d and f of a call: byte offsets within a few rows stay below 2^32
constexpr int64_t kFewWidth = int64_t{1} << 20;

struct LayerArgs {
  const uint16_t* x;           // [T][d]
  const uint16_t* w_g;         // [E][d], or null: logits
  const float* bias;
  const float* logits;
  int T, d, f, E, k, renorm;
  const void* w_gu;            // bf16, or codes with scales
  const uint8_t* w_gu_scales;
  const void* w2;
  const uint8_t* w2_scales;
  const uint16_t* y_add;
  int32_t* topk_idx;
  float* topk_w;
  uint16_t* y;
};

size_t layer_fwd_workspace(int64_t T, int k, int E, int64_t d, int64_t f);
hipError_t launch_layer_fwd(bool mx, const LayerArgs& a, void* ws,
                            hipStream_t s);

}  // namespace moe
