// Rotation of q and k rows with optional per-head norms (see qk_rotary.cu).
#pragma once

#include "common.cuh"

namespace slora {

constexpr int kMaxHeadDim = 256;
constexpr int kMaxSlicedChannels = 32768;  // heads * head_dim of a sliced tensor

// A checked slora_rotary: turns per position of each pair in units of 2^-64
// turn (exact modulo one turn under integer multiplication), and the factor on
// the rotated channels.
struct RotaryPlan {
  int inter = 0;
  int dims = 0;
  float mscale = 1.0f;
  unsigned long long turns[kMaxHeadDim / 2] = {};
};
slora_status rotary_plan(const char* fn, const slora_rotary* rot, int head_dim, RotaryPlan* out);

struct QkDesc {
  int dt, gdt;  // element types of x, Y, dX, g and of dY
  TokenInfo ti;
  int head_dim;
  float eps;
  RotaryPlan rot;
  const int32_t* pos;
  slora_qk_rows part[2];
  int nparts;
};
// With plan == true only the arena is sized (no pointer is touched).
slora_status qk_rotary_run(const QkDesc& D, bool backward, const slora_tokens* tok, Arena& ar,
                           bool plan, cudaStream_t st);
// Raised when a sliced tensor's channel list held a bad or repeated entry.
slora_status qk_check_error(bool clear);

}  // namespace slora
