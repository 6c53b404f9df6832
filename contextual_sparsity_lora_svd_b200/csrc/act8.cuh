// Activation checkpoints in 8 bits (act8.cu).
#pragma once

#include "common.cuh"

namespace slora {

constexpr int kActBlock = 32;  // channels that share a step
inline int64_t act8_cols(int64_t d) { return (d + kActBlock - 1) / kActBlock * kActBlock; }

slora_status act8_pack_run(int dt, int64_t T, int64_t d, const void* X, int64_t ldx,
                           const slora_act8& out, cudaStream_t st);
slora_status act8_unpack_run(int dt, int64_t T, int64_t d, const slora_act8& in, void* X,
                             int64_t ldx, cudaStream_t st);

// RMS norm that writes checkpoints of H and / or N (null: not written), and
// its backward from H's checkpoint (norm.cu).
slora_status rmsnorm_fwd_act8_run(const void* X, const void* A, const void* g, int64_t T,
                                  int64_t d, float eps, void* Hout, void* N, float* rstd,
                                  const slora_act8* H8, const slora_act8* N8, cudaStream_t st);
slora_status rmsnorm_bwd_act8_run(const slora_act8& H8, const float* rstd, const void* g,
                                  const void* dN0, const void* dN1, const void* dN2,
                                  const void* dRes, int64_t T, int64_t d, void* dX,
                                  cudaStream_t st);

}  // namespace slora
