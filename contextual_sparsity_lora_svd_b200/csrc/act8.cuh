// Activation checkpoints in 8 bits and the contraction that reads them (act8.cu).
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

// out[q * ldo + (kmap ? kmap[c] : c)] (+)= scale * sum over m < M of P(m, q) X(m, c)
// for q < cols, c < K, X a checkpoint of M rows and K channels and P given as
// its bf16 terms, split by prep_r_batch (three terms, padded column count,
// rows of roundup(M, 64)).
struct Act8Dot {
  slora_act8 X = {nullptr, nullptr};
  int64_t M = 0, K = 0;
  const void* P = nullptr;
  int cols = 0;
  float* out = nullptr;
  int64_t ldo = 0;
  const int32_t* kmap = nullptr;  // sanitized: every entry is a column of out
  float scale = 1.0f;
  int accumulate = 0;
};
// Partial sums (floats) and arrival counters (unsigned, zero on entry, left
// zero) that act8_dot needs.
int64_t act8_dot_part_floats(int64_t M, int64_t K, int cols);
int64_t act8_dot_counters(int64_t K, int cols);
slora_status act8_dot(const Act8Dot& d, float* part, unsigned* counters, cudaStream_t st);

}  // namespace slora
