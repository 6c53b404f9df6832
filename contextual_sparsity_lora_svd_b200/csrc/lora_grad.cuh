// The rank-r contractions of a LoRA linear's backward, with fp32 rank operands
// and activations in bf16 or as 8-bit checkpoints (see lora_grad.cu).
#pragma once

#include "act8.cuh"
#include "common.cuh"

namespace slora {

// Rows of a rank projection: p[m, q] = sum over c < K of Y(m, c) R(c, q), q <
// cols, for m < M.  Y bf16 with 16-byte aligned rows whose columns past K, up
// to a multiple of 8, are zero; R split by prep_r_batch into one bf16 term.
// Written to out1 (fp32, row map1 ? map1[m] : m, ld1) and, scaled by s2, to
// out2 (bf16, row m, ld2).
struct RankRows {
  const void* Y = nullptr;
  int64_t ld = 0, M = 0, K = 0;
  const void* R = nullptr;
  float* out1 = nullptr;
  int64_t ld1 = 0;
  const int32_t* map1 = nullptr;
  void* out2 = nullptr;
  int64_t ld2 = 0;
};
// Up to two of them in one launch.
slora_status rank_rows(const RankRows* jobs, int n, int cols, float s2, cudaStream_t st);

// Sum over tokens: v[c, q] = scale * sum over m < M of X(m, c) P(map ? map[m] : m, q)
// for c < K, q < cols, P fp32 [.. x ldp], X bf16 (16-byte aligned rows of ld,
// a multiple of 8) or a checkpoint.  Written to out[q * ldo + c] (trans) or out[c * ldo + q].
struct RankSum {
  const void* X = nullptr;
  slora_act8 X8 = {nullptr, nullptr};  // codes: the checkpoint, else X
  int64_t ld = 0, M = 0, K = 0;
  const float* P = nullptr;
  int64_t ldp = 0;
  const int32_t* map = nullptr;
  float* out = nullptr;
  int64_t ldo = 0;
  int trans = 0;
};
constexpr int kRankSums = 3;  // of one launch
// Workspace of a launch: partial sums (floats) and arrival counters (unsigned,
// zero on entry, left zero).  M and K of the jobs alone decide.
int64_t rank_sums_part(const RankSum* jobs, int n, int cols);
int64_t rank_sums_counters(const RankSum* jobs, int n, int cols);
slora_status rank_sums(const RankSum* jobs, int n, int cols, float scale, float* part,
                       unsigned* counters, cudaStream_t st);

// Raised when a rank_sums wait ran out of its budget.
slora_status rank_check_error(bool clear);

}  // namespace slora
