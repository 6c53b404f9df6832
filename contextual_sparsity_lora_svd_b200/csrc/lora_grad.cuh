// The rank-r contractions of a LoRA linear's backward, with fp32 rank operands
// and activations in bf16 or as 8-bit checkpoints (see lora_grad.cu).
#pragma once

#include "act8.cuh"
#include "common.cuh"

namespace slora {

// An fp32 rank operand P [M x cols] as rank_sums reads it: three bf16 terms,
// transposed, [3][cols rounded up to 16][rank_terms_ld(M)]; columns past M are not read,
// rows past cols reach no output.
int64_t rank_terms_ld(int64_t M);
int64_t rank_terms_elems(int64_t M, int cols);

// What the contractions and products of one backward read, laid out in one launch:
// the rows of each kind and their M tiles (SLORA_SLICE_NONE: plain tiles over all
// rows, no maps), XA [T x cols] as terms (by full row, or by row kind in compact order),
// up to two copies of rows of B [. x cols], transposed to [cols rounded up to 16][rows
// rounded up to 64] (rank_rows' R), the kept rows of W, up to two transposes of A
// [cols x .] to rows of ldo, and the zeroed counters.  idx null: every row or column;
// an index outside `limit` stands for zeros and raises the flag of rank_check_error.
struct LoraCopy {
  const void* src = nullptr;
  const int32_t* idx = nullptr;
  int64_t n = 0, limit = 0;
  void* dst = nullptr;
};
struct LoraSetup {
  bool plain = false;
  int32_t *ctx_rows = nullptr, *out_rows = nullptr;
  int4 *ctiles = nullptr, *otiles = nullptr;  // plain: ctiles alone
  const float* XA = nullptr;
  void *terms = nullptr, *terms_out = nullptr;  // terms_out: by row kind, `terms` the context's
  LoraCopy B[2], W, A[2];
  int64_t wcols = 0, ldo = 0;  // columns of a row of W (a multiple of 8, 16-byte aligned rows)
  unsigned* zero = nullptr;
  int64_t nzero = 0;
  float* sums = nullptr;  // zeroed: what two jobs of rank_sums add to (16-byte aligned)
  int64_t nsums = 0;
};
slora_status lora_setup(const LoraSetup& d, const slora_tokens* tok, const TokenInfo& ti, int cols,
                        cudaStream_t st);

// Rows of a rank projection: p[m, q] = sum over c < K of Y(m, c) R(c, q), q <
// cols, for m < M.  Y bf16 with 16-byte aligned rows whose columns past K, up
// to a multiple of 8, are zero; R as lora_setup copies it.
// Written as terms (column m) and, scaled by s and in bf16, to out (row m).
// With map_*, map[m] stands for m: in the row of Y, the terms' column, out's row.
struct RankRows {
  const void* Y = nullptr;
  int64_t ld = 0, M = 0, K = 0;
  const void* R = nullptr;
  const int32_t* map = nullptr;
  bool map_y = false, map_terms = false, map_out = false;
  void* terms = nullptr;
  int64_t ldt = 0;
  void* out = nullptr;
  int64_t ldo = 0;
};
// Up to two of them in one launch.
slora_status rank_rows(const RankRows* jobs, int n, int cols, float s, cudaStream_t st);

// Sum over tokens: v[c, q] = scale * sum over m < M of X(m, c) P(m, q) for c < K,
// q < cols, P given as its terms, X bf16 (16-byte aligned rows of ld, a multiple
// of 8) or a checkpoint.  Written to out[q * ldo + c] (trans) or out[c * ldo + q];
// with `add`, added there, at channel idx[c] where idx is given (outside `limit`:
// left out).  Of distinct channels at most two jobs add to a zero, so their order
// does not show.
struct RankSum {
  const void* X = nullptr;
  slora_act8 X8 = {nullptr, nullptr};  // codes: the checkpoint, else X
  int64_t ld = 0, M = 0, K = 0;
  const void* terms = nullptr;
  float* out = nullptr;
  int64_t ldo = 0;
  int trans = 0;
  bool add = false;
  const int32_t* idx = nullptr;
  int64_t limit = 0;
};
constexpr int kRankSums = 3;  // of one launch
// Workspace of a launch: partial sums (floats) and arrival counters (unsigned,
// zero on entry, left zero).  M and K of the jobs alone decide.
int64_t rank_sums_part(const RankSum* jobs, int n, int cols);
int64_t rank_sums_counters(const RankSum* jobs, int n, int cols);
// beside: the launch may run beside the kernel before it on the stream and ends after
// it.  That kernel may not write what is read here, nor touch what is written, and what
// is read here was complete before that kernel called grid_ahead().
slora_status rank_sums(const RankSum* jobs, int n, int cols, float scale, float* part,
                       unsigned* counters, bool beside, cudaStream_t st);

// Budget of rank_sums' pipeline waits, in SM clocks; negative: the default.
slora_status rank_set_wait_budget(long long cycles);
// Raised when a rank_sums wait ran out of its budget, or by an index outside its weight.
slora_status rank_check_error(bool clear);

}  // namespace slora
