// The rank-r contractions of a LoRA linear's backward (y = x W0^T + s (x A^T) B^T):
//   lora_setup  the operands' layouts, the row maps and the tile lists
//   rank_rows   p = dY B, row by row               (reads dY)
//   rank_sums   dA = s p^T X, dB = s dY^T (X A^T)  (sums over tokens; read X and dY)
// Each streams a large activation past a matrix with r columns, so both are
// bound by that stream; X may be an 8-bit checkpoint (1.03 bytes a value).
//
// lora_setup: what six launches did (indices checked, row maps, terms, rows of W, two
// transposes of A) in one whose blocks each take a piece of one of them: none waits for
// another, so the small ones run beside the copy of W's rows, and every block works out
// the compact place of a row from the sequences' offsets instead of reading a map.
//
// rank_rows: mma.sync m16n8k16 with fragments loaded straight from global
// memory.  The channel order inside a reduction is free, so lane t of a quad
// takes 8 consecutive channels (one 16-byte load a row, the same 8 channels of
// B's transposed copy), two k-steps of fragments.  A block owns 16 rows, its
// sixteen warps take every sixteenth 32-channel group and are summed in order
// in shared memory: no partial sums leave the block.  p is written as the
// GEMM's LoRA operand (s p rounded to bf16, as in the bf16 backward, whose dX this is
// to the bit; with an unrounded operand dX differs by 7e-4 to 1.8e-3 of its norm, where its
// own rounding to bf16 is 1.7e-3) and as the three bf16 terms that rank_sums reads.
// 12.7 us for 4096 x 4096 (5 for the 34 MB of dY from memory), bound by the latency
// of three rounds of loads a warp: blocks of 32 rows, which read B's copy half as
// often, take as long, clusters of four that split the channels of 64 rows 20 us.
//
// lora_setup takes 8 us for the q projection of 4096 rows at half its channels
// (27 us in six launches before), 14 us for a down projection of 11008 (53 us).
//
// rank_sums: tcgen05.mma with 128 channels as M, the tokens as the reduction and
// N = 48: 16 rank columns in three bf16 terms (an fp32 operand to 2^-24), so the
// sums are those of fp32 operands.  For 4096 x 4096 codes at r = 16 they take
// 15 us (legacy mma.sync 21, packed fp32 FMAs 30): 2 until the first stage is in,
// 6 for the stages, 1.5 to hand the partial sums over, 2 to join them.  X lies in shared memory as
// it does in global memory, a token's 128 channels in a row (an M-major operand,
// 128-byte swizzle): bf16 rows and the rank operand's terms come by TMA; codes
// come by TMA into a ring and eight warps expand them into the operand (a byte
// permute pairs two codes, two logic operations and an addition make them bf16,
// a product applies the step: all exact).  A stage is 64 tokens, four are in
// flight.  The stages take turns on four accumulators: the tensor core truncates
// each addition, and four short chains added in fp32 are off by a quarter of one
// long one.  Blocks that share channels leave partial sums that the last to
// arrive adds in order: the result does not depend on timing.  The launch runs
// beside the last tiles of the product before it (its blocks fit on SMs that have
// none left) and its blocks leave after that: 116 -> 114 us for the q projection's
// backward of 4096 rows, 20 -> 16 for 256 rows of 256 -> 688.  It lets nothing start
// early itself: blocks of a small grid would crowd on the SMs that end first.  Every wait is
// bounded; on expiry the block raises a device flag (slora_device_error:
// SLORA_ERR_TIMEOUT) and leaves after its own copies and products ended.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include <algorithm>

#include "act8_dev.cuh"
#include "lora_grad.cuh"

namespace slora {

constexpr long long kWaitBudget = 2000000000LL;  // ~1 s of SM clocks per wait
__device__ int g_rank_error = 0;
__device__ int g_rank_bad_index = 0;
// Budget of rank_sums' pipeline waits (settable for tests of the error path); what a block
// waits for before it may leave has the full one.
__device__ long long g_rank_budget = kWaitBudget;

namespace {

constexpr int kCols = 16;   // rank columns of a block (more: further blocks)
constexpr int kTerms = 3;   // bf16 terms of an fp32 rank operand

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------------ setup
constexpr int kSetupThreads = 256;
constexpr int kSetupRows = 64;  // rows of XA or B of a block
constexpr int kSmallBatch = 64;  // sequences in the small parameter block

template <int CAP>
struct SetupParams {
  LoraSetup d;
  int seq, batch, cols, cp;
  long long ldt, ldto;  // columns of the terms' rows
  long long T;
  // first block of: the rows of W, the tokens, B's copies, A's transposes, the zeros
  int w0, t0, b0, b1, a0, a1, z0;
  int off[CAP + 1];  // context rows before each sequence
};

__device__ __forceinline__ long long setup_index(const LoraCopy& c, long long i) {
  const long long v = c.idx ? (long long)c.idx[i] : i;
  if (v >= 0 && v < c.limit) return v;
  atomicExch(&g_rank_bad_index, 1);
  return -1;
}
// v as the sum of its terms.  The first holds what rounds past bf16's largest number as
// that number, and an infinity alone (its difference to itself is no zero).
__device__ __forceinline__ void put_terms(__nv_bfloat16* o, long long plane, float v) {
  __nv_bfloat16 h = __float2bfloat16_rn(v);
  if (__hisinf(h)) {
    if (isinf(v)) {
      o[0] = h;
#pragma unroll
      for (int k = 1; k < kTerms; ++k) o[k * plane] = __float2bfloat16_rn(0.0f);
      return;
    }
    h = __float2bfloat16_rz(v);
  }
  o[0] = h;
#pragma unroll
  for (int k = 1; k < kTerms; ++k) {
    v -= __bfloat162float(h);
    h = __float2bfloat16_rn(v);
    o[k * plane] = h;
  }
}

template <int CAP>
__global__ void __launch_bounds__(kSetupThreads)
    lora_setup_kernel(const __grid_constant__ SetupParams<CAP> P) {
  grid_wait();
  grid_ahead();
  const LoraSetup& d = P.d;
  const int tid = threadIdx.x, blk = blockIdx.x, seq = P.seq;
  if (blk < P.w0) {  // tile lists and counters
    for (int64_t i = tid; i < d.nzero; i += kSetupThreads) d.zero[i] = 0u;
    if (d.plain) {
      for (long long r = 128ll * tid; r < P.T; r += 128ll * kSetupThreads)
        d.ctiles[r / 128] = make_int4(int(r), int(r), int(min(128ll, P.T - r)), 0);
      return;
    }
    __shared__ int ct[CAP], ot[CAP];
    if (tid == 0) {
      int c = 0, o = 0;
      for (int b = 0; b < P.batch; ++b) {
        const int len = P.off[b + 1] - P.off[b];
        ct[b] = c;
        ot[b] = o;
        c += (len + 127) / 128;
        o += (seq - len + 127) / 128;
      }
    }
    __syncthreads();
    for (int b = tid; b < P.batch; b += kSetupThreads) {
      const int c0 = P.off[b], len = P.off[b + 1] - c0, row = b * seq;
      for (int j = 0; j * 128 < len; ++j)
        d.ctiles[ct[b] + j] = make_int4(row + 128 * j, c0 + 128 * j, min(128, len - 128 * j), 0);
      for (int j = 0; j * 128 < seq - len; ++j)
        d.otiles[ot[b] + j] = make_int4(row + len + 128 * j, row - c0 + 128 * j,
                                        min(128, seq - len - 128 * j), 0);
    }
  } else if (blk < P.t0) {  // a warp a row of W, eight 16-byte loads a lane in flight
    const long long j = (long long)(blk - P.w0) * (kSetupThreads / 32) + (tid >> 5);
    if (j >= d.W.n) return;
    const long long src = setup_index(d.W, j);
    const int lane = tid & 31, n16 = int(d.wcols / 8);
    const uint4* in = static_cast<const uint4*>(d.W.src) + max(src, 0ll) * n16;
    uint4* out = static_cast<uint4*>(d.W.dst) + j * n16;
    for (int c0 = lane; c0 < n16; c0 += 32 * 8) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = src >= 0 && c0 + 32 * u < n16 ? __ldg(in + c0 + 32 * u) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (c0 + 32 * u < n16) out[c0 + 32 * u] = v[u];
    }
  } else if (blk < P.b0) {  // tokens: maps and XA's terms; the row runs fastest in what is written
    const long long t = (long long)(blk - P.t0) * kSetupRows + tid % kSetupRows;
    if (t >= P.T) return;
    long long at = t;
    __nv_bfloat16* terms = static_cast<__nv_bfloat16*>(d.terms);
    long long ldt = P.ldt;
    if (!d.plain) {
      const int b = int(t / seq), i = int(t % seq), c0 = P.off[b], len = P.off[b + 1] - c0;
      const bool ctx = i < len;
      const int place = ctx ? c0 + i : b * seq - c0 + (i - len);
      if (tid < kSetupRows) (ctx ? d.ctx_rows : d.out_rows)[place] = int(t);
      if (d.terms_out) {
        at = place;
        if (!ctx) {
          terms = static_cast<__nv_bfloat16*>(d.terms_out);
          ldt = P.ldto;
        }
      }
    }
    for (int q = tid / kSetupRows; q < P.cols; q += kSetupThreads / kSetupRows)
      put_terms(terms + q * ldt + at, P.cp * ldt, __ldg(d.XA + t * P.cols + q));
  } else if (blk < P.a0) {  // rows of B, transposed; zeros to whole rows of 64
    const bool second = blk >= P.b1;
    const LoraCopy& c = d.B[second ? 1 : 0];
    const long long i = (long long)(blk - (second ? P.b1 : P.b0)) * kSetupRows + tid % kSetupRows;
    const long long ld = (max((long long)c.n, 1ll) + kSetupRows - 1) / kSetupRows * kSetupRows;
    const long long src = i < c.n ? setup_index(c, i) : -1;
    const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(c.src) + max(src, 0ll) * P.cols;
    for (int q = tid / kSetupRows; q < P.cp; q += kSetupThreads / kSetupRows)
      static_cast<__nv_bfloat16*>(c.dst)[q * ld + i] =
          src >= 0 && q < P.cols ? in[q] : __float2bfloat16_rn(0.0f);
  } else if (blk >= P.z0) {  // four values a thread
    const int64_t i = ((int64_t)(blk - P.z0) * kSetupThreads + tid) * 4;
    if (i + 3 < d.nsums) *reinterpret_cast<float4*>(d.sums + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    else
      for (int64_t e = i; e < d.nsums; ++e) d.sums[e] = 0.0f;
  } else {  // A's transposes: a thread eight columns of a row
    const bool second = blk >= P.a1;
    const LoraCopy& c = d.A[second ? 1 : 0];
    const long long e = (long long)(blk - (second ? P.a1 : P.a0)) * kSetupThreads + tid;
    const long long i = e % c.n, q0 = e / c.n * 8;  // rows run fastest: A is read along its rows
    if (q0 >= d.ldo) return;
    const long long src = setup_index(c, i);
    alignas(16) __nv_bfloat16 v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      v[q] = src >= 0 && q0 + q < P.cols
                 ? static_cast<const __nv_bfloat16*>(c.src)[(q0 + q) * c.limit + src]
                 : __float2bfloat16_rn(0.0f);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(c.dst) + i * d.ldo + q0) =
        *reinterpret_cast<const uint4*>(v);
  }
}

// ------------------------------------------------------------------- rows
constexpr int kRowWarps = 16;

struct RowsJob {
  const __nv_bfloat16* Y;
  const __nv_bfloat16* R;  // [cols rounded up to 16][K64]
  long long ld, M, K, K64;
  const int32_t* map;
  int map_y, map_terms, map_out;
  __nv_bfloat16* terms;  // [kTerms][cp][ldt]
  long long ldt;
  __nv_bfloat16* out;
  long long ldo;
};
struct RowsParams {
  RowsJob job[2];
  int blocks0;  // 16-row blocks of job 0
  int cols, cp;
  float s;
};

__global__ void __launch_bounds__(kRowWarps * 32, 2)
    rank_rows_kernel(const __grid_constant__ RowsParams P) {
  __shared__ float red[kRowWarps][16][kCols + 1];
  grid_wait();
  grid_ahead();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const bool second = int(blockIdx.x) >= P.blocks0;
  const RowsJob& j = P.job[second ? 1 : 0];
  const long long m0 = (long long)(int(blockIdx.x) - (second ? P.blocks0 : 0)) * 16;
  const int q0 = blockIdx.y * kCols;
  const bool on0 = m0 + g < j.M, on1 = m0 + g + 8 < j.M;
  auto row = [&](long long m, bool on, int mapped) -> long long {
    return !on ? 0 : (mapped ? (long long)j.map[m] : m);
  };
  const __nv_bfloat16* y0 = j.Y + row(m0 + g, on0, j.map_y) * j.ld;
  const __nv_bfloat16* y1 = j.Y + row(m0 + g + 8, on1, j.map_y) * j.ld;
  const __nv_bfloat16* r0 = j.R + (q0 + g) * j.K64;
  const __nv_bfloat16* r1 = r0 + 8 * j.K64;
  float acc[2][4] = {};
  const uint4 none = make_uint4(0, 0, 0, 0);
  constexpr int kDeep = 3;  // groups of 32 channels in flight
  // every 8-channel load lies inside the row's whole 16-byte units or is left out
  for (long long c0 = warp * 32; c0 < j.K; c0 += kRowWarps * 32 * kDeep) {
    uint4 a[kDeep], b[kDeep], r[kDeep], s[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      const long long c = c0 + i * kRowWarps * 32 + 8 * t;
      const bool on = c < j.K;
      a[i] = on && on0 ? *reinterpret_cast<const uint4*>(y0 + c) : none;
      b[i] = on && on1 ? *reinterpret_cast<const uint4*>(y1 + c) : none;
      r[i] = on ? __ldg(reinterpret_cast<const uint4*>(r0 + c)) : none;
      s[i] = on ? __ldg(reinterpret_cast<const uint4*>(r1 + c)) : none;
    }
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      mma_bf16(acc[0], a[i].x, b[i].x, a[i].y, b[i].y, r[i].x, r[i].y);
      mma_bf16(acc[1], a[i].x, b[i].x, a[i].y, b[i].y, s[i].x, s[i].y);
      mma_bf16(acc[0], a[i].z, b[i].z, a[i].w, b[i].w, r[i].z, r[i].w);
      mma_bf16(acc[1], a[i].z, b[i].z, a[i].w, b[i].w, s[i].z, s[i].w);
    }
  }
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[warp][g + 8 * (e >> 1)][n * 8 + 2 * t + (e & 1)] = acc[n][e];
  __syncthreads();
  if (threadIdx.x >= 256) return;
  // a thread a value: the row runs fastest, as in the terms' rows
  const int mr = threadIdx.x % 16, q = threadIdx.x / 16;
  const long long m = m0 + mr;
  if (m >= j.M || q0 + q >= P.cols) return;
  float v = 0.0f;
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) v += red[w][mr][q];
  j.out[row(m, true, j.map_out) * j.ldo + q0 + q] = __float2bfloat16_rn(P.s * v);
  put_terms(j.terms + (q0 + q) * j.ldt + row(m, true, j.map_terms), P.cp * j.ldt, v);
}

// ------------------------------------------------------------------- sums
constexpr int kCh = 128;            // channels of a block (M)
constexpr int kTok = 64;            // tokens of a stage
constexpr int kAcc = 4;             // accumulators the stages take turns on
constexpr int kTile = kCh * kCols;  // outputs of a block
constexpr int kRing = 4;            // stages in flight
constexpr int kSlots8 = 2;          // operand slots that codes are expanded into
constexpr int kXWarps = 8;          // warps that expand codes
constexpr int kSumThreads = kXWarps * 32 + 64;  // and the products' warp, the copies' warp
constexpr int kABytes = kTok * kCh * 2;             // 16 KB: two 64-channel halves
constexpr int kBBytes = kTerms * kCols * kTok * 2;  // 6 KB
constexpr int kXBytes = kTok * kCh;                 // 8 KB of codes
// bf16: a ring of (X, P) operands; codes: a ring of (codes, P) and the slots.
constexpr int kSumSmem = 1024 + kRing * (kABytes + kBBytes);  // 89 KB
static_assert(kRing * (kXBytes + kBBytes) + kSlots8 * kABytes <= kRing * (kABytes + kBBytes),
              "codes' layout inside the bf16 layout's memory");
constexpr int kTmemCols = 256;  // kAcc * 64, of which 48 each are used

struct alignas(64) SumJob {
  CUtensorMap xmap;       // codes: 128 x 64 boxes; bf16: 64 x 64, 128-byte swizzle
  CUtensorMap pmap;       // the terms of P^T, 64 tokens x 16 columns, 128-byte swizzle
  const uint8_t* scales;  // null: bf16
  long long ld8;          // scale bytes of a row
  long long M, K;
  float* out;
  long long ldo;
  const int32_t* idx;
  long long limit;
  int add;
  int trans, nsplit, blocks;  // blocks: channel blocks * splits
  int stages;                 // of one split
  int tile0;                  // first output tile (partials and counters)
};
struct SumParams {
  SumJob job[kRankSums];
  int n, cols, cp, tiles;  // tiles: output tiles of one column slice
  int beside;
  float scale;
  float* part;
  unsigned* counters;
};

__device__ __forceinline__ uint32_t su32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(su32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
// One poll (try_wait may park the thread until the phase completes).
__device__ __forceinline__ bool mbar_test(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(su32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void wait_expired(volatile int* abort) {
  *abort = 1;
  atomicExch(&g_rank_error, 1);
}
// Bounded wait for the phase of parity `parity`; false on abort or expiry (a budget of 0:
// unless the first poll succeeds).
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity, volatile int* abort,
                                          long long budget) {
  if (mbar_test(b, parity)) return true;
  const long long t0 = clock64();
  while (budget > 0) {
    if (mbar_try(b, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > budget) break;
  }
  wait_expired(abort);
  return false;
}
// What a block has in flight, before it leaves.
__device__ __forceinline__ void mbar_drain(uint64_t* b, uint32_t parity, volatile int* abort) {
  const long long t0 = clock64();
  while (!mbar_try(b, parity))
    if (clock64() - t0 > kWaitBudget) {
      wait_expired(abort);
      return;
    }
}
// Shared-memory matrix descriptor, 128-byte swizzle.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | uint64_t((lbo >> 4) & 0x3FFFu) << 16 |
         uint64_t((sbo >> 4) & 0x3FFFu) << 32 | uint64_t(1) << 46 | uint64_t(2) << 61;
}
// kind::f16, bf16 operands, fp32 accumulator, A M-major, B K-major, 128 x 48.
constexpr uint32_t kSumDesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) |
                              (uint32_t(kTerms * kCols) >> 3 << 17) | (uint32_t(kCh) >> 4 << 24);
__device__ __forceinline__ void mma_1sm(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(kSumDesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   su32(bar))
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void mbar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* m, uint64_t* bar, int x,
                                         int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(su32(bar)), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
// Byte offset of 16-byte unit u (0 .. 15: 8 channels each) of token t in an X
// slot: two halves of 64 channels, 128-byte rows, unit index XOR row mod 8.
__device__ __forceinline__ uint32_t x_at(int t, int u) {
  return uint32_t((u >> 3) * (kTok * 128) + t * 128 + (((u & 7) ^ (t & 7)) << 4));
}
// Two codes (bytes J, J + 1 of w) times their step as packed bf16: 128 + the low
// seven bits, less 128 or, for a negative code, 256.
template <int J>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, __nv_bfloat162 step) {
  const uint32_t u = __byte_perm(w, 0u, 0x4040 | J | ((J + 1) << 8));
  const uint32_t a = (u & 0x007f007fu) | 0x43004300u;
  const uint32_t c = (u & 0x00800080u) | 0xc300c300u;
  const __nv_bfloat162 v = __hadd2(act8_as_bf162(a), act8_as_bf162(c));
  const __nv_bfloat162 r = __hmul2(v, step);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 16 codes of a token, two 16-byte units of the operand slot (they differ in the
// lowest bit of the swizzled unit index).
__device__ __forceinline__ void expand16(uint32_t dst, const uint4& w, uint32_t byte) {
  const __nv_bfloat162 step =
      act8_as_bf162(byte == 255u ? 0x7fff7fffu : (byte - 6u) * 0x800080u);
  sts128(dst, make_uint4(code_pair<0>(w.x, step), code_pair<2>(w.x, step),
                         code_pair<0>(w.y, step), code_pair<2>(w.y, step)));
  sts128(dst ^ 16u, make_uint4(code_pair<0>(w.z, step), code_pair<2>(w.z, step),
                               code_pair<0>(w.w, step), code_pair<2>(w.w, step)));
}

__global__ void __launch_bounds__(kSumThreads, 2) rank_sums_kernel(const __grid_constant__ SumParams P) {
  extern __shared__ uint8_t s_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  // copied: a ring place's copies have landed; ready: its X operand is complete
  // (codes); empty: its products are done
  __shared__ uint64_t copied[kRing], ready[kRing], empty[kRing], done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ unsigned s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int blk = blockIdx.x, w = 0;
  while (w + 1 < P.n && blk >= P.job[w].blocks) blk -= P.job[w++].blocks;
  const SumJob& j = P.job[w];
  const int nch = j.blocks / j.nsplit;
  const int cb = blk % nch, split = blk / nch, q0 = blockIdx.y * kCols;
  const long long ch0 = (long long)cb * kCh;
  const long long m0 = (long long)split * j.stages * kTok;
  const int stages = int(max(0ll, min((long long)j.stages, (j.M - m0 + kTok - 1) / kTok)));
  const bool codes = j.scales != nullptr;
  const uint32_t sB = su32(smem), sX = sB + kRing * kBBytes;  // sX: operands, or codes
  const uint32_t sA = sX + kRing * kXBytes;                   // codes' operand slots
  auto copy = [&](int st) {
    const int place = st % kRing, m = int(m0) + st * kTok;
    mbar_expect(&copied[place], kBBytes + (codes ? kXBytes : kABytes));
#pragma unroll
    for (int s = 0; s < kTerms; ++s)
      tma_load(sB + place * kBBytes + s * kCols * 128, &j.pmap, &copied[place], m,
               s * P.cp + q0);
    if (codes) {
      tma_load(sX + place * kXBytes, &j.xmap, &copied[place], int(ch0), m);
    } else {
      tma_load(sX + place * kABytes, &j.xmap, &copied[place], int(ch0), m);
      tma_load(sX + place * kABytes + kTok * 128, &j.xmap, &copied[place], int(ch0) + 64, m);
    }
  };
  if (tid == kSumThreads - 32) {  // the copies' thread fills the ring while memory is allocated
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&copied[i], 1);
      mbar_init(&ready[i], kXWarps / kSlots8);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (!P.beside) grid_wait();
    for (int st = 0; st < min(stages, kRing); ++st) copy(st);
  }
  if (warp == kXWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     su32(&s_tmem)),
                 "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (!P.beside) grid_wait();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tbase = s_tmem;
  volatile int* abort = &s_abort;
  const long long budget = g_rank_budget;
  // the products of stage st (which used its ring place and operand slot) are done
  auto products_done = [&](int st) {
    return st < 0 || mbar_wait(&empty[st % kRing], uint32_t(st / kRing) & 1u, abort, budget);
  };

  if (warp == kXWarps + 1) {
    // ------------------------------------------------------------ copies
    if (lane == 0) {
      int issued = min(stages, kRing);
      for (; issued < stages && products_done(issued - kRing); ++issued) copy(issued);
      // the copies land before the block may leave (normally long since read)
      for (int st = max(0, issued - kRing); st < issued; ++st)
        mbar_drain(&copied[st % kRing], uint32_t(st / kRing) & 1u, abort);
    }
  } else if (warp == kXWarps) {
    // ---------------------------------------------------------- products
    if (lane == 0 && stages > 0) {
      for (int st = 0; st < stages; ++st) {
        const int place = st % kRing;
        const uint32_t phase = uint32_t(st / kRing) & 1u;
        if (!mbar_wait(&copied[place], phase, abort, budget)) break;
        if (codes && !mbar_wait(&ready[place], phase, abort, budget)) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t a = codes ? sA + (st % kSlots8) * kABytes : sX + place * kABytes;
        const uint32_t b = sB + place * kBBytes;
        const uint32_t d = tbase + uint32_t(st % kAcc) * 64u;
#pragma unroll
        for (int k = 0; k < kTok / 16; ++k)
          mma_1sm(d, sdesc(a + k * 2048, kTok * 128, 1024), sdesc(b + k * 32, 16, 1024),
                  st >= kAcc || k > 0 ? 1u : 0u);
        mma_commit(&empty[place]);
      }
      mma_commit(&done);
      // nothing of this block may be in flight when it leaves, aborted or not
      mbar_drain(&done, 0, abort);
    }
  } else if (codes) {
    // --------------------------------------------------------- expansion
    // The stages take turns on groups of four warps, a slot each: a group's barriers
    // and its proxy fence come once in two stages.  This thread: 16 channels (unit
    // tid % 8) of every sixteenth token.
    const int group = warp / (kXWarps / kSlots8), gt = tid % (kXWarps / kSlots8 * 32);
    const int xt = gt >> 3, xu = gt & 7;
    const long long ch = ch0 + 16 * xu;
    const bool inside = ch < j.ld8 * kActBlock;  // rows are whole blocks
    const uint8_t* sc = j.scales + (inside ? (m0 + xt) * j.ld8 + (ch >> 5) : 0);
    const int rows = int(min((long long)stages * kTok, j.M - m0));
    constexpr int kEach = kTok / 16;
    uint32_t b[kEach], next[kEach];
    auto bytes_of = [&](int st, uint32_t (&v)[kEach]) {  // of the split's tokens xt + ...
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int at = st * kTok + 16 * i;
        v[i] = inside && at + xt < rows ? sc[at * j.ld8] : 7u;
      }
    };
    const uint32_t dst = sA + group * kABytes + x_at(xt, 2 * xu);  // 16 tokens on: 2 KB on
    bytes_of(group, b);
    for (int st = group; st < stages; st += kSlots8) {
      const int place = st % kRing;
      bytes_of(st + kSlots8, next);
      if (!mbar_wait(&copied[place], uint32_t(st / kRing) & 1u, abort, budget)) break;
      uint4 w[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) w[i] = lds128(sX + place * kXBytes + gt * 16 + i * 2048);
      if (!products_done(st - kSlots8)) break;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        expand16(dst + i * 2048, w[i], b[i]);
        b[i] = next[i];
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&ready[place]);
    }
  }
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");

  const int tile = int(blockIdx.y) * P.tiles + j.tile0 + cb;
  const long long ch = ch0 + 32 * warp + lane;  // TMEM lane = channel (warps 0 .. 3)
  float4* mine = reinterpret_cast<float4*>(
      P.part + ((long long)blockIdx.y * gridDim.x + blockIdx.x) * kTile) + 32 * (warp & 3) + lane;
  auto emit = [&](const auto& v, long long c, int first) {
    if (c >= j.K) return;
    if (j.idx) c = j.idx[c];
    if (j.idx && (c < 0 || c >= j.limit)) return;
    float* out = j.out + (j.trans ? c : c * j.ldo);
    const long long step = j.trans ? j.ldo : 1;
#pragma unroll
    for (int i = 0; i < int(sizeof(v) / sizeof(float)); ++i) {
      const int q = q0 + first + i;
      if (q >= P.cols) continue;
      if (j.add) atomicAdd(out + q * step, v[i] * P.scale);
      else out[q * step] = v[i] * P.scale;
    }
  };
  if (warp < 4) {
    float v[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) v[q] = 0.0f;
    for (int a = 0; a < min(stages, kAcc); ++a)
#pragma unroll
      for (int s = kTerms - 1; s >= 0; --s) {  // the small terms first
        float t[16];
        tmem_ld16(tbase + (uint32_t(32 * warp) << 16) + uint32_t(a * 64 + s * kCols), t);
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] += t[q];
      }
    if (j.nsplit == 1) {
      emit(v, ch, 0);
    } else {  // [4 columns of 4][128 channels] of float4
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mine[q * kCh] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == kXWarps) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase),
                 "n"(kTmemCols)
                 : "memory");
  }
  if (j.nsplit == 1) {
    grid_wait();
    return;
  }
  if (tid == 0) {
    __threadfence();
    const unsigned prev = atomicAdd(&P.counters[tile], 1u);
    s_last = prev + 1 == unsigned(j.nsplit);
    if (s_last) P.counters[tile] = 0u;
  }
  __syncthreads();
  if (!s_last || warp >= kXWarps) {
    grid_wait();
    return;
  }
  __threadfence();
  // split s of this channel block ran as block (blockIdx.x - blk) + s * nch + cb
  // (eight warps: a thread half the columns of a channel, eight splits' loads at once)
  const int c = tid % kCh, half = tid / kCh * 2;
  const float4* src = reinterpret_cast<const float4*>(
      P.part + ((long long)blockIdx.y * gridDim.x + blockIdx.x - blk + cb) * kTile) + half * kCh + c;
  const long long step = (long long)nch * kTile / 4;
  float v[8] = {};
  for (int s0 = 0; s0 < j.nsplit; s0 += 8) {
    float4 f[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        f[i][q] = s0 + i < j.nsplit ? __ldcg(src + (s0 + i) * step + q * kCh)
                                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        v[4 * q] += f[i][q].x;
        v[4 * q + 1] += f[i][q].y;
        v[4 * q + 2] += f[i][q].z;
        v[4 * q + 3] += f[i][q].w;
      }
  }
  emit(v, ch0 + c, 4 * half);
  grid_wait();
}

int slices(int cols) { return (cols + kCols - 1) / kCols; }
int64_t channel_blocks(const RankSum& j) { return (j.K + kCh - 1) / kCh; }
// Splits of each job over the tokens: the fewest stages a block for which the
// launch is one wave of two blocks an SM (a second wave would double it), at
// most 32 splits (the last block of a tile adds them).
void plan_splits(const RankSum* jobs, int n, int cols, int* nsplit, int* per) {
  int64_t stages[kRankSums], nch[kRankSums], most = 1;
  for (int i = 0; i < n; ++i) {
    stages[i] = std::max<int64_t>((jobs[i].M + kTok - 1) / kTok, 1);
    nch[i] = channel_blocks(jobs[i]) * slices(cols);
    most = std::max(most, stages[i]);
  }
  auto splits = [&](int i, int64_t each) { return (stages[i] + each - 1) / each; };
  auto fits = [&](int64_t each) {
    int64_t blocks = 0;
    for (int i = 0; i < n; ++i) {
      if (splits(i, each) > 32) return false;
      blocks += nch[i] * splits(i, each);
    }
    return blocks <= 2 * num_sms();
  };
  int64_t lo = 1, hi = most;  // `most` is one split each: taken even where it does not fit
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (fits(mid)) hi = mid;
    else lo = mid + 1;
  }
  for (int i = 0; i < n; ++i) {
    const int64_t k = std::min<int64_t>(splits(i, lo), 32);
    per[i] = int((stages[i] + k - 1) / k);
    nsplit[i] = int((stages[i] + per[i] - 1) / per[i]);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

// 2-D tensor map with zero fill outside [rows x cols].
slora_status encode(CUtensorMap* m, CUtensorMapDataType type, int es, const void* ptr,
                    int64_t rows, int64_t cols, int64_t ld, int box_x, int box_y,
                    CUtensorMapSwizzle swz) {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) SLORA_FAIL(SLORA_ERR_CUDA, "cuTensorMapEncodeTiled entry point not available");
  cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
  cuuint64_t strides[1] = {cuuint64_t(ld) * es};
  cuuint32_t box[2] = {cuuint32_t(box_x), cuuint32_t(box_y)}, one[2] = {1, 1};
  const CUresult r = g_encode(m, type, 2, const_cast<void*>(ptr), dims, strides, box, one,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    SLORA_FAIL(SLORA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) rows=%lld cols=%lld ld=%lld",
               int(r), (long long)rows, (long long)cols, (long long)ld);
  return SLORA_OK;
}

int64_t padded_cols(int cols) { return int64_t(slices(cols)) * kCols; }

}  // namespace

int64_t rank_terms_ld(int64_t M) { return (std::max<int64_t>(M, 1) + 63) / 64 * 64; }
int64_t rank_terms_elems(int64_t M, int cols) {
  return kTerms * padded_cols(cols) * rank_terms_ld(M);
}

namespace {
template <int CAP>
slora_status setup(const LoraSetup& d, const slora_tokens* tok, const TokenInfo& ti, int cols,
                   cudaStream_t st) {
  SetupParams<CAP> p{};
  p.d = d;
  p.seq = ti.seq; p.batch = ti.batch; p.cols = cols;
  p.cp = int(padded_cols(cols));
  p.T = ti.T;
  p.ldt = rank_terms_ld(d.terms_out ? ti.T_C : ti.T);
  p.ldto = rank_terms_ld(ti.T_O);
  for (int b = 0; b < ti.batch; ++b) p.off[b + 1] = p.off[b] + tok->ctx_len[b];
  int64_t at = 1;
  auto add = [&](int64_t items, int64_t each) {
    const int64_t first = at;
    at += (items + each - 1) / each;
    return int(first);
  };
  p.w0 = add(d.W.n, kSetupThreads / 32);
  p.t0 = add(ti.T, kSetupRows);
  p.b0 = add(d.B[0].dst ? std::max<int64_t>(d.B[0].n, 1) : 0, kSetupRows);
  p.b1 = add(d.B[1].dst ? std::max<int64_t>(d.B[1].n, 1) : 0, kSetupRows);
  p.a0 = add(d.A[0].n * (d.ldo / 8), kSetupThreads);
  p.a1 = add(d.A[1].n * (d.ldo / 8), kSetupThreads);
  p.z0 = add(d.nsums, kSetupThreads * 4);
  double bytes = double(ti.T) * cols * (4 + 2 * kTerms) + 4.0 * double(d.W.n) * d.wcols;
  for (int i = 0; i < 2; ++i) bytes += 4.0 * double(d.B[i].n + d.A[i].n) * cols;
  LaunchScope ls(kAux, bytes, st);
  SLORA_CUDA(launch_early(lora_setup_kernel<CAP>, dim3(unsigned(at)), kSetupThreads, 0, st, p));
  return SLORA_OK;
}
}  // namespace

slora_status lora_setup(const LoraSetup& d, const slora_tokens* tok, const TokenInfo& ti, int cols,
                        cudaStream_t st) {
  return ti.batch <= kSmallBatch ? setup<kSmallBatch>(d, tok, ti, cols, st)
                                 : setup<kMaxBatch>(d, tok, ti, cols, st);
}

slora_status rank_rows(const RankRows* jobs, int n, int cols, float s, cudaStream_t st) {
  if (n < 1 || n > 2) SLORA_FAIL(SLORA_ERR_SHAPE, "rank_rows: %d jobs", n);
  RowsParams p{};
  int64_t blocks[2] = {0, 0};
  double bytes = 0.0;
  for (int i = 0; i < n; ++i) {
    const RankRows& r = jobs[i];
    RowsJob& j = p.job[i];
    j.Y = static_cast<const __nv_bfloat16*>(r.Y);
    j.R = static_cast<const __nv_bfloat16*>(r.R);
    j.ld = r.ld; j.M = r.M; j.K = r.K;
    j.K64 = (std::max<int64_t>(r.K, 1) + 63) / 64 * 64;
    j.map = r.map; j.map_y = r.map_y; j.map_terms = r.map_terms; j.map_out = r.map_out;
    j.terms = static_cast<__nv_bfloat16*>(r.terms); j.ldt = r.ldt;
    j.out = static_cast<__nv_bfloat16*>(r.out); j.ldo = r.ldo;
    blocks[i] = (r.M + 15) / 16;
    bytes += double(r.M) * r.K * 2;
    if (r.M > 0 && r.K > 0 && (!aligned16(r.Y) || r.ld % 8))
      SLORA_FAIL(SLORA_ERR_ALIGN, "rank_rows: rows are not whole 16-byte units");
  }
  if (blocks[0] + blocks[1] == 0) return SLORA_OK;
  p.blocks0 = int(blocks[0]);
  p.cols = cols;
  p.cp = int(padded_cols(cols));
  p.s = s;
  LaunchScope ls(kSkinny, bytes, st);
  SLORA_CUDA(launch_early(rank_rows_kernel,
                          dim3(unsigned(blocks[0] + blocks[1]), unsigned(slices(cols))),
                          kRowWarps * 32, 0, st, p));
  return SLORA_OK;
}

int64_t rank_sums_part(const RankSum* jobs, int n, int cols) {
  int nsplit[kRankSums];
  int per[kRankSums];
  int64_t blocks = 0;
  plan_splits(jobs, n, cols, nsplit, per);
  for (int i = 0; i < n; ++i) blocks += channel_blocks(jobs[i]) * nsplit[i];
  return std::max<int64_t>(blocks * slices(cols) * kTile, 1);
}
int64_t rank_sums_counters(const RankSum* jobs, int n, int cols) {
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) tiles += channel_blocks(jobs[i]);
  return std::max<int64_t>(tiles * slices(cols), 1);
}

slora_status rank_sums(const RankSum* jobs, int n, int cols, float scale, float* part,
                       unsigned* counters, bool beside, cudaStream_t st) {
  if (n < 1 || n > kRankSums) SLORA_FAIL(SLORA_ERR_SHAPE, "rank_sums: %d jobs", n);
  int nsplit[kRankSums];
  int per[kRankSums];
  int64_t blocks = 0, tiles = 0;
  plan_splits(jobs, n, cols, nsplit, per);
  SumParams p{};
  double bytes = 0.0;
  for (int i = 0; i < n; ++i) {
    const RankSum& s = jobs[i];
    SumJob& j = p.job[i];
    const bool codes = s.X8.codes != nullptr;
    j.M = s.M; j.K = s.K;
    j.out = s.out; j.ldo = s.ldo; j.trans = s.trans;
    j.add = s.add; j.idx = s.idx; j.limit = s.limit;
    j.nsplit = nsplit[i];
    j.stages = per[i];
    j.blocks = int(channel_blocks(s)) * nsplit[i];
    j.tile0 = int(tiles);
    tiles += channel_blocks(s);
    blocks += j.blocks;
    bytes += double(s.M) * s.K * (codes ? 1.03125 : 2.0);
    if (s.M <= 0 || s.K <= 0) continue;  // no stage: its outputs are zeros
    if (codes) {
      j.scales = s.X8.scales;
      j.ld8 = act8_cols(s.K) / kActBlock;
      SLORA_TRY(encode(&j.xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, s.X8.codes, s.M, act8_cols(s.K),
                       act8_cols(s.K), kCh, kTok, CU_TENSOR_MAP_SWIZZLE_NONE));
    } else {
      if (!aligned16(s.X) || s.ld % 8)
        SLORA_FAIL(SLORA_ERR_ALIGN, "rank_sums: rows are not whole 16-byte units");
      SLORA_TRY(encode(&j.xmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, s.X, s.M, s.K, s.ld, 64, kTok,
                       CU_TENSOR_MAP_SWIZZLE_128B));
    }
    SLORA_TRY(encode(&j.pmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, s.terms,
                     kTerms * padded_cols(cols), s.M, rank_terms_ld(s.M), kTok, kCols,
                     CU_TENSOR_MAP_SWIZZLE_128B));
  }
  if (blocks == 0) return SLORA_OK;
  p.n = n;
  p.cols = cols;
  p.cp = int(padded_cols(cols));
  p.tiles = int(tiles);
  p.scale = scale;
  p.part = part;
  p.counters = counters;
  p.beside = beside;
  SLORA_CUDA(cudaFuncSetAttribute(rank_sums_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  kSumSmem));
  LaunchScope ls(kSkinny, bytes * slices(cols), st);
  SLORA_CUDA(launch_early(rank_sums_kernel, dim3(unsigned(blocks), unsigned(slices(cols))),
                          kSumThreads, kSumSmem, st, p));
  return SLORA_OK;
}

slora_status rank_set_wait_budget(long long cycles) {
  const long long v = cycles < 0 ? kWaitBudget : cycles;
  SLORA_CUDA(cudaMemcpyToSymbol(g_rank_budget, &v, sizeof(v)));
  return SLORA_OK;
}

slora_status rank_check_error(bool clear) {
  int v = 0, bad = 0;
  SLORA_CUDA(cudaMemcpyFromSymbol(&v, g_rank_error, sizeof(int)));
  SLORA_CUDA(cudaMemcpyFromSymbol(&bad, g_rank_bad_index, sizeof(int)));
  if (clear && (v || bad)) {
    const int z = 0;
    SLORA_CUDA(cudaMemcpyToSymbol(g_rank_error, &z, sizeof(int)));
    SLORA_CUDA(cudaMemcpyToSymbol(g_rank_bad_index, &z, sizeof(int)));
  }
  if (bad)
    SLORA_FAIL(SLORA_ERR_INVALID_ARG, "a channel index lies outside its weight (read as zeros)");
  if (v) SLORA_FAIL(SLORA_ERR_TIMEOUT, "a rank contraction's bounded wait expired");
  return SLORA_OK;
}

}  // namespace slora
