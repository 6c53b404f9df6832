// The rank-r contractions of a LoRA linear's backward (y = x W0^T + s (x A^T) B^T):
//   rank_rows   p = dY B, row by row               (reads dY)
//   rank_sums   dA = s p^T X, dB = s dY^T (X A^T)  (sums over tokens; read X and dY)
// Each streams a large activation past a matrix with r columns, so both are
// bound by that stream; X may be an 8-bit checkpoint (1.03 bytes a value).
//
// rank_rows: mma.sync m16n8k16 with fragments loaded straight from global
// memory.  The channel order inside a reduction is free, so lane t of a quad
// takes 8 consecutive channels (one 16-byte load a row, the same 8 channels of
// B's transposed copy), two k-steps of fragments.  A block owns 16 rows, its
// eight warps take every eighth 32-channel group and are summed in order in
// shared memory: no partial sums leave the block.
//
// rank_sums: tcgen05.mma with 128 channels as M, the tokens as the reduction and
// N = 48: 16 rank columns in three bf16 terms (an fp32 operand to 2^-24), so the
// sums are those of fp32 operands.  Legacy mma.sync took 21 us for 4096 x 4096
// codes at r = 16, packed fp32 FMAs 30 us.  X lies in shared memory as it does
// in global memory, a token's 128 channels in a row (an M-major operand, 128-byte
// swizzle): bf16 rows are copied there asynchronously; codes are copied to a
// ring beside it and expanded by the thread that asked for them (a byte permute
// pairs two codes, two logic operations and an addition make them bf16, a
// product applies the step: all exact).  The same eight warps split the token's P
// row into its terms.  A stage is 64 tokens, three stages are on their way; a
// ninth warp issues the products.  The stages take turns on four accumulators:
// the tensor core truncates each addition, and four short chains added in fp32
// are off by a quarter of one long one.  Blocks that share channels leave partial
// sums that the last to arrive adds in order: the result does not depend on
// timing.  Every wait is bounded; on expiry the block raises a device flag
// (slora_device_error: SLORA_ERR_TIMEOUT) and leaves after its own work ended.
#include <algorithm>

#include "act8_dev.cuh"
#include "lora_grad.cuh"

namespace slora {

__device__ int g_rank_error = 0;

namespace {

constexpr int kWarps = 8;
constexpr int kCols = 16;  // rank columns of a block (more: further blocks)

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------------- rows
struct RowsJob {
  const __nv_bfloat16* Y;
  const __nv_bfloat16* R;  // [cols rounded up to 16][K64]
  long long ld, M, K, K64;
  float* out1;
  long long ld1;
  const int32_t* map1;
  __nv_bfloat16* out2;
  long long ld2;
};
struct RowsParams {
  RowsJob job[2];
  int blocks0;  // 16-row blocks of job 0
  int cols;
  float s2;
};

__global__ void __launch_bounds__(kWarps * 32) rank_rows_kernel(const __grid_constant__ RowsParams P) {
  __shared__ float red[kWarps][16][kCols + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const bool second = int(blockIdx.x) >= P.blocks0;
  const RowsJob& j = P.job[second ? 1 : 0];
  const long long m0 = (long long)(int(blockIdx.x) - (second ? P.blocks0 : 0)) * 16;
  const int q0 = blockIdx.y * kCols;
  const bool on0 = m0 + g < j.M, on1 = m0 + g + 8 < j.M;
  const __nv_bfloat16* y0 = j.Y + (m0 + g) * j.ld;
  const __nv_bfloat16* y1 = y0 + 8 * j.ld;
  const __nv_bfloat16* r0 = j.R + (q0 + g) * j.K64;
  const __nv_bfloat16* r1 = r0 + 8 * j.K64;
  float acc[2][4] = {};
  const uint4 none = make_uint4(0, 0, 0, 0);
  // four groups of 32 channels in flight; every 8-channel load lies inside the
  // row's whole 16-byte units or is left out
  for (long long c0 = warp * 32; c0 < j.K; c0 += kWarps * 32 * 4) {
    uint4 a[4], b[4], r[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long c = c0 + i * kWarps * 32 + 8 * t;
      const bool on = c < j.K;
      a[i] = on && on0 ? *reinterpret_cast<const uint4*>(y0 + c) : none;
      b[i] = on && on1 ? *reinterpret_cast<const uint4*>(y1 + c) : none;
      r[i] = on ? __ldg(reinterpret_cast<const uint4*>(r0 + c)) : none;
      s[i] = on ? __ldg(reinterpret_cast<const uint4*>(r1 + c)) : none;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
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
  const int row = threadIdx.x / kCols, q = threadIdx.x % kCols;  // 256 threads: one value each
  const long long m = m0 + row;
  if (m >= j.M || q0 + q >= P.cols) return;
  float v = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += red[w][row][q];
  j.out1[(j.map1 ? (long long)j.map1[m] : m) * j.ld1 + q0 + q] = v;
  j.out2[m * j.ld2 + q0 + q] = __float2bfloat16_rn(P.s2 * v);
}

// ------------------------------------------------------------------- sums
constexpr int kCh = 128;            // channels of a block (M)
constexpr int kTok = 64;            // tokens of a stage
constexpr int kTerms = 3;           // bf16 terms of an fp32 rank operand
constexpr int kAcc = 4;             // accumulators the stages take turns on
constexpr int kTile = kCh * kCols;  // outputs of a block
constexpr int kFetch = 3;           // stages on their way beside the current one (bf16: 2)
constexpr int kABytes = kTok * kCh * 2;              // 16 KB: two 64-channel halves
constexpr int kBBytes = kTerms * kCols * kTok * 2;   // 6 KB
constexpr int kPBytes = kTok * kCols * 4;            // 4 KB: raw P rows
constexpr int kXBytes = kTok * kCh;                  // 8 KB: raw codes
// Operand slots: bf16 rows arrive in them, codes are expanded into them.
constexpr int kSlotsB16 = 4, kSlots8 = 2;
constexpr int kSumSmem = 1024 + kSlotsB16 * (kABytes + kBBytes) + (kFetch + 1) * kPBytes;  // 105 KB
static_assert(kSlots8 * (kABytes + kBBytes) + (kFetch + 1) * kXBytes <= kSlotsB16 * (kABytes + kBBytes),
              "codes' layout inside the bf16 layout's memory");
constexpr int kTmemCols = 256;  // kAcc * 64, of which 48 each are used
constexpr long long kWaitBudget = 2000000000LL;  // ~1 s of SM clocks per wait

struct SumJob {
  const uint8_t* X;       // codes, or bf16 values
  const uint8_t* scales;  // null: bf16
  long long ld;           // elements of a row
  long long M, K;
  const float* P;
  long long ldp;
  const int32_t* map;
  float* out;
  long long ldo;
  int trans, nsplit, blocks;  // blocks: channel blocks * splits
  int stages;                 // of one split
  int tile0;                  // first output tile (partials and counters)
};
struct SumParams {
  SumJob job[kRankSums];
  int n, cols, tiles;  // tiles: output tiles of one column slice
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
// Bounded wait for the phase of parity `parity`; false on abort or expiry.
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity, volatile int* abort) {
  if (mbar_try(b, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_try(b, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitBudget) {
      *abort = 1;
      atomicExch(&g_rank_error, 1);
      return false;
    }
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
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool on) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 4 : 0)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
__device__ __forceinline__ void sts16(uint32_t a, __nv_bfloat16 v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(__bfloat16_as_ushort(v)) : "memory");
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

// The eight producer warps' work on one (channel block, split).
template <bool kCodes>
__device__ __forceinline__ bool sum_produce(const SumJob& j, long long ch0, int q0, int cols,
                                            long long m0, int stages, uint8_t* smem,
                                            uint64_t* full, uint64_t* empty,
                                            volatile int* abort, int tid) {
  constexpr int kSlots = kCodes ? kSlots8 : kSlotsB16;
  // bf16 rows arrive in their operand slot: one stage fewer, so that a copy
  // waits for products issued two stages ago
  constexpr int kAhead = kCodes ? kFetch : kFetch - 1;
  const uint32_t sA = su32(smem), sB = sA + kSlots * kABytes;
  const uint32_t sX = sB + kSlots * kBBytes;  // codes
  const uint32_t sP = sA + kSumSmem - 1024 - (kFetch + 1) * kPBytes;
  const int lane = tid & 31;
  // this thread's share of P: token tid / 4, columns q0 + 4 (tid % 4) ...
  const int pt = tid >> 2, pq = 4 * (tid & 3);
  const bool vec = q0 + kCols <= cols && j.ldp % 4 == 0;
  auto row_of = [&](int st) -> long long {  // its row of P in stage st, or -1
    const long long m = m0 + (long long)st * kTok + pt;
    if (st >= stages || m >= j.M) return -1;
    return j.map ? (long long)j.map[m] : m;
  };
  auto slot_free = [&](int st) {  // the products of the slot's last stage are done
    return st < kSlots || mbar_wait(&empty[st % kSlots], uint32_t(st / kSlots - 1) & 1u, abort);
  };
  auto fetch = [&](int st, long long prow) {
    if (st < stages) {
      const long long mb = m0 + (long long)st * kTok;
      if constexpr (kCodes) {
        const uint32_t dst = sX + (st % (kFetch + 1)) * kXBytes + tid * 16;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int id = tid + 256 * i, t = id >> 3;
          const long long ch = ch0 + 16 * (id & 7);
          const bool on = mb + t < j.M && ch < j.ld;
          cp_async<16>(dst + 4096 * i, j.X + (on ? (mb + t) * j.ld + ch : 0), on);
        }
      } else {
        const uint32_t dst = sA + (st % kSlots) * kABytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int id = tid + 256 * i, t = id >> 4, u = id & 15;
          const long long ch = ch0 + 8 * u;
          const bool on = mb + t < j.M && ch < j.ld;
          cp_async<16>(dst + x_at(t, u), j.X + (on ? ((mb + t) * j.ld + ch) * 2 : 0), on);
        }
      }
      const uint32_t dp = sP + (st % (kFetch + 1)) * kPBytes + tid * 16;
      const float* src = j.P + (prow >= 0 ? prow * j.ldp + q0 + pq : 0);
      if (vec) {
        cp_async<16>(dp, src, prow >= 0);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool on = prow >= 0 && q0 + pq + e < cols;
          cp_async<4>(dp + 4 * e, on ? src + e : j.P, on);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // scale bytes of this thread's two code chunks in stage st
  auto bytes_of = [&](int st, uint32_t (&b)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int id = tid + 256 * i;
      const long long m = m0 + (long long)st * kTok + (id >> 3), ch = ch0 + 16 * (id & 7);
      b[i] = st < stages && m < j.M && ch < j.ld ? j.scales[(m * j.ld + ch) >> 5] : 7u;
    }
  };
  uint32_t byte[kAhead][2];
  long long prow[kAhead + 1];
#pragma unroll
  for (int st = 0; st <= kAhead; ++st) prow[st] = row_of(st);
#pragma unroll
  for (int st = 0; st < kAhead; ++st) {
    fetch(st, prow[st]);
    if constexpr (kCodes) bytes_of(st, byte[st]);
  }
  long long next_row = prow[kAhead];
  bool ok = true;
  for (int st = 0; st < stages; ++st) {
    if constexpr (!kCodes) {
      if (!slot_free(st + kAhead < stages ? st + kAhead : 0)) { ok = false; break; }
    }
    fetch(st + kAhead, next_row);
    next_row = row_of(st + kAhead + 1);
    uint32_t nb[2] = {7u, 7u};
    if constexpr (kCodes) bytes_of(st + kAhead, nb);
    cp_wait<kAhead>();  // stage st of this thread has arrived
    if constexpr (kCodes) {
      if (!slot_free(st)) { ok = false; break; }
      const uint32_t src = sX + (st % (kFetch + 1)) * kXBytes + tid * 16;
      const uint32_t dst = sA + (st % kSlots) * kABytes;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int id = tid + 256 * i, t = id >> 3, u = 2 * (id & 7);
        const uint4 w = lds128(src + 4096 * i);
        const uint32_t b = byte[0][i];
        const uint32_t e = b == 255u ? 0x7fff7fffu : ((b - 6u) << 7) * 0x10001u;
        const __nv_bfloat162 step = act8_as_bf162(e);
        sts128(dst + x_at(t, u), make_uint4(code_pair<0>(w.x, step), code_pair<2>(w.x, step),
                                            code_pair<0>(w.y, step), code_pair<2>(w.y, step)));
        sts128(dst + x_at(t, u + 1), make_uint4(code_pair<0>(w.z, step), code_pair<2>(w.z, step),
                                                code_pair<0>(w.w, step), code_pair<2>(w.w, step)));
      }
#pragma unroll
      for (int f = 0; f + 1 < kAhead; ++f) {
        byte[f][0] = byte[f + 1][0];
        byte[f][1] = byte[f + 1][1];
      }
      byte[kAhead - 1][0] = nb[0];
      byte[kAhead - 1][1] = nb[1];
    }
    {  // the three terms of this thread's four P values, transposed: row (term, column), token
      const uint4 w = lds128(sP + (st % (kFetch + 1)) * kPBytes + tid * 16);
      const uint32_t dst = sB + (st % kSlots) * kBBytes;
      const float v[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z),
                          __uint_as_float(w.w)};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float rest = v[e];
#pragma unroll
        for (int s = 0; s < kTerms; ++s) {
          const __nv_bfloat16 h = __float2bfloat16_rn(rest);
          rest -= __bfloat162float(h);
          const int row = s * kCols + pq + e;
          sts16(dst + row * 128 + (((pt >> 3) ^ (row & 7)) << 4) + (pt & 7) * 2, h);
        }
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[st % kSlots]);
  }
  cp_wait<0>();
  return ok;
}

__global__ void __launch_bounds__(kWarps * 32 + 32, 2) rank_sums_kernel(const __grid_constant__ SumParams P) {
  extern __shared__ uint8_t s_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kSlotsB16], empty[kSlotsB16], done;
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
  if (tid == 0) {
    for (int i = 0; i < kSlotsB16; ++i) {
      mbar_init(&full[i], kWarps);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     su32(&s_tmem)),
                 "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tbase = s_tmem;
  volatile int* abort = &s_abort;

  if (warp < kWarps) {
    if (codes)
      sum_produce<true>(j, ch0, q0, P.cols, m0, stages, smem, full, empty, abort, tid);
    else
      sum_produce<false>(j, ch0, q0, P.cols, m0, stages, smem, full, empty, abort, tid);
  } else if (lane == 0) {
    const int slots = codes ? kSlots8 : kSlotsB16;
    const uint32_t sA = su32(smem), sB = sA + slots * kABytes;
    for (int st = 0; st < stages; ++st) {
      const int slot = st % slots;
      if (!mbar_wait(&full[slot], uint32_t(st / slots) & 1u, abort)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t d = tbase + uint32_t(st % kAcc) * 64u;
#pragma unroll
      for (int k = 0; k < kTok / 16; ++k)
        mma_1sm(d, sdesc(sA + slot * kABytes + k * 2048, kTok * 128, 1024),
                sdesc(sB + slot * kBBytes + k * 32, 16, 1024), st >= kAcc || k > 0 ? 1u : 0u);
      mma_commit(&empty[slot]);
    }
    if (stages > 0) {
      mma_commit(&done);
      // nothing of this block may be in flight when it leaves, aborted or not
      const long long t0 = clock64();
      while (!mbar_try(&done, 0) && clock64() - t0 < kWaitBudget) {
      }
      if (!mbar_try(&done, 0)) {
        s_abort = 1;
        atomicExch(&g_rank_error, 1);
      }
    }
  }
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");

  const int tile = int(blockIdx.y) * P.tiles + j.tile0 + cb;
  const long long ch = ch0 + 32 * warp + lane;  // TMEM lane = channel (warps 0 .. 3)
  float4* mine = reinterpret_cast<float4*>(
      P.part + ((long long)blockIdx.y * gridDim.x + blockIdx.x) * kTile) + 32 * (warp & 3) + lane;
  auto emit = [&](const float (&v)[16]) {
    if (ch >= j.K) return;
#pragma unroll
    for (int q = 0; q < kCols; ++q)
      if (q0 + q < P.cols)
        j.out[j.trans ? (q0 + q) * j.ldo + ch : ch * j.ldo + q0 + q] = v[q] * P.scale;
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
      emit(v);
    } else {  // [4 columns of 4][128 channels] of float4
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mine[q * kCh] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == kWarps) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase),
                 "n"(kTmemCols)
                 : "memory");
  }
  if (j.nsplit == 1) return;
  if (tid == 0) {
    __threadfence();
    const unsigned prev = atomicAdd(&P.counters[tile], 1u);
    s_last = prev + 1 == unsigned(j.nsplit);
    if (s_last) P.counters[tile] = 0u;
  }
  __syncthreads();
  if (!s_last || warp >= 4) return;
  __threadfence();
  // split s of this channel block ran as block (blockIdx.x - blk) + s * nch + cb
  const float4* src = reinterpret_cast<const float4*>(
      P.part + ((long long)blockIdx.y * gridDim.x + blockIdx.x - blk + cb) * kTile) + 32 * warp + lane;
  float v[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) v[q] = 0.0f;
#pragma unroll 2
  for (int s = 0; s < j.nsplit; ++s) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 f = __ldcg(src + ((long long)s * nch * kTile) / 4 + q * kCh);
      v[4 * q] += f.x;
      v[4 * q + 1] += f.y;
      v[4 * q + 2] += f.z;
      v[4 * q + 3] += f.w;
    }
  }
  emit(v);
}

int slices(int cols) { return (cols + kCols - 1) / kCols; }
int64_t channel_blocks(const RankSum& j) { return (j.K + kCh - 1) / kCh; }
// Splits of each job over the tokens: two blocks an SM over the launch, shared
// in proportion to the jobs' sizes, none without a stage, at most 32 (the last
// block of a tile adds them).
void plan_splits(const RankSum* jobs, int n, int cols, int* nsplit, int* per) {
  double total = 0.0;
  for (int i = 0; i < n; ++i) total += double(jobs[i].M) * double(jobs[i].K);
  for (int i = 0; i < n; ++i) {
    const int64_t nch = std::max<int64_t>(channel_blocks(jobs[i]), 1);
    const int64_t stages = std::max<int64_t>((jobs[i].M + kTok - 1) / kTok, 1);
    const double share = total > 0.0 ? double(jobs[i].M) * double(jobs[i].K) / total : 0.0;
    int64_t want = int64_t(2.0 * num_sms() * share / double(nch * slices(cols)) + 0.5);
    want = std::max<int64_t>(1, std::min<int64_t>({want, stages, 32}));
    const int64_t each = (stages + want - 1) / want;
    nsplit[i] = int((stages + each - 1) / each);
    per[i] = int(each);
  }
}

}  // namespace

slora_status rank_rows(const RankRows* jobs, int n, int cols, float s2, cudaStream_t st) {
  if (n < 1 || n > 2) SLORA_FAIL(SLORA_ERR_SHAPE, "rank_rows: %d jobs", n);
  RowsParams p{};
  int64_t blocks[2] = {0, 0};
  double bytes = 0.0;
  for (int i = 0; i < n; ++i) {
    const RankRows& s = jobs[i];
    RowsJob& j = p.job[i];
    j.Y = static_cast<const __nv_bfloat16*>(s.Y);
    j.R = static_cast<const __nv_bfloat16*>(s.R);
    j.ld = s.ld; j.M = s.M; j.K = s.K;
    j.K64 = (std::max<int64_t>(s.K, 1) + 63) / 64 * 64;
    j.out1 = s.out1; j.ld1 = s.ld1; j.map1 = s.map1;
    j.out2 = static_cast<__nv_bfloat16*>(s.out2); j.ld2 = s.ld2;
    blocks[i] = (s.M + 15) / 16;
    bytes += double(s.M) * s.K * 2;
    if (s.M > 0 && s.K > 0 && (!aligned16(s.Y) || s.ld % 8))
      SLORA_FAIL(SLORA_ERR_ALIGN, "rank_rows: rows are not whole 16-byte units");
  }
  if (blocks[0] + blocks[1] == 0) return SLORA_OK;
  p.blocks0 = int(blocks[0]);
  p.cols = cols;
  p.s2 = s2;
  LaunchScope ls(kSkinny, bytes, st);
  rank_rows_kernel<<<dim3(unsigned(blocks[0] + blocks[1]), unsigned(slices(cols))), kWarps * 32, 0,
                     st>>>(p);
  SLORA_CHECK_LAUNCH();
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
                       unsigned* counters, cudaStream_t st) {
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
    j.X = codes ? reinterpret_cast<const uint8_t*>(s.X8.codes) : static_cast<const uint8_t*>(s.X);
    j.scales = codes ? s.X8.scales : nullptr;
    j.ld = codes ? act8_cols(s.K) : s.ld;
    j.M = s.M; j.K = s.K;
    j.P = s.P; j.ldp = s.ldp; j.map = s.map;
    j.out = s.out; j.ldo = s.ldo; j.trans = s.trans;
    j.nsplit = nsplit[i];
    j.stages = per[i];
    j.blocks = int(channel_blocks(s)) * nsplit[i];
    j.tile0 = int(tiles);
    tiles += channel_blocks(s);
    blocks += j.blocks;
    bytes += double(s.M) * s.K * (codes ? 1.03125 : 2.0);
    if (!codes && s.M > 0 && s.K > 0 && (!aligned16(s.X) || s.ld % 8))
      SLORA_FAIL(SLORA_ERR_ALIGN, "rank_sums: rows are not whole 16-byte units");
  }
  if (blocks == 0) return SLORA_OK;
  p.n = n;
  p.cols = cols;
  p.tiles = int(tiles);
  p.scale = scale;
  p.part = part;
  p.counters = counters;
  SLORA_CUDA(cudaFuncSetAttribute(rank_sums_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  kSumSmem));
  LaunchScope ls(kSkinny, bytes * slices(cols), st);
  rank_sums_kernel<<<dim3(unsigned(blocks), unsigned(slices(cols))), kWarps * 32 + 32, kSumSmem,
                     st>>>(p);
  SLORA_CHECK_LAUNCH();
  return SLORA_OK;
}

slora_status rank_check_error(bool clear) {
  int v = 0;
  SLORA_CUDA(cudaMemcpyFromSymbol(&v, g_rank_error, sizeof(int)));
  if (clear && v) {
    const int z = 0;
    SLORA_CUDA(cudaMemcpyToSymbol(g_rank_error, &z, sizeof(int)));
  }
  if (v) SLORA_FAIL(SLORA_ERR_TIMEOUT, "a rank contraction's bounded wait expired");
  return SLORA_OK;
}

}  // namespace slora
