// Activation checkpoints in 8 bits: packing, unpacking, and the token-summed
// contraction of a LoRA gradient that reads its activation as codes.
//
// Format (slora.h): blocks of 32 channels of a row share a power-of-two step,
// so dividing by it is exact, a code is one rounding of the value, and code *
// step is exact in bf16 (7 bits of magnitude): the tensor cores take the
// checkpoint's values without a further rounding.
//
// Packing and unpacking are bound by memory, 2 + 1 + 1/32 bytes a value in
// bf16.  A thread holds 8 channels (a 16-byte load, an 8-byte store), four
// neighbouring lanes share a block and its maximum (two shuffles), and each
// thread has four chunks in flight.
#include <algorithm>
#include <type_traits>

#include "act8.cuh"
#include "act8_dev.cuh"

namespace slora {
namespace {

// n / d for n < 2^31 and 4 <= d < 2^31: (n * mul) >> (32 + shift).
struct FastDiv {
  uint32_t d, mul, shift;
};
FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((uint64_t(1) << l) < d) ++l;  // ceil(log2 d), at least 2
  FastDiv f;
  f.d = d;
  f.shift = l - 1;
  f.mul = uint32_t(((uint64_t(1) << (31 + l)) + d - 1) / d);
  return f;
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) {
  return __umulhi(n, f.mul) >> f.shift;
}

constexpr int kThreads = 256;
constexpr int kChunks = 4;  // chunks of 8 channels a thread has in flight

__device__ __forceinline__ void load8(const float* p, int n, bool vec, float (&f)[8]) {
  if (vec && n >= 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0];
    const float4 b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? p[i] : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int n, bool vec, const float (&f)[8]) {
  if (vec && n >= 8) {
    if constexpr (std::is_same<T, float>::value) {
      reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      uint4 u;
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      *reinterpret_cast<uint4*>(p) = u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (std::is_same<T, float>::value) p[i] = f[i];
        else p[i] = __float2bfloat16_rn(f[i]);
      }
  }
}

// A chunk as packed bf16 (rows that are no whole 16-byte units by elements).
__device__ __forceinline__ uint4 load8_bf16(const __nv_bfloat16* p, int n, bool vec) {
  if (vec && n >= 8) return *reinterpret_cast<const uint4*>(p);
  uint4 u = make_uint4(0, 0, 0, 0);
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i / 2] |= uint32_t(__bfloat16_as_ushort(p[i])) << (16 * (i & 1));
  return u;
}

// Chunk i of the rows: row i / per_row, channels 8 (i % per_row) ...; a block
// of threads takes kChunks * 256 consecutive chunks, each thread every 256th.
template <typename T>
__global__ void __launch_bounds__(kThreads) act8_pack_kernel(
    const T* __restrict__ X, int64_t ldx, int64_t d, uint32_t total, const FastDiv per_row,
    bool vec, uint2* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr bool kF = std::is_same<T, float>::value;
  const uint32_t base = blockIdx.x * uint32_t(kThreads * kChunks) + threadIdx.x;
  float f[kF ? kChunks : 1][8];
  uint4 u[kF ? 1 : kChunks];
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    const uint32_t i = base + k * kThreads;
    const uint32_t row = div_by(i, per_row), c = (i - row * per_row.d) * 8;
    const int64_t left = i < total ? d - int64_t(c) : 0;
    const T* x = X + (left > 0 ? int64_t(row) * ldx + c : 0);
    const int n = int(left < 8 ? left : 8);
    if constexpr (kF) load8(x, n, vec, f[k]);
    else u[k] = load8_bf16(x, n, vec);
  }
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    const uint32_t i = base + k * kThreads;
    uint32_t byte;
    uint2 c;
    if constexpr (kF) {
      byte = act8_byte(act8_block_max(act8_chunk_bits(f[k])));
      c = act8_codes8_f32(f[k], byte);
    } else {
      byte = act8_byte_bf16(u[k]);
      c = act8_codes8_bf16(u[k], byte);
    }
    if (i >= total) continue;
    codes[i] = c;
    if ((threadIdx.x & 3) == 0) scales[i >> 2] = uint8_t(byte);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) act8_unpack_kernel(
    const uint2* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t ldx, int64_t d,
    uint32_t total, const FastDiv per_row, bool vec, T* __restrict__ X) {
  const uint32_t base = blockIdx.x * uint32_t(kThreads * kChunks) + threadIdx.x;
  uint2 c[kChunks];
  uint32_t b[kChunks];
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    const uint32_t i = base + k * kThreads;
    if (i < total) {
      c[k] = codes[i];
      b[k] = scales[i >> 2];
    }
  }
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    const uint32_t i = base + k * kThreads;
    if (i >= total) continue;
    const uint32_t row = div_by(i, per_row), col = (i - row * per_row.d) * 8;
    const int64_t left = d - int64_t(col);
    if (left <= 0) continue;
    float f[8];
    act8_values8(c[k], b[k], f);
    store8(X + int64_t(row) * ldx + col, int(left < 8 ? left : 8), vec, f);
  }
}

// ------------------------------------------------------- LoRA contraction
// dA = s P^T X over the tokens, P = dY B (fp32, three bf16 terms), X a
// checkpoint: mma.sync m16n8k16 with channels as rows, tokens as the reduction
// and 16 rank columns.  Bound by the codes' stream (1.03 bytes a value, half
// of bf16's), so they go from global memory to registers with no staging: a
// warp owns 128 channels, and a lane loads 16 channels of 4 consecutive tokens
// (four 16-byte loads: the 8 lanes of a quad group cover a 128-byte line of
// each token).  The reduction index is free, so lane t of a quad takes tokens
// 4t .. 4t + 3 in the places of 2t, 2t + 1, 2t + 8, 2t + 9, and the same four
// tokens of P are one 8-byte load; the channels' order inside the fragments is
// free too.  A byte permute pairs two tokens' codes, two logic operations and
// one addition turn them into bf16 (128 + the low seven bits, less 128 or, for
// a negative code, 256), one product applies the two tokens' steps, all exact.
// The eight warps of a block take different tokens and are summed in order in
// shared memory; blocks that share channels leave partial sums that the last
// one to arrive adds in order, so the result does not depend on timing.
constexpr int kDotCh = 128, kDotWarps = 8, kDotStep = 16 * kDotWarps, kDotCols = 16;
constexpr int kDotTile = kDotCh * kDotCols;
// A warp's tile in shared memory: [16 columns] of 128 channels and 4 floats of
// padding, channel c at (c % 16) * 8 + c / 16, so that the 32 lanes of one
// accumulator register store to 32 banks.
constexpr int kDotRow = kDotCh + 4;
constexpr int kDotSmem = kDotWarps * kDotCols * kDotRow * 4;  // 66 KB

struct DotParams {
  const uint8_t* codes;
  const uint8_t* scales;
  long long ld;   // codes a row (a multiple of 32)
  long long M, K, I64;
  const __nv_bfloat16* P;  // [3][cp][I64]
  int cp, cols, nsplit;
  long long steps;  // of kDotStep tokens, per split
  float* part;
  unsigned* counters;
  float* out;
  long long ldo;
  const int32_t* kmap;
  float scale;
  int accumulate;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Codes of one channel at two tokens (byte j of each word) times the tokens'
// steps, as packed bf16.
template <int J>
__device__ __forceinline__ uint32_t code_pair(uint32_t lo, uint32_t hi, __nv_bfloat162 step) {
  const uint32_t u = __byte_perm(lo, hi, J | ((4 + J) << 8));  // bytes 0 and 2: the two codes
  const uint32_t a = (u & 0x007f007fu) | 0x43004300u;  // 128 + the low seven bits
  const uint32_t c = (u & 0x00800080u) | 0xc300c300u;  // -128, or -256 for a negative code
  const __nv_bfloat162 v = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&c));
  const __nv_bfloat162 r = __hmul2(v, step);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t step_bits(uint32_t byte) {  // bf16 of 2^(byte - 133)
  return byte == 255u ? 0x7fffu : (byte - 6u) << 7;
}

struct DotRows {
  uint4 x[4];
  uint32_t b[4];
};

__global__ void __launch_bounds__(kDotWarps * 32, 2) act8_dot_kernel(const __grid_constant__ DotParams p) {
  extern __shared__ __align__(16) float s_acc[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const long long ch0 = (long long)blockIdx.x * kDotCh + 16 * g;  // this lane's 16 channels
  const int split = blockIdx.y, q0 = blockIdx.z * kDotCols;
  const bool inside = ch0 < p.ld;  // rows are whole blocks of 32, so all 16 or none
  float acc[8][2][4] = {};
  const long long step0 = split * p.steps;
  const long long step1 = min(step0 + p.steps, (p.M + kDotStep - 1) / kDotStep);
  auto load = [&](long long step, DotRows& r) {
    const long long m0 = step * kDotStep + warp * 16 + 4 * t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool on = inside && step < step1 && m0 + i < p.M;
      const long long o = on ? (m0 + i) * p.ld + ch0 : 0;
      r.x[i] = on ? *reinterpret_cast<const uint4*>(p.codes + o) : make_uint4(0, 0, 0, 0);
      r.b[i] = on ? p.scales[o >> 5] : 7u;
    }
  };
  DotRows cur, nxt;
  load(step0, cur);
  for (long long step = step0; step < step1; ++step) {
    load(step + 1, nxt);
    const long long m0 = step * kDotStep + warp * 16 + 4 * t;
    // rows of P^T past the padded token count read as zero
    uint2 b[3][2];
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
      for (int n = 0; n < 2; ++n)
        b[s][n] = m0 < p.I64
                      ? *reinterpret_cast<const uint2*>(
                            p.P + ((long long)s * p.cp + q0 + n * 8 + g) * p.I64 + m0)
                      : make_uint2(0, 0);
    const uint32_t s01 = step_bits(cur.b[0]) | (step_bits(cur.b[1]) << 16);
    const uint32_t s23 = step_bits(cur.b[2]) | (step_bits(cur.b[3]) << 16);
    const __nv_bfloat162 e01 = *reinterpret_cast<const __nv_bfloat162*>(&s01);
    const __nv_bfloat162 e23 = *reinterpret_cast<const __nv_bfloat162*>(&s23);
    const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&cur.x[0]);
    const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&cur.x[1]);
    const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&cur.x[2]);
    const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&cur.x[3]);
    // fragment f holds channels 2f (row g) and 2f + 1 (row g + 8) of each lane's 16
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      const int w = f / 2;
      uint32_t a0, a1, a2, a3;
      if (f % 2 == 0) {
        a0 = code_pair<0>(w0[w], w1[w], e01);
        a1 = code_pair<1>(w0[w], w1[w], e01);
        a2 = code_pair<0>(w2[w], w3[w], e23);
        a3 = code_pair<1>(w2[w], w3[w], e23);
      } else {
        a0 = code_pair<2>(w0[w], w1[w], e01);
        a1 = code_pair<3>(w0[w], w1[w], e01);
        a2 = code_pair<2>(w2[w], w3[w], e23);
        a3 = code_pair<3>(w2[w], w3[w], e23);
      }
#pragma unroll
      for (int s = 0; s < 3; ++s)
#pragma unroll
        for (int n = 0; n < 2; ++n) mma_bf16(acc[f][n], a0, a1, a2, a3, b[s][n].x, b[s][n].y);
    }
    cur = nxt;
  }
  float* mine = s_acc + warp * kDotCols * kDotRow;
#pragma unroll
  for (int f = 0; f < 8; ++f)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)  // row g + 8 (e / 2), column 2t + (e % 2)
        mine[(n * 8 + 2 * t + (e & 1)) * kDotRow + (2 * f + (e >> 1)) * 8 + g] = acc[f][n][e];
  __syncthreads();
  const int blocks_x = int(gridDim.x);
  const long long tile = (long long)blockIdx.z * blocks_x + blockIdx.x;  // output tile of this block
  auto emit = [&](int i, float v) {
    const int q = q0 + i / kDotCh;
    const long long c = (long long)blockIdx.x * kDotCh + i % kDotCh;
    if (q >= p.cols || c >= p.K) return;
    float* o = p.out + q * p.ldo + (p.kmap ? (long long)p.kmap[c] : c);
    v *= p.scale;
    *o = p.accumulate ? *o + v : v;
  };
  for (int i = threadIdx.x; i < kDotTile; i += blockDim.x) {
    const int c = i % kDotCh, at = i / kDotCh * kDotRow + (c & 15) * 8 + (c >> 4);
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kDotWarps; ++w) v += s_acc[w * kDotCols * kDotRow + at];
    if (p.nsplit == 1) emit(i, v);
    else p.part[(tile * p.nsplit + split) * kDotTile + i] = v;
  }
  if (p.nsplit == 1) return;
  __shared__ unsigned s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const unsigned prev = atomicAdd(&p.counters[tile], 1u);
    s_last = prev + 1 == unsigned(p.nsplit);
    if (s_last) p.counters[tile] = 0u;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int i = threadIdx.x; i < kDotTile; i += blockDim.x) {
    float v = 0.0f;
    for (int s = 0; s < p.nsplit; ++s) v += __ldcg(&p.part[(tile * p.nsplit + s) * kDotTile + i]);
    emit(i, v);
  }
}

int col_slices(int cols) { return (cols + kDotCols - 1) / kDotCols; }
// Splits over the tokens: about two blocks an SM in all, at most 32, none
// without a step.
int dot_splits(int64_t M, int64_t K, int cols) {
  const int64_t tiles = std::max<int64_t>((K + kDotCh - 1) / kDotCh, 1) * col_slices(cols);
  const int64_t steps = std::max<int64_t>((M + kDotStep - 1) / kDotStep, 1);
  const int64_t want = std::max<int64_t>(1, (2 * num_sms() + tiles - 1) / tiles);
  const int64_t per = (steps + std::min<int64_t>(want, 32) - 1) / std::min<int64_t>(want, 32);
  return int((steps + per - 1) / per);
}

// Rows of one launch: fewer than 2^30 chunks.
int64_t rows_per_launch(int64_t d) {
  return std::max<int64_t>(1, (int64_t(1) << 30) / (act8_cols(d) / 8));
}

}  // namespace

slora_status act8_pack_run(int dt, int64_t T, int64_t d, const void* X, int64_t ldx,
                           const slora_act8& out, cudaStream_t st) {
  const int64_t d32 = act8_cols(d), per = d32 / 8;
  const FastDiv fd = fast_div(uint32_t(per));
  const bool vec = ldx % 8 == 0 || T == 1;
  const int64_t step = rows_per_launch(d);
  for (int64_t t0 = 0; t0 < T; t0 += step) {
    const int64_t rows = std::min(step, T - t0);
    const uint32_t total = uint32_t(rows * per);
    const unsigned grid = (total + kThreads * kChunks - 1) / (kThreads * kChunks);
    uint2* codes = reinterpret_cast<uint2*>(out.codes + t0 * d32);
    uint8_t* scales = out.scales + t0 * (d32 / kActBlock);
    LaunchScope ls(kElementwise, double(rows) * d * (dt_size(dt) + 1.03125), st);
    if (dt == kF32)
      act8_pack_kernel<float><<<grid, kThreads, 0, st>>>(static_cast<const float*>(X) + t0 * ldx,
                                                         ldx, d, total, fd, vec, codes, scales);
    else
      act8_pack_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(
          static_cast<const __nv_bfloat16*>(X) + t0 * ldx, ldx, d, total, fd, vec, codes, scales);
    SLORA_CHECK_LAUNCH();
  }
  return SLORA_OK;
}

slora_status act8_unpack_run(int dt, int64_t T, int64_t d, const slora_act8& in, void* X,
                             int64_t ldx, cudaStream_t st) {
  const int64_t d32 = act8_cols(d), per = d32 / 8;
  const FastDiv fd = fast_div(uint32_t(per));
  const bool vec = ldx % 8 == 0 || T == 1;
  const int64_t step = rows_per_launch(d);
  for (int64_t t0 = 0; t0 < T; t0 += step) {
    const int64_t rows = std::min(step, T - t0);
    const uint32_t total = uint32_t(rows * per);
    const unsigned grid = (total + kThreads * kChunks - 1) / (kThreads * kChunks);
    const uint2* codes = reinterpret_cast<const uint2*>(in.codes + t0 * d32);
    const uint8_t* scales = in.scales + t0 * (d32 / kActBlock);
    LaunchScope ls(kElementwise, double(rows) * d * (dt_size(dt) + 1.03125), st);
    if (dt == kF32)
      act8_unpack_kernel<float><<<grid, kThreads, 0, st>>>(
          codes, scales, ldx, d, total, fd, vec, static_cast<float*>(X) + t0 * ldx);
    else
      act8_unpack_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(
          codes, scales, ldx, d, total, fd, vec, static_cast<__nv_bfloat16*>(X) + t0 * ldx);
    SLORA_CHECK_LAUNCH();
  }
  return SLORA_OK;
}

int64_t act8_dot_part_floats(int64_t M, int64_t K, int cols) {
  const int64_t tiles = std::max<int64_t>((K + kDotCh - 1) / kDotCh, 1) * col_slices(cols);
  return tiles * dot_splits(M, K, cols) * kDotTile;
}
int64_t act8_dot_counters(int64_t K, int cols) {
  return std::max<int64_t>((K + kDotCh - 1) / kDotCh, 1) * col_slices(cols);
}

slora_status act8_dot(const Act8Dot& d, float* part, unsigned* counters, cudaStream_t st) {
  if (d.K <= 0 || d.cols <= 0) return SLORA_OK;
  DotParams p;
  p.codes = reinterpret_cast<const uint8_t*>(d.X.codes);
  p.scales = d.X.scales;
  p.ld = act8_cols(d.K);
  p.M = d.M; p.K = d.K;
  p.I64 = (std::max<int64_t>(d.M, 1) + 63) / 64 * 64;
  p.P = static_cast<const __nv_bfloat16*>(d.P);
  p.cp = (d.cols + 15) / 16 * 16;
  p.cols = d.cols;
  p.nsplit = dot_splits(d.M, d.K, d.cols);
  const int64_t steps = std::max<int64_t>((d.M + kDotStep - 1) / kDotStep, 1);
  p.steps = (steps + p.nsplit - 1) / p.nsplit;
  p.part = part;
  p.counters = counters;
  p.out = d.out; p.ldo = d.ldo; p.kmap = d.kmap; p.scale = d.scale; p.accumulate = d.accumulate;
  SLORA_CUDA(cudaFuncSetAttribute(act8_dot_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  kDotSmem));
  const dim3 grid(unsigned((d.K + kDotCh - 1) / kDotCh), unsigned(p.nsplit),
                  unsigned(col_slices(d.cols)));
  LaunchScope ls(kSkinny, double(d.M) * p.ld * 1.03125 * col_slices(d.cols), st);
  act8_dot_kernel<<<grid, kDotWarps * 32, kDotSmem, st>>>(p);
  SLORA_CHECK_LAUNCH();
  return SLORA_OK;
}

}  // namespace slora
