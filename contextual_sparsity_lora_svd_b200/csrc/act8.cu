// Activation checkpoints in 8 bits: packing and unpacking.
//
// Format (slora.h): blocks of 32 channels of a row share a power-of-two step,
// so dividing by it is exact, a code is one rounding of the value, and code *
// step is exact in bf16 (7 bits of magnitude).
//
// Packing and unpacking are bound by memory, 2 + 1 + 1/32 bytes a value in
// bf16.  A thread holds 8 channels (a 16-byte load, an 8-byte store), four
// neighbouring lanes share a block and its maximum (two shuffles), and each
// thread has four chunks in flight.  Packing and unpacking 8192 x 14336 bf16
// values, 710 MB in all, take 114 us, 6.2 TB/s, the rate of a plain copy of 590 MB.
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
  grid_wait();
  grid_ahead();
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
  grid_wait();
  grid_ahead();
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
      SLORA_CUDA(launch_early(act8_pack_kernel<float>, dim3(grid), kThreads, 0, st,
                              static_cast<const float*>(X) + t0 * ldx, ldx, d, total, fd, vec,
                              codes, scales));
    else
      SLORA_CUDA(launch_early(act8_pack_kernel<__nv_bfloat16>, dim3(grid), kThreads, 0, st,
                              static_cast<const __nv_bfloat16*>(X) + t0 * ldx, ldx, d, total, fd,
                              vec, codes, scales));
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
      SLORA_CUDA(launch_early(act8_unpack_kernel<float>, dim3(grid), kThreads, 0, st, codes, scales,
                              ldx, d, total, fd, vec, static_cast<float*>(X) + t0 * ldx));
    else
      SLORA_CUDA(launch_early(act8_unpack_kernel<__nv_bfloat16>, dim3(grid), kThreads, 0, st, codes,
                              scales, ldx, d, total, fd, vec,
                              static_cast<__nv_bfloat16*>(X) + t0 * ldx));
  }
  return SLORA_OK;
}

}  // namespace slora
