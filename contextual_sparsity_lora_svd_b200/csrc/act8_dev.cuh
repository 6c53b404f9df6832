// Device helpers of the 8-bit checkpoints (format: slora.h): a block of 32
// channels shares the step 2^(byte - 133).
#pragma once

#include "common.cuh"

namespace slora {

// Scale byte of a block from the bits of its largest |x| (fp32, sign cleared):
// the exponent field, at least 7 so that the step stays a normal number; 255
// for an infinity or a NaN.
__device__ __forceinline__ uint32_t act8_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e < 7u ? 7u : e;
}
// 2^(133 - byte), the reciprocal of the step: a normal fp32 number for every
// byte in 7 .. 254.
__device__ __forceinline__ float act8_inv_step(uint32_t byte) {
  return __uint_as_float((260u - byte) << 23);
}
__device__ __forceinline__ float act8_step(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float((byte - 6u) << 23);
}
// The product with a power of two is exact, so this is the one rounding of a
// value (to nearest, ties to even); 127.5 steps and more saturate at 127.
__device__ __forceinline__ uint32_t act8_code(float x, float inv_step) {
  const int q = __float2int_rn(fminf(fmaxf(x * inv_step, -127.0f), 127.0f));
  return uint32_t(q) & 255u;
}
// Largest bits over the four lanes that hold one block's 8-channel chunks.
__device__ __forceinline__ uint32_t act8_block_max(uint32_t v) {
  v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return max(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ uint32_t act8_chunk_bits(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ uint2 act8_codes8(const float (&f)[8], uint32_t byte) {
  if (byte == 255u) return make_uint2(0x01010101u, 0x01010101u);  // NaN times a nonzero code
  const float inv = act8_inv_step(byte);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = act8_code(f[i], inv);
  return make_uint2(c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24),
                    c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24));
}
__device__ __forceinline__ void act8_values8(uint2 c, uint32_t byte, float (&f)[8]) {
  const float step = act8_step(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = i < 4 ? c.x : c.y;
    f[i] = float(int(w << (24 - 8 * (i & 3))) >> 24) * step;
  }
}

}  // namespace slora
