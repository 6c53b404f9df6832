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
__device__ __forceinline__ uint32_t act8_chunk_bits(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  return m;
}
// Largest bits over the four lanes that hold one block's 8-channel chunks.
__device__ __forceinline__ uint32_t act8_block_max(uint32_t v) {
  v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return max(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
// Codes of 8 values of a block: clamped to +-127 steps, scaled (exact) and
// rounded to nearest even by the addition of 1.5 * 2^23, whose low byte is then
// the code in two's complement; one instruction for the product and the
// rounding.  A block of NaNs gets nonzero codes.
__device__ __forceinline__ uint2 act8_codes8(const float (&f)[8], uint32_t byte) {
  const float inv = act8_inv_step(byte);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __float_as_uint(fmaf(f[i], inv, 12582912.0f));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __byte_perm(c[2 * i], c[2 * i + 1], 0x0040);
  const uint2 r = make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
  return byte == 255u ? make_uint2(0x01010101u, 0x01010101u) : r;
}
__device__ __forceinline__ uint2 act8_codes8_f32(float (&f)[8], uint32_t byte) {
  const float top = 127.0f * act8_step(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = fminf(fmaxf(f[i], -top), top);
  return act8_codes8(f, byte);
}
// The same from 8 packed bf16 values: the maximum and the clamp (127 steps are
// exact in bf16) on pairs.
__device__ __forceinline__ void act8_unpack_bf16(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ __nv_bfloat162 act8_as_bf162(uint32_t w) {
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}
// Scale byte of the 32-channel block whose four chunks neighbouring lanes hold.
__device__ __forceinline__ uint32_t act8_byte_bf16(const uint4& u) {
  __nv_bfloat162 m = __hmax2_nan(
      __hmax2_nan(__habs2(act8_as_bf162(u.x)), __habs2(act8_as_bf162(u.y))),
      __hmax2_nan(__habs2(act8_as_bf162(u.z)), __habs2(act8_as_bf162(u.w))));
  m = __hmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = __hmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
  return max(max(w >> 23, (w >> 7) & 255u), 7u);
}
__device__ __forceinline__ uint2 act8_codes8_bf16(uint4 u, uint32_t byte) {
  const uint32_t top = __float_as_uint(127.0f * act8_step(byte)) >> 16;
  const __nv_bfloat162 hi = act8_as_bf162(top | (top << 16));
  const __nv_bfloat162 lo = __hneg2(hi);
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __hmin2(__hmax2(act8_as_bf162(w[i]), lo), hi);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  float f[8];
  act8_unpack_bf16(u, f);
  return act8_codes8(f, byte);
}
// Values of 8 codes: each byte, with its sign bit flipped, under the exponent
// of 2^23 is 2^23 + 128 + code.
__device__ __forceinline__ void act8_values8(uint2 c, uint32_t byte, float (&f)[8]) {
  const float step = act8_step(byte);
  const uint32_t x = c.x ^ 0x80808080u, y = c.y ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __byte_perm(i < 4 ? x : y, 0x4b000000u, 0x7440 | (i & 3));
    f[i] = (__uint_as_float(b) - 8388736.0f) * step;
  }
}

}  // namespace slora
