// act8.cuh -- 8-bit activation checkpoints: what the kernels that write and read them share.
//
// A group of consecutive channels with largest magnitude m holds codes rint(x * fl(127 / m)) in int8
// (the exact product, half to even) and one fp32 scale fl(m / 127); a code stands for code * scale.
// Symmetric int8 with its step set by the group's own maximum is off by at most half a step,
// m / 254, whatever the value's own size: for the roughly normal activations of the layer that is a
// quarter of what an 8-bit float with its 4 significant bits loses.  The product is rounded once: adding
// 1.5 * 2^23 inside one fused multiply-add puts the integer in the low bits of the sum, so the codes
// are the same on every machine.
// m below 2^-100 counts as zero (127 / m would overflow); a group that holds an infinity or a NaN gets
// a NaN scale, so every value read back from it is NaN.
#pragma once

#include "gdn_internal.cuh"

namespace gdn {
namespace act8 {

// max |x| of 8 values as the bits of its magnitude (integer order equals magnitude order, infinities
// and NaNs above every finite value)
__device__ __forceinline__ uint32_t amax8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  return m;
}

// the group's scale and the factor its values are multiplied with
__device__ __forceinline__ void scale_of(uint32_t amax_bits, float& scale, float& inv) {
  const float m = __uint_as_float(amax_bits);
  if (amax_bits >= 0x7f800000u) {
    scale = __uint_as_float(0x7fc00000u);
    inv = 0.0f;
  } else if (m < 7.888609e-31f) {  // 2^-100
    scale = 0.0f;
    inv = 0.0f;
  } else {
    scale = __fdiv_rn(m, 127.0f);
    inv = __fdiv_rn(127.0f, m);
  }
}

__device__ __forceinline__ uint32_t code(float x, float inv) {
  return __float_as_uint(fmaf(x, inv, 12582912.0f)) & 0xffu;
}

// 8 codes, lowest channel in the lowest byte; zeros where inv is (0 * infinity is not taken)
__device__ __forceinline__ uint2 pack8(const float (&f)[8], float inv) {
  if (inv == 0.0f) return make_uint2(0u, 0u);
  uint2 u;
  u.x = code(f[0], inv) | code(f[1], inv) << 8 | code(f[2], inv) << 16 | code(f[3], inv) << 24;
  u.y = code(f[4], inv) | code(f[5], inv) << 8 | code(f[6], inv) << 16 | code(f[7], inv) << 24;
  return u;
}

__device__ __forceinline__ void unpack4(uint32_t u, float scale, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(u >> (8 * i)) * scale;
}

}  // namespace act8
}  // namespace gdn
