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

// max |x| of 8 raw values as the bits of its magnitude (integer order equals magnitude order, infinities
// and NaNs above every finite value).  bf16: the magnitudes of two values per word compared as two
// 16-bit integers at once, then moved to the upper half, where they are fp32 bits.
__device__ __forceinline__ uint32_t amax8(const Raw8<__nv_bfloat16>& r) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t w = __vmaxu2(__vmaxu2(r.u.x & m, r.u.y & m), __vmaxu2(r.u.z & m, r.u.w & m));
  return max(w << 16, w & 0xffff0000u);
}
__device__ __forceinline__ uint32_t amax8(const Raw8<float>& r) {
  const uint32_t m = 0x7fffffffu;
  const uint32_t a = max(max(__float_as_uint(r.a.x) & m, __float_as_uint(r.a.y) & m),
                         max(__float_as_uint(r.a.z) & m, __float_as_uint(r.a.w) & m));
  const uint32_t b = max(max(__float_as_uint(r.b.x) & m, __float_as_uint(r.b.y) & m),
                         max(__float_as_uint(r.b.z) & m, __float_as_uint(r.b.w) & m));
  return max(a, b);
}

// the group's scale and the factor its values are multiplied with
__device__ __forceinline__ void scale_of(uint32_t amax_bits, float& scale, float& inv) {
  const float m = __uint_as_float(amax_bits);
  scale = __fdiv_rn(m, 127.0f);
  inv = __fdiv_rn(127.0f, m);
  if (amax_bits >= 0x7f800000u) {
    scale = __uint_as_float(0x7fc00000u);
    inv = 0.0f;
  } else if (m < 7.888609e-31f) {  // 2^-100
    scale = 0.0f;
    inv = 0.0f;
  }
}

__device__ __forceinline__ uint32_t code(float x, float inv) {  // in the lowest byte
  return __float_as_uint(fmaf(x, inv, 12582912.0f));
}

// 8 codes, lowest channel in the lowest byte; zeros where inv is (0 * infinity is not taken)
__device__ __forceinline__ uint2 pack8(const float (&f)[8], float inv) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = code(f[i], inv);
  uint2 u;
  u.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  u.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
  return inv == 0.0f ? make_uint2(0u, 0u) : u;
}

__device__ __forceinline__ void unpack4(uint32_t u, float scale, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(u >> (8 * i)) * scale;
}

}  // namespace act8
}  // namespace gdn
