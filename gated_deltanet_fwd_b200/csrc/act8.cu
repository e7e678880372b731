// act8.cu -- 8-bit activation checkpoints: writing (pack) and reading back (unpack).  The format and
// why it was taken are in act8.cuh.
//
// HBM-bound: pack reads an activation and writes one byte (and 4 / group bytes of scale) for it, unpack
// the reverse.  group / 8 lanes share a group (8 elements = one 16-byte bf16 load and one 8-byte code
// store each), the maximum is a shuffle reduction, and each thread keeps ACT_U groups in flight.
// 16384 rows of 8192 bf16 in groups of 128: pack 75 us, unpack 66 us for 407 MB each (5.4 and 6.2 TB/s; a
// copy reaches 6.55).
#include "act8.cuh"

namespace gdn {
namespace {

constexpr int ACT_U = 4;

template <typename T, int TPG>
__global__ void __launch_bounds__(256) act_pack8_kernel(const T* __restrict__ x, int64_t groups,
                                                        int8_t* __restrict__ codes,
                                                        float* __restrict__ scales) {
  constexpr int GROUP = TPG * 8, PER = 256 / TPG;
  const int sub = threadIdx.x % TPG, gsub = threadIdx.x / TPG;
  const int64_t stride = (int64_t)gridDim.x * PER;
  for (int64_t gb = (int64_t)blockIdx.x * PER; gb < groups; gb += ACT_U * stride) {
    Raw8<T> raw[ACT_U];
#pragma unroll
    for (int u = 0; u < ACT_U; ++u) {
      const int64_t g = gb + u * stride + gsub;
      if (g < groups)
        raw[u].load(x + g * GROUP + sub * 8);
      else
        raw[u].zero();
    }
#pragma unroll
    for (int u = 0; u < ACT_U; ++u) {
      const int64_t g = gb + u * stride + gsub;
      uint32_t m = act8::amax8(raw[u]);
#pragma unroll
      for (int o = TPG / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (g < groups) {
        float f[8], sc, inv;
        raw[u].to_float(f);
        act8::scale_of(m, sc, inv);
        *reinterpret_cast<uint2*>(codes + g * GROUP + sub * 8) = act8::pack8(f, inv);
        if (sub == 0) scales[g] = sc;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) act_unpack8_kernel(const int8_t* __restrict__ codes,
                                                          const float* __restrict__ scales,
                                                          int64_t n8, int shift,
                                                          T* __restrict__ x) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t b = (int64_t)blockIdx.x * 256 + threadIdx.x; b < n8; b += ACT_U * stride) {
    uint2 c[ACT_U];
    float sc[ACT_U];
#pragma unroll
    for (int u = 0; u < ACT_U; ++u) {
      const int64_t i = b + u * stride;
      if (i < n8) {
        c[u] = reinterpret_cast<const uint2*>(codes)[i];
        sc[u] = __ldg(scales + (i >> shift));
      }
    }
#pragma unroll
    for (int u = 0; u < ACT_U; ++u) {
      const int64_t i = b + u * stride;
      if (i < n8) {
        float f[8];
        act8::unpack4(c[u].x, sc[u], f);
        act8::unpack4(c[u].y, sc[u], f + 4);
        store8(x + i * 8, f);
      }
    }
  }
}

// blocks for `work` thread-block passes: at most one wave of resident blocks
template <typename K>
unsigned wave(K kern, int64_t work) {
  int dev = 0, sms = 148, per = 1;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, 256, 0);
  const int64_t cap = (int64_t)sms * (per > 0 ? per : 1);
  return (unsigned)(work < 1 ? 1 : work < cap ? work : cap);
}

template <typename T>
cudaError_t pack_t(const T* x, int64_t groups, int group, int8_t* codes, float* scales,
                   cudaStream_t s) {
  const int tpg = group / 8;
  const int64_t work = (groups * tpg + 256 * ACT_U - 1) / (256 * ACT_U);
  switch (tpg) {
#define GDN_CASE(N)                                                                         \
  case N:                                                                                   \
    act_pack8_kernel<T, N><<<wave(act_pack8_kernel<T, N>, work), 256, 0, s>>>(x, groups, codes, \
                                                                              scales);      \
    break;
    GDN_CASE(1)
    GDN_CASE(2)
    GDN_CASE(4)
    GDN_CASE(8)
    GDN_CASE(16)
    GDN_CASE(32)
#undef GDN_CASE
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t unpack_t(const int8_t* codes, const float* scales, int64_t groups, int group, T* x,
                     cudaStream_t s) {
  int shift = 0;
  while ((8 << shift) < group) ++shift;
  const int64_t n8 = groups * (group / 8), work = (n8 + 256 * ACT_U - 1) / (256 * ACT_U);
  act_unpack8_kernel<T><<<wave(act_unpack8_kernel<T>, work), 256, 0, s>>>(codes, scales, n8, shift,
                                                                          x);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_act_pack8(const void* x, gdn_dtype dt, int64_t groups, int group, int8_t* codes,
                             float* scales, cudaStream_t s) {
  return dt == GDN_BF16 ? pack_t((const __nv_bfloat16*)x, groups, group, codes, scales, s)
                        : pack_t((const float*)x, groups, group, codes, scales, s);
}

cudaError_t launch_act_unpack8(const int8_t* codes, const float* scales, gdn_dtype dt,
                               int64_t groups, int group, void* x, cudaStream_t s) {
  return dt == GDN_BF16 ? unpack_t(codes, scales, groups, group, (__nv_bfloat16*)x, s)
                        : unpack_t(codes, scales, groups, group, (float*)x, s);
}

}  // namespace gdn
