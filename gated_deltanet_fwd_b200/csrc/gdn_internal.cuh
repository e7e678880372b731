// gdn_internal.cuh -- helpers shared by the libgdn kernels (device side) and the launchers'
// internal declarations.  Nothing here is exported.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

// ---------------------------------------------------------------- element I/O -------------
// Activations are bf16 or fp32; math is fp32.  Loads of 8 consecutive elements are one 16-byte
// transaction for bf16 and two for fp32.

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// 8 consecutive elements <-> 8 floats.  `p` must be 16-byte aligned.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  uint4 u = *reinterpret_cast<const uint4*>(p);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 t = __bfloat1622float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  float4 a = reinterpret_cast<const float4*>(p)[0];
  float4 b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = u;
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Raw (still encoded) 8-element vectors, so loads can be issued early without holding 8 floats.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void to_float(float (&f)[8]) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 t = __bfloat1622float2(h[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void to_float(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

// 4 consecutive elements -> 4 floats (8-byte bf16 load or one float4).
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&f)[4]) {
  uint2 u = *reinterpret_cast<const uint2*>(p);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
  float2 a = __bfloat1622float2(h[0]), b = __bfloat1622float2(h[1]);
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}
__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
  float4 a = *reinterpret_cast<const float4*>(p);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
}

__device__ __forceinline__ float sigmoidf_(float x) { return 1.0f / (1.0f + expf(-x)); }
__device__ __forceinline__ float siluf_(float x) { return x / (1.0f + expf(-x)); }
// SiLU for kernels whose result is rounded to bf16: the fast exponential and division intrinsics
// (relative error ~1e-6, far below bf16's 2^-8) keep these HBM-bound kernels off the ALU roof.
// For x < -87 the exponential overflows to +inf and the quotient is the correct limit, -0.
__device__ __forceinline__ float silu_fast(float x) { return __fdividef(x, 1.0f + __expf(-x)); }
__device__ __forceinline__ float softplusf_(float x) {
  return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x)));
}

// The log-decay that the chunked kernels add up.  e^-256 is zero in fp32 and in every product, and so is every decay
// across such a token; but a sum that passes a larger magnitude (a state reset by -1e9 or -infinity) has lost
// the differences between the tokens behind it.  NaN stays NaN.
__device__ __forceinline__ float floor_decay(float g) { return g < -256.0f ? -256.0f : g; }

// Device-side fault reporting: the first error wins; never traps.
__device__ __forceinline__ void report(int* status, int code) {
  if (status) atomicCAS(status, 0, code);
}

// Sequence lookup for packed (varlen) token streams.  Returns the sequence that owns token t
// (cu[n] <= t < cu[n+1]); with cu == nullptr sequence n is batch row t / T.
__device__ __forceinline__ int seq_of_token(const int32_t* cu, int N, int64_t T, int64_t t) {
  if (!cu) return (int)(t / T);
  int lo = 0, hi = N - 1;  // last n with cu[n] <= t
  while (lo < hi) {
    int mid = (lo + hi + 1) >> 1;
    if ((int64_t)cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ---------------------------------------------------------------- launchers ---------------
// Each returns cudaSuccess or the launch error; arguments were validated by the caller.

cudaError_t launch_gates(const void* a, const void* b, gdn_dtype dt, const float* A_log,
                         const float* dt_bias, int64_t n_tok, int Hv, float* g, float* beta,
                         cudaStream_t s);

cudaError_t launch_conv(const void* x, gdn_dtype dt, const float* w, const float* bias, int B,
                        int64_t T, int C, int K, const int32_t* cu, int N, int n_l2, int group,
                        float l2_eps, const float* cs_in, float* cs_out, void* y,
                        cudaStream_t s);

cudaError_t launch_rmsnorm(const void* x, const void* z, gdn_dtype dt, const float* w, float eps,
                           int64_t rows, int dim, void* y, cudaStream_t s);

cudaError_t launch_recurrent(const void* q, const void* k, const void* v, const float* g,
                             const float* beta, gdn_dtype dt, float scale, float* state, int N,
                             int Hk, int Hv, int dk, int dv, void* out, cudaStream_t s);

cudaError_t launch_decode_fused(const void* mix, const void* a, const void* b, const void* z,
                                gdn_dtype dt, const float* conv_w, const float* conv_bias, int K,
                                const float* cs_in, float* cs_out, const float* A_log,
                                const float* dt_bias, const float* norm_w, float l2_eps,
                                float norm_eps, float scale, float* state, int N, int Hk, int Hv,
                                void* y, cudaStream_t s);

// ---- training: backward passes and 8-bit activation checkpoints.  `part` holds up to max_parts partial
// rows of the sums over tokens.

// Allows a kernel `bytes` of dynamic shared memory on the current device.  Asked at every launch (60 ns): the
// setting belongs to the device's context, and a process may use several devices, or reset one.
template <typename Kernel>
inline cudaError_t allow_smem(Kernel* kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}
inline cudaError_t sm_count(int& sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
}

// With cu set only the tokens of [cu[0], cu[N]) take part, clamped to the tensor.
struct TokRange {
  const int32_t* cu;
  int N;
};
__device__ __forceinline__ void tok_range(const TokRange& r, int64_t n_tok, int64_t& beg, int64_t& end) {
  beg = 0;
  end = n_tok;
  if (r.cu) {
    beg = max((int64_t)0, min((int64_t)r.cu[0], n_tok));
    end = max(beg, min((int64_t)r.cu[r.N], n_tok));
  }
}

cudaError_t launch_gates_bwd(const void* a, const void* b, gdn_dtype dt, const float* A_log,
                             const float* dt_bias, const void* dg, const void* dbeta, TokRange range,
                             int64_t n_tok, int Hv, void* da, void* db, float* dA, float* ddt,
                             float* part, int64_t max_parts, cudaStream_t s);

cudaError_t launch_rmsnorm_ckpt8(const void* x, const void* z, gdn_dtype dt, const float* w,
                                 float eps, int64_t rows, int dim, void* y, int8_t* xc, float* xs,
                                 int8_t* zc, float* zs, cudaStream_t s);

// xs, zs set: x and z are int8 codes with one scale per row.  A token of the range is `rpt` rows.
cudaError_t launch_rmsnorm_bwd(const void* dy, const void* x, const float* xs, const void* z,
                               const float* zs, gdn_dtype dt, const float* w, float eps, TokRange range,
                               int64_t rpt, int64_t rows, int dim, void* dx, void* dz, float* dw, float* part,
                               int64_t max_parts, cudaStream_t s);

struct ConvBwdArgs {
  const void* dy;
  const void* x;        // of dtype, or int8 codes when xs is set
  const float* xs;      // [tokens, C / xgroup] or null
  int xgroup, xgroups;  // channels of a scale, scales of a token
  const float *w, *bias;
  int64_t n_tok, T;
  int C, K, N, n_l2, group;
  const int32_t* cu;
  float eps;
  const float *cs_in, *dcs_out;
  void* dx;
  float *dw, *dbias, *dcs_in;
  float* part;          // [ranges][C * K + C]
  int64_t max_parts;
};
cudaError_t launch_conv_bwd(const ConvBwdArgs& a, gdn_dtype dt, cudaStream_t s);

cudaError_t launch_act_pack8(const void* x, gdn_dtype dt, int64_t groups, int group, int8_t* codes,
                             float* scales, cudaStream_t s);
cudaError_t launch_act_unpack8(const int8_t* codes, const float* scales, gdn_dtype dt,
                               int64_t groups, int group, void* x, cudaStream_t s);

// The first `width` columns of `parts` partial rows (`stride` apart) added in row order: column c to
// out[c] below `split`, to out2[c - split] from there on.
cudaError_t launch_sum_parts(const float* part, int64_t parts, int64_t width, int64_t split,
                             float* out, float* out2, int64_t stride, cudaStream_t s);

// Element distances between consecutive tokens of q, k and v (dense: Hk*dk, Hk*dk, Hv*dv).
struct TokStrides {
  int64_t q, k, v;
};

// CUDA-core chunk path (any supported shape / dtype).
cudaError_t launch_chunk_simt(const void* q, const void* k, const void* v, TokStrides ts,
                              const float* g,
                              const float* beta, gdn_dtype dt, float scale, const float* S0,
                              const int32_t* cu, int N, int B, int64_t T, int Hk, int Hv, int dk,
                              int dv, int chunk, void* out, float* S_T, int* status,
                              cudaStream_t s);

// Optional fusions of the layer's neighbouring steps into the two-kernel tensor-core prefill: the
// gates computed from their pre-activations inside the prep kernel (a, b set), and the gated
// RMSNorm applied to the outputs in the chain's output epilogue (z set; `out` then receives y).
struct ChunkFusion {
  const __nv_bfloat16* a = nullptr;  // [tokens, Hv] gate pre-activations (fused gates when set)
  const __nv_bfloat16* b = nullptr;
  const float* A_log = nullptr;
  const float* dt_bias = nullptr;
  // set: the backward pass's operands, its records and its scale Gamma Q tiles at these byte offsets
  size_t bwd_gd_off = 0, bwd_qg_off = 0;
  const CUtensorMap *bwd_k = nullptr, *bwd_q = nullptr;
  float scale = 0.0f;
};

// TMA tensor maps (tma_maps.cu), 128-byte swizzle, bf16:
//   make_tok_map:    [rows, heads, 128] with `tok_stride` elements between rows; box {64, 1, 64}
//   make_rows64_map: [rows, 64] dense;                                          box {64, box_rows}
bool make_tok_map(CUtensorMap* m, const void* base, int heads, int64_t rows, int64_t tok_stride);
bool make_rows64_map(CUtensorMap* m, const void* base, int64_t rows, uint32_t box_rows);

// Two-kernel tensor-core prefill (bf16, dk = dv = 128, chunk = 64): the parallel prep kernel,
// then the chain kernel.  `ws` holds at least tm::workspace_bytes(N, B*T, Hv) bytes.
cudaError_t launch_chunk_prep(const void* q, const void* k, TokStrides ts, const float* g,
                              const float* beta, const int32_t* cu, int N, int B, int64_t T,
                              int Hk, int Hv, void* ws, int* status, cudaStream_t s,
                              const ChunkFusion& fuse = ChunkFusion());
// phase 0: one chain per (sequence, v-head); phases 1 and 3 (with launch_scan_prefix between
// them): the intra-sequence scan with segments of lseg tokens (chunk_tm.cuh), for which `ws` holds
// at least tm::workspace_bytes_scan(N, B*T, Hv, lseg) bytes.
cudaError_t launch_chunk_chain(const void* q, const void* k, const void* v, TokStrides ts,
                               float scale, const float* S0, const int32_t* cu, int N, int B,
                               int64_t T, int Hk, int Hv, void* out, float* S_T, void* ws,
                               int phase, int64_t lseg, int* status, cudaStream_t s);
// One-thread planner: writes the call's segment length (0, lseg, 2 lseg or 4 lseg) into the
// workspace for the two chain phases and the prefix to read.
cudaError_t launch_scan_plan(const int32_t* cu, int N, int B, int64_t T, int Hv, int sms,
                             int64_t lseg, void* ws, int* status, cudaStream_t s);
cudaError_t launch_scan_prefix(const int32_t* cu, int N, int B, int64_t T, int Hv, int64_t lseg,
                               void* ws, int* status, cudaStream_t s);

// Tensor-core chunk path without scratch (one CTA pair per sequence and head): bf16,
// dk = dv = 128, chunk = 64.
cudaError_t launch_chunk_tc(const void* q, const void* k, const void* v, TokStrides ts,
                            const float* g,
                            const float* beta, float scale, const float* S0, const int32_t* cu,
                            int N, int B, int64_t T, int Hk, int Hv, void* out, float* S_T,
                            int* status, cudaStream_t s);

}  // namespace gdn
