// rmsnorm_bwd.cu -- the gated RMSNorm for training: the forward that writes its 8-bit checkpoint in the
// same pass, and the backward pass, from the activations or from their checkpoints.
//
//   y = x inv (1 + w) silu(z),  inv = (mean x^2 + eps)^{-1/2};   with t = dy (1 + w) silu(z):
//   dx = inv (t - x inv^2 mean(t x))        dz = dy x inv (1 + w) silu'(z)
//   dw = sum over rows of dy x inv silu(z)
// with sigma = 1 / (1 + e^-z), silu'(z) = sigma (1 + z (1 - sigma)).
//
// HBM-bound: dy, x, z in, dx, dz out, once each.  The layout is the forward's (rmsnorm.cu): dim / 8
// lanes share a row, both row sums (x^2 and t x) go through one shuffle sequence.  dw is summed per
// thread over its rows, then over the block through shared memory, and each block writes one partial
// row to the workspace; a second kernel adds the partial rows in order (no atomics: the same inputs
// give the same bits).  1,048,576 rows of 128 bf16: 223 us for 1.34 GB (6.0 TB/s, 92 % of a copy), the partial
// rows 5 us.  131,072 rows: the checkpointing forward 31 us, the backward pass from checkpoints 35 us, for
// 135 MB each; launch and first loads take 8 us of each.
#include "act8.cuh"

namespace gdn {
namespace {

// rows in flight per thread: three streams of 16 bytes each
template <typename T>
constexpr int rows_u() {
  return sizeof(T) == 2 ? 4 : 2;
}

template <typename T, int TPR>
__global__ void __launch_bounds__(256) rmsnorm_ckpt8_kernel(
    const T* x, const T* __restrict__ z, const float* __restrict__ w, float eps, int64_t rows,
    T* y, int8_t* __restrict__ xc, float* __restrict__ xs, int8_t* __restrict__ zc,
    float* __restrict__ zs) {
  constexpr int DIM = TPR * 8, PER = 256 / TPR, U = rows_u<T>();
  const int sub = threadIdx.x % TPR, rsub = threadIdx.x / TPR;
  float wv[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) wv[i] = 1.0f + __ldg(w + sub * 8 + i);
  const int64_t stride = (int64_t)gridDim.x * PER;
  for (int64_t rb = (int64_t)blockIdx.x * PER; rb < rows; rb += U * stride) {
    Raw8<T> xr[U], zr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = rb + u * stride + rsub;
      if (r < rows) {
        xr[u].load(x + r * DIM + sub * 8);
        zr[u].load(z + r * DIM + sub * 8);
      } else {
        xr[u].zero();
        zr[u].zero();
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = rb + u * stride + rsub;
      float xv[8], zv[8], ss = 0.0f;
      xr[u].to_float(xv);
      zr[u].to_float(zv);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(xv[i], xv[i], ss);
      uint32_t mx = act8::amax8(xr[u]), mz = act8::amax8(zr[u]);
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mz = max(mz, __shfl_xor_sync(0xffffffffu, mz, o));
      }
      if (r < rows) {
        const float inv = rsqrtf(ss * (1.0f / DIM) + eps);
        float yv[8], sx, ix, sz, iz;
#pragma unroll
        for (int i = 0; i < 8; ++i) yv[i] = xv[i] * inv * wv[i] * silu_fast(zv[i]);
        store8(y + r * DIM + sub * 8, yv);
        act8::scale_of(mx, sx, ix);
        act8::scale_of(mz, sz, iz);
        *reinterpret_cast<uint2*>(xc + r * DIM + sub * 8) = act8::pack8(xv, ix);
        *reinterpret_cast<uint2*>(zc + r * DIM + sub * 8) = act8::pack8(zv, iz);
        if (sub == 0) {
          xs[r] = sx;
          zs[r] = sz;
        }
      }
    }
  }
}

// One activation as it is kept: itself, or codes and one scale per row.
template <typename T, bool CK>
struct Kept {
  Raw8<T> raw;
  __device__ __forceinline__ void load(const void* p, const float*, int64_t r, int64_t at) {
    raw.load((const T*)p + at);
  }
  __device__ __forceinline__ void zero() { raw.zero(); }
  __device__ __forceinline__ void to_float(float (&f)[8]) const { raw.to_float(f); }
};
template <typename T>
struct Kept<T, true> {
  uint2 c;
  float sc;
  __device__ __forceinline__ void load(const void* p, const float* s, int64_t r, int64_t at) {
    c = *reinterpret_cast<const uint2*>((const int8_t*)p + at);
    sc = __ldg(s + r);
  }
  __device__ __forceinline__ void zero() {
    c = make_uint2(0u, 0u);
    sc = 0.0f;
  }
  __device__ __forceinline__ void to_float(float (&f)[8]) const {
    act8::unpack4(c.x, sc, f);
    act8::unpack4(c.y, sc, f + 4);
  }
};

// The first `rows` rows; dw's sums over them go to this block's partial row.
template <typename T, int TPR, bool CK>
__device__ __forceinline__ void bwd_rows(
    const T* __restrict__ dy, const void* __restrict__ x, const float* __restrict__ xs,
    const void* __restrict__ z, const float* __restrict__ zs, const float* __restrict__ w, float eps,
    int64_t rows, T* __restrict__ dx, T* __restrict__ dz, float* __restrict__ part) {
  constexpr int DIM = TPR * 8, PER = 256 / TPR, U = rows_u<T>();
  const int sub = threadIdx.x % TPR, rsub = threadIdx.x / TPR;
  float wv[8], dw[8] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) wv[i] = 1.0f + __ldg(w + sub * 8 + i);
  const int64_t stride = (int64_t)gridDim.x * PER;
  for (int64_t rb = (int64_t)blockIdx.x * PER; rb < rows; rb += U * stride) {
    Raw8<T> dr[U];
    Kept<T, CK> xr[U], zr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = rb + u * stride + rsub, at = r * DIM + sub * 8;
      if (r < rows) {
        dr[u].load(dy + at);
        xr[u].load(x, xs, r, at);
        zr[u].load(z, zs, r, at);
      } else {
        dr[u].zero();
        xr[u].zero();
        zr[u].zero();
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = rb + u * stride + rsub;
      float d[8], xv[8], zv[8], t[8], ss = 0.0f, tx = 0.0f;
      dr[u].to_float(d);
      xr[u].to_float(xv);
      zr[u].to_float(zv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float sg = __fdividef(1.0f, 1.0f + __expf(-zv[i]));
        const float si = zv[i] * sg;
        t[i] = d[i] * si;                                              // dy silu(z)
        d[i] = d[i] * wv[i] * sg * fmaf(zv[i], 1.0f - sg, 1.0f);       // dy (1 + w) silu'(z)
        ss = fmaf(xv[i], xv[i], ss);
        tx = fmaf(t[i] * wv[i], xv[i], tx);
      }
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        tx += __shfl_xor_sync(0xffffffffu, tx, o);
      }
      if (r < rows) {
        const float inv = rsqrtf(ss * (1.0f / DIM) + eps);
        const float c = inv * inv * tx * (1.0f / DIM);
        float ox[8], oz[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xn = xv[i] * inv;
          ox[i] = inv * fmaf(-xv[i], c, t[i] * wv[i]);
          oz[i] = d[i] * xn;
          dw[i] = fmaf(t[i], xn, dw[i]);
        }
        store8(dx + r * DIM + sub * 8, ox);
        store8(dz + r * DIM + sub * 8, oz);
      }
    }
  }
  __shared__ float sh[256 * 8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sh[rsub * DIM + sub * 8 + i] = dw[i];
  __syncthreads();
  for (int c = threadIdx.x; c < DIM; c += 256) {
    float acc = 0.0f;
    for (int q = 0; q < PER; ++q) acc += sh[q * DIM + c];
    part[(int64_t)blockIdx.x * DIM + c] = acc;
  }
}

// The rows of a range of tokens, `rpt` rows each.  The range moves the pointers: as bounds of the loop it cost bf16
// 216 registers for 125, one block an SM for two, and 27 of 244 us.
template <typename T, int TPR, bool CK>
__global__ void __launch_bounds__(256) rmsnorm_bwd_kernel(
    const T* __restrict__ dy, const void* __restrict__ x, const float* __restrict__ xs,
    const void* __restrict__ z, const float* __restrict__ zs, const float* __restrict__ w, float eps,
    TokRange range, int64_t rpt, int64_t n_tok, T* __restrict__ dx, T* __restrict__ dz,
    float* __restrict__ part) {
  int64_t beg, end;
  tok_range(range, n_tok, beg, end);
  const int64_t row = beg * rpt, at = row * (TPR * 8), kept = at * (CK ? 1 : sizeof(T));
  bwd_rows<T, TPR, CK>(dy + at, (const unsigned char*)x + kept, CK ? xs + row : nullptr,
                       (const unsigned char*)z + kept, CK ? zs + row : nullptr, w, eps, (end - beg) * rpt,
                       dx + at, dz + at, part);
}

template <typename K>
int64_t wave_cap(K kern) {
  int dev = 0, sms = 148, per = 1;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, 256, 0);
  return (int64_t)sms * (per > 0 ? per : 1);
}

template <typename T>
cudaError_t ckpt_t(const T* x, const T* z, const float* w, float eps, int64_t rows, int dim, T* y,
                   int8_t* xc, float* xs, int8_t* zc, float* zs, cudaStream_t s) {
  const int tpr = dim / 8;
  const int64_t per = 256 / tpr * rows_u<T>();
  auto run = [&](auto kern) {
    const int64_t need = (rows + per - 1) / per, cap = wave_cap(kern);
    kern<<<(unsigned)(need < cap ? need : cap), 256, 0, s>>>(x, z, w, eps, rows, y, xc, xs, zc, zs);
  };
  switch (tpr) {
    case 1: run(rmsnorm_ckpt8_kernel<T, 1>); break;
    case 2: run(rmsnorm_ckpt8_kernel<T, 2>); break;
    case 4: run(rmsnorm_ckpt8_kernel<T, 4>); break;
    case 8: run(rmsnorm_ckpt8_kernel<T, 8>); break;
    case 16: run(rmsnorm_ckpt8_kernel<T, 16>); break;
    case 32: run(rmsnorm_ckpt8_kernel<T, 32>); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

template <typename T, bool CK>
cudaError_t bwd_t(const T* dy, const void* x, const float* xs, const void* z, const float* zs,
                  const float* w, float eps, TokRange range, int64_t rpt, int64_t rows, int dim, T* dx,
                  T* dz, float* dw, float* part, int64_t max_parts, cudaStream_t s) {
  const int tpr = dim / 8;
  const int64_t per = 256 / tpr * rows_u<T>();
  int64_t blocks = 0;
  auto run = [&](auto kern) {
    const int64_t cap = wave_cap(kern);
    blocks = (rows + per - 1) / per;
    blocks = blocks < cap ? blocks : cap;
    blocks = blocks < max_parts ? blocks : max_parts;
    if (blocks > 0)
      kern<<<(unsigned)blocks, 256, 0, s>>>(dy, x, xs, z, zs, w, eps, range, rpt, rows / rpt, dx, dz, part);
  };
  switch (tpr) {
    case 1: run(rmsnorm_bwd_kernel<T, 1, CK>); break;
    case 2: run(rmsnorm_bwd_kernel<T, 2, CK>); break;
    case 4: run(rmsnorm_bwd_kernel<T, 4, CK>); break;
    case 8: run(rmsnorm_bwd_kernel<T, 8, CK>); break;
    case 16: run(rmsnorm_bwd_kernel<T, 16, CK>); break;
    case 32: run(rmsnorm_bwd_kernel<T, 32, CK>); break;
    default: return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_sum_parts(part, blocks, dim, dim, dw, nullptr, dim, s);
  return e;
}

}  // namespace

cudaError_t launch_rmsnorm_ckpt8(const void* x, const void* z, gdn_dtype dt, const float* w,
                                 float eps, int64_t rows, int dim, void* y, int8_t* xc, float* xs,
                                 int8_t* zc, float* zs, cudaStream_t s) {
  if (dt == GDN_BF16)
    return ckpt_t((const __nv_bfloat16*)x, (const __nv_bfloat16*)z, w, eps, rows, dim,
                  (__nv_bfloat16*)y, xc, xs, zc, zs, s);
  return ckpt_t((const float*)x, (const float*)z, w, eps, rows, dim, (float*)y, xc, xs, zc, zs, s);
}

cudaError_t launch_rmsnorm_bwd(const void* dy, const void* x, const float* xs, const void* z,
                               const float* zs, gdn_dtype dt, const float* w, float eps, TokRange range,
                               int64_t rpt, int64_t rows, int dim, void* dx, void* dz, float* dw,
                               float* part, int64_t max_parts, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (dt == GDN_BF16)
    return xs ? bwd_t<B, true>((const B*)dy, x, xs, z, zs, w, eps, range, rpt, rows, dim, (B*)dx, (B*)dz,
                               dw, part, max_parts, s)
              : bwd_t<B, false>((const B*)dy, x, xs, z, zs, w, eps, range, rpt, rows, dim, (B*)dx, (B*)dz,
                                dw, part, max_parts, s);
  return xs ? bwd_t<float, true>((const float*)dy, x, xs, z, zs, w, eps, range, rpt, rows, dim, (float*)dx,
                                 (float*)dz, dw, part, max_parts, s)
            : bwd_t<float, false>((const float*)dy, x, xs, z, zs, w, eps, range, rpt, rows, dim, (float*)dx,
                                  (float*)dz, dw, part, max_parts, s);
}

}  // namespace gdn
