// conv_bwd.cu -- gradients of the causal conv + SiLU + q/k L2 norm (conv.cu), from the conv's input or
// from its 8-bit checkpoint.
//
//   pre[t] = bias + sum_i w[i] x[t-(K-1)+i],  act = pre sigma(pre),  y = act rn,
//   rn = (sum_group act^2 + eps)^{-1/2}     (1 for channels that are not normalised)
//   dact = rn (dy - act rn^2 sum_group(act dy)),  dpre = dact sigma (1 + pre (1 - sigma))
//   dx[t] = sum_i w[i] dpre[t+(K-1)-i],  dw[i] = sum_t dpre[t] x[t-(K-1)+i],  dbias = sum_t dpre[t]
// An input in front of its sequence is conv_state_in; its gradient is the same sum at a negative place.
// conv_state_out is a copy of the last K-1 of (history, inputs), so dconv_state_out is added there.
//
// HBM-bound: dy and x in, dx out, once each (and K-1 tokens of halo at the ends of a token range).
// A thread holds 4 channels and streams a range of tokens forward: x[t-KT+1 .. t] and
// dpre[t-KT+1 .. t] are register windows, so each token is loaded and each dpre computed once; dx is
// stored KT-1 tokens late.  A warp spans 128 channels, so the norm's sums for groups up to 128 are
// shuffles; a group of 256 spans the block's two warps, which exchange their sums through shared memory.
// dw and dbias are summed in registers over the range; each range writes one partial row, added in
// order by a second kernel.  Kernels exist for 2, 4 and 8 taps; a smaller K has leading zero taps.
#include "act8.cuh"

namespace gdn {
namespace {

constexpr int CB_THREADS = 64;
constexpr int CB_CH = 4;  // channels per thread

template <typename T>
struct Raw4;
template <>
struct Raw4<__nv_bfloat16> {
  uint2 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = __ldg(reinterpret_cast<const uint2*>(p));
  }
  __device__ __forceinline__ void to_float(float (&f)[4]) const {
    f[0] = __uint_as_float(u.x << 16);
    f[1] = __uint_as_float(u.x & 0xffff0000u);
    f[2] = __uint_as_float(u.y << 16);
    f[3] = __uint_as_float(u.y & 0xffff0000u);
  }
};
template <>
struct Raw4<float> {
  float4 u;
  __device__ __forceinline__ void load(const float* p) {
    u = __ldg(reinterpret_cast<const float4*>(p));
  }
  __device__ __forceinline__ void to_float(float (&f)[4]) const {
    f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
  }
};

__device__ __forceinline__ void put4(__nv_bfloat16* p, const float (&f)[4]) {
  __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}
__device__ __forceinline__ void put4(float* p, const float (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}

// 4 channels of the conv's input: as they are, or codes and their group's scale
template <typename T, bool CK>
struct XIn {
  Raw4<T> r;
  __device__ __forceinline__ void load(const ConvBwdArgs& P, int64_t t, int c) {
    r.load((const T*)P.x + t * P.C + c);
  }
  __device__ __forceinline__ void to_float(float (&f)[4]) const { r.to_float(f); }
};
template <typename T>
struct XIn<T, true> {
  uint32_t u;
  float sc;
  __device__ __forceinline__ void load(const ConvBwdArgs& P, int64_t t, int c) {
    u = __ldg(reinterpret_cast<const uint32_t*>((const int8_t*)P.x + t * P.C + c));
    sc = __ldg(P.xs + t * (P.C / P.xgroup) + c / P.xgroup);
  }
  __device__ __forceinline__ void to_float(float (&f)[4]) const { act8::unpack4(u, sc, f); }
};

template <typename T, int KT, bool CK>
__global__ void __launch_bounds__(CB_THREADS) conv_bwd_kernel(const ConvBwdArgs P) {
  constexpr int D = KT - 1;                // tokens that dx lags behind
  constexpr int PF = KT == 8 ? 4 : 8;      // tokens loaded ahead
  __shared__ float2 ex[2][2];              // sums of a 256-channel group, two tokens in turn
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = blockIdx.x * (CB_THREADS * CB_CH) + tid * CB_CH;
  const bool on = c < P.C;
  const int K = P.K, pad = KT - K;
  const int64_t per = (P.n_tok + gridDim.y - 1) / gridDim.y;
  const int64_t r0 = (int64_t)blockIdx.y * per, r1 = min(r0 + per, P.n_tok);
  const bool norm = on && c < P.n_l2;
  const int gl = P.group / CB_CH;  // lanes of a group
  const bool any = P.n_l2 > (P.group > 128 ? blockIdx.x * (CB_THREADS * CB_CH) : c - lane * CB_CH);

  float w[KT][4], bias[4] = {}, dw[KT][4] = {}, db[4] = {};
#pragma unroll
  for (int i = 0; i < KT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[i][q] = on && i >= pad ? __ldg(P.w + (int64_t)(c + q) * K + i - pad) : 0.0f;
  if (on && P.bias)
#pragma unroll
    for (int q = 0; q < 4; ++q) bias[q] = __ldg(P.bias + c + q);

  auto bound = [&](int m, int64_t& b, int64_t& e) {  // sequence m's tokens, clamped to the tensor
    b = P.cu ? P.cu[m] : (int64_t)m * P.T;
    e = P.cu ? P.cu[m + 1] : b + P.T;
    b = max((int64_t)0, min(b, P.n_tok));
    e = max(b, min(e, P.n_tok));
  };
  if (blockIdx.y == 0 && P.dcs_in && on) {  // empty sequences: the history passes through
    for (int m = 0; m < P.N; ++m) {
      int64_t b, e;
      bound(m, b, e);
      if (e > b) continue;
      const int64_t at = ((int64_t)m * P.C + c) * (K - 1);
      for (int q = 0; q < 4 * (K - 1); ++q) P.dcs_in[at + q] = P.dcs_out ? P.dcs_out[at + q] : 0.0f;
    }
  }
  if (r0 < r1) {
    int n = seq_of_token(P.cu, P.N, P.T, r0);
    for (; n < P.N; ++n) {
      int64_t s_beg, s_end;
      bound(n, s_beg, s_end);
      if (s_beg >= r1) break;
      const int64_t a = max(r0, s_beg), e = min(r1, s_end);
      if (a >= e) continue;
      const int64_t te = min(e + D, s_end);
      const int64_t cs = ((int64_t)n * P.C + c) * (K - 1);
      float xw[KT][4], dp[KT][4] = {};  // x[t - d], dpre[t - d]
#pragma unroll
      for (int d = 1; d < KT; ++d) {
        const int64_t p = a - d;
#pragma unroll
        for (int q = 0; q < 4; ++q) xw[d - 1][q] = 0.0f;
        if (on && d < K) {
          if (p >= s_beg) {
            XIn<T, CK> xi;
            xi.load(P, p, c);
            xi.to_float(xw[d - 1]);
          } else if (P.cs_in) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              xw[d - 1][q] = __ldg(P.cs_in + cs + (int64_t)q * (K - 1) + (K - 1) + (p - s_beg));
          }
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) xw[KT - 1][q] = 0.0f;
      // the gradient of the input at place p (a token, or a place of the history) once dp[0] is dpre[p + D]
      auto emit = [&](int64_t p) {
        if (!on) return;
        float v[4] = {};
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = fmaf(w[i][q], dp[i][q], v[q]);
        const int64_t jo = p - (s_end - (K - 1));  // place in the history left behind
        if (P.dcs_out && jo >= 0 && jo < K - 1)
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] += __ldg(P.dcs_out + cs + (int64_t)q * (K - 1) + jo);
        if (p >= a) {
          if (p < e) put4((T*)P.dx + p * P.C + c, v);
        } else if (p < s_beg && a == s_beg && P.dcs_in) {
          const int64_t j = p - s_beg + (K - 1);
          if (j >= 0)
#pragma unroll
            for (int q = 0; q < 4; ++q) P.dcs_in[cs + (int64_t)q * (K - 1) + j] = v[q];
        }
      };
      auto shift = [&]() {
#pragma unroll
        for (int d = KT - 1; d > 0; --d)
#pragma unroll
          for (int q = 0; q < 4; ++q) dp[d][q] = dp[d - 1][q];
      };
      XIn<T, CK> xn[PF];
      Raw4<T> yn[PF];
      auto fetch = [&](int64_t t) {
#pragma unroll
        for (int u = 0; u < PF; ++u)
          if (on && t + u < te) {
            xn[u].load(P, t + u, c);
            yn[u].load((const T*)P.dy + (t + u) * P.C + c);
          }
      };
      fetch(a);
      for (int64_t tb = a; tb < te; tb += PF) {
        XIn<T, CK> xc[PF];
        Raw4<T> yc[PF];
#pragma unroll
        for (int u = 0; u < PF; ++u) {
          xc[u] = xn[u];
          yc[u] = yn[u];
        }
        fetch(tb + PF);
#pragma unroll
        for (int u = 0; u < PF; ++u) {
          const int64_t t = tb + u;
          if (t >= te) break;
#pragma unroll
          for (int d = KT - 1; d > 0; --d)
#pragma unroll
            for (int q = 0; q < 4; ++q) xw[d][q] = xw[d - 1][q];
          shift();
          float dyv[4] = {};
          if (on) {
            xc[u].to_float(xw[0]);
            yc[u].to_float(dyv);
          }
          float act[4], slope[4], ss = 0.0f, ad = 0.0f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float pre = bias[q];
#pragma unroll
            for (int d = 0; d < KT; ++d) pre = fmaf(w[KT - 1 - d][q], xw[d][q], pre);
            const float sg = __fdividef(1.0f, 1.0f + __expf(-pre));
            act[q] = pre * sg;
            slope[q] = sg * fmaf(pre, 1.0f - sg, 1.0f);
            ss = fmaf(act[q], act[q], ss);
            ad = fmaf(act[q], dyv[q], ad);
          }
          if (any) {
            for (int o = min(gl, 32) >> 1; o > 0; o >>= 1) {
              ss += __shfl_xor_sync(0xffffffffu, ss, o);
              ad += __shfl_xor_sync(0xffffffffu, ad, o);
            }
            if (gl == 64) {
              const int par = (int)(t & 1);
              if (lane == 0) ex[par][warp] = make_float2(ss, ad);
              __syncthreads();
              const float2 e0 = ex[par][0], e1 = ex[par][1];
              ss = e0.x + e1.x;
              ad = e0.y + e1.y;
            }
            if (norm) {
              const float rn = rsqrtf(ss + P.eps), f = rn * rn * ad;
#pragma unroll
              for (int q = 0; q < 4; ++q) dyv[q] = rn * fmaf(-act[q], f, dyv[q]);
            }
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) dp[0][q] = dyv[q] * slope[q];
          if (t < e) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              db[q] += dp[0][q];
#pragma unroll
              for (int d = 0; d < KT; ++d)
                dw[KT - 1 - d][q] = fmaf(dp[0][q], xw[d][q], dw[KT - 1 - d][q]);
            }
          }
          emit(t - D);
        }
      }
      if (te == s_end) {  // nothing follows the sequence
#pragma unroll 1
        for (int m = 1; m <= D; ++m) {
          shift();
#pragma unroll
          for (int q = 0; q < 4; ++q) dp[0][q] = 0.0f;
          emit(s_end - 1 + m - D);
        }
      }
      if (gl == 64 && any) __syncthreads();  // the exchange starts over on the next sequence
    }
  }
  if (on) {
    float* row = P.part + (int64_t)blockIdx.y * P.C * (K + 1);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
        if (i >= pad) row[(int64_t)(c + q) * K + i - pad] = dw[i][q];
      row[(int64_t)P.C * K + c + q] = db[q];
    }
  }
}

template <typename T, int KT, bool CK>
cudaError_t run(ConvBwdArgs a, cudaStream_t s) {
  int dev = 0, sms = 148, per_sm = 1;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, conv_bwd_kernel<T, KT, CK>, CB_THREADS, 0);
  const int64_t tiles = (a.C + CB_THREADS * CB_CH - 1) / (CB_THREADS * CB_CH);
  // one wave of blocks, with at least 16 tokens in a range (the halo costs up to KT - 1)
  int64_t ranges = (int64_t)sms * (per_sm > 0 ? per_sm : 1) / tiles;
  if (ranges > (a.n_tok + 15) / 16) ranges = (a.n_tok + 15) / 16;
  if (ranges > a.max_parts) ranges = a.max_parts;
  if (ranges < 1) ranges = 1;
  conv_bwd_kernel<T, KT, CK><<<dim3((unsigned)tiles, (unsigned)ranges), CB_THREADS, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t wk = (int64_t)a.C * a.K;
  return launch_sum_parts(a.part, ranges, a.dbias ? wk + a.C : wk, wk, a.dw, a.dbias, wk + a.C, s);
}

template <typename T, bool CK>
cudaError_t taps(const ConvBwdArgs& a, cudaStream_t s) {
  return a.K <= 2 ? run<T, 2, CK>(a, s) : a.K <= 4 ? run<T, 4, CK>(a, s) : run<T, 8, CK>(a, s);
}

}  // namespace

cudaError_t launch_conv_bwd(const ConvBwdArgs& a, gdn_dtype dt, cudaStream_t s) {
  if (dt == GDN_BF16)
    return a.xs ? taps<__nv_bfloat16, true>(a, s) : taps<__nv_bfloat16, false>(a, s);
  return a.xs ? taps<float, true>(a, s) : taps<float, false>(a, s);
}

}  // namespace gdn
