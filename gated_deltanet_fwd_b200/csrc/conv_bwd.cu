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
// dy and x in, dx out, once each (and K-1 tokens of halo at the ends of a token range).  2 x 16384 tokens of 8192
// channels bf16, 4 taps: 461 us for 1.61 GB, 3.5 TB/s, 53 % of a copy, and 14 us for the partial rows.  The 149
// instructions for four channels of a token (packed arithmetic, two channels each; eight on the special-function
// unit) would take 269 us of that if every issue slot were used, and 58 % are: what bounds it is latency inside
// a warp, with sixteen warps an SM (128 registers).  For each pair of tokens the norm's sums are seven dependent
// shuffles, a reciprocal root and two exchanges before a dpre exists.
// A thread holds 4 channels and streams a range of tokens forward: x[t-KT+1 .. t] and
// dpre[t-KT+1 .. t] are register windows, so each token is loaded and each dpre computed once; dx is
// stored KT-1 tokens late.  Whole batches of tokens inside a range and a sequence run unrolled without
// conditions, their inputs copied up to three batches ahead into a private ring in shared memory
// (registers are taken by the windows and sums); the ends run token by token.
// A warp spans 128 channels, so the norm's sums for groups up to 128 are shuffles -- for 128 itself two
// tokens' four sums share them.  A group of 256 spans the block's two warps, which exchange their sums
// through shared memory.
// dw and dbias are summed in registers over the range; each range writes one partial row, added in
// order by a second kernel.  Kernels exist for 2, 4 and 8 taps; a smaller K has leading zero taps.
#include "act8.cuh"
#include "f32x2.cuh"

namespace gdn {
namespace {

constexpr int CB_THREADS = 64;
constexpr int CB_CH = 4;  // channels per thread

struct Four {  // 4 channels as two packed pairs
  f32x2 a, b;
};
__device__ __forceinline__ Four zero4() { return {0ull, 0ull}; }

template <typename T>
struct Raw4;
template <>
struct Raw4<__nv_bfloat16> {
  uint2 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = __ldg(reinterpret_cast<const uint2*>(p));
  }
  __device__ __forceinline__ Four get() const { return {widen(u.x), widen(u.y)}; }
};
template <>
struct Raw4<float> {
  float4 u;
  __device__ __forceinline__ void load(const float* p) {
    u = __ldg(reinterpret_cast<const float4*>(p));
  }
  __device__ __forceinline__ Four get() const { return {two(u.x, u.y), two(u.z, u.w)}; }
};

__device__ __forceinline__ void put4(__nv_bfloat16* p, const Four& f) {
  const float2 x = parts(f.a), y = parts(f.b);
  __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(y.x, y.y);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}
__device__ __forceinline__ void put4(float* p, const Four& f) {
  const float2 x = parts(f.a), y = parts(f.b);
  *reinterpret_cast<float4*>(p) = make_float4(x.x, x.y, y.x, y.y);
}

// asynchronous copy of N bytes into this thread's own shared memory
template <int N>
__device__ __forceinline__ void ring_copy(unsigned char* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ring_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 4 channels of the conv's input: as they are, or codes and their group's scale.  `at` = t * C + c.
template <typename T, bool CK>
struct XIn {
  Raw4<T> r;
  static constexpr int SLOT = 4 * sizeof(T);  // bytes of a ring entry
  __device__ __forceinline__ void load(const ConvBwdArgs& P, int64_t at, int64_t t, int) {
    r.load((const T*)P.x + at);
  }
  __device__ __forceinline__ Four get() const { return r.get(); }
  static __device__ __forceinline__ void copy(unsigned char* slot, const ConvBwdArgs& P, int64_t at,
                                              int64_t, int) {
    ring_copy<SLOT>(slot, (const T*)P.x + at);
  }
};
template <typename T>
struct XIn<T, true> {
  uint32_t u;
  float sc;
  static constexpr int SLOT = 8;
  static __device__ __forceinline__ void copy(unsigned char* slot, const ConvBwdArgs& P, int64_t at,
                                              int64_t t, int group) {
    ring_copy<4>(slot, (const int8_t*)P.x + at);
    ring_copy<4>(slot + 4, P.xs + t * P.xgroups + group);
  }
  __device__ __forceinline__ void load(const ConvBwdArgs& P, int64_t at, int64_t t, int group) {
    u = __ldg(reinterpret_cast<const uint32_t*>((const int8_t*)P.x + at));
    sc = __ldg(P.xs + t * P.xgroups + group);
  }
  __device__ __forceinline__ Four get() const {
    float f[4];
    act8::unpack4(u, sc, f);
    return {two(f[0], f[1]), two(f[2], f[3])};
  }
};

// G128: the normalised groups are 128 channels, one warp each
template <typename T, int KT, bool CK, bool G128>
__global__ void __launch_bounds__(CB_THREADS, KT == 8 ? 4 : 8) conv_bwd_kernel(const ConvBwdArgs P) {
  constexpr int D = KT - 1;                // tokens that dx lags behind
  constexpr int PF = 4, AHEAD = 3;         // tokens of a batch, batches copied ahead
  constexpr int XS = XIn<T, CK>::SLOT, YS = 4 * sizeof(T), RING = PF * (AHEAD + 1);
  __shared__ __align__(16) unsigned char ring_x[RING * CB_THREADS * XS];
  __shared__ __align__(16) unsigned char ring_y[RING * CB_THREADS * YS];
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
  const int xg = CK && on ? c / P.xgroup : 0;

  Four w[KT], bias = zero4(), dw[KT], db = zero4();
#pragma unroll
  for (int i = 0; i < KT; ++i) {
    const float* p = P.w + (int64_t)c * K + i - pad;
    const bool has = on && i >= pad;
    w[i].a = two(has ? __ldg(p) : 0.0f, has ? __ldg(p + K) : 0.0f);
    w[i].b = two(has ? __ldg(p + 2 * K) : 0.0f, has ? __ldg(p + 3 * K) : 0.0f);
    dw[i] = zero4();
  }
  if (on && P.bias) {
    bias.a = two(__ldg(P.bias + c), __ldg(P.bias + c + 1));
    bias.b = two(__ldg(P.bias + c + 2), __ldg(P.bias + c + 3));
  }
  // a history place of this thread's channels (K - 1 apart)
  auto hist = [&](const float* p) -> Four {
    return {two(__ldg(p), __ldg(p + K - 1)), two(__ldg(p + 2 * (K - 1)), __ldg(p + 3 * (K - 1)))};
  };
  // up to 32 entries of cu_seqlens are held by the lanes, one each: one load instead of a search
  const bool held = P.cu && P.N < 32;
  const int mine = held && lane <= P.N ? P.cu[lane] : 0x7fffffff;
  auto bound = [&](int m, int64_t& b, int64_t& e) {  // sequence m's tokens, clamped to the tensor
    if (held) {
      b = __shfl_sync(0xffffffffu, mine, m);
      e = __shfl_sync(0xffffffffu, mine, m + 1);
    } else {
      b = P.cu ? P.cu[m] : (int64_t)m * P.T;
      e = P.cu ? P.cu[m + 1] : b + P.T;
    }
    b = max((int64_t)0, min(b, P.n_tok));
    e = max(b, min(e, P.n_tok));
  };
  if (blockIdx.y == gridDim.y - 1 && P.dcs_in) {  // empty sequences: the history passes through
    for (int m = 0; m < P.N; ++m) {
      int64_t b, e;
      bound(m, b, e);
      if (e > b || !on) continue;
      const int64_t at = ((int64_t)m * P.C + c) * (K - 1);
      float v[4 * D];
#pragma unroll
      for (int q = 0; q < 4 * D; ++q)
        v[q] = P.dcs_out && q < 4 * (K - 1) ? __ldg(P.dcs_out + at + q) : 0.0f;
#pragma unroll
      for (int q = 0; q < 4 * D; ++q)
        if (q < 4 * (K - 1)) P.dcs_in[at + q] = v[q];
    }
  }
  if (r0 < r1) {
    const f32x2 one = two(1.0f, 1.0f), minus = two(-1.0f, -1.0f);
    Four xw[KT], dp[KT];  // x[t - d], dpre[t - d]
    // 1 / (1 + 2^(-v log2 e)); the approximate reciprocal of an overflowed sum is 0
    const f32x2 neg_log2e = two(-1.4426950408889634f, -1.4426950408889634f);
    auto sig = [&](f32x2 v) {
      const float2 f = parts(mul2(v, neg_log2e));
      float2 e;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(f.x));
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(f.y));
      e = parts(add2(two(e.x, e.y), one));
      asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
      asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
      return two(e.x, e.y);
    };
    // the activation of the token whose input came last, and its slope sigma (1 + pre (1 - sigma)) -- as a
    // product: it is 0, not infinity - infinity, far to the left
    auto activate = [&](const Four& x, Four& act, Four& slope) {
#pragma unroll
      for (int d = KT - 1; d > 0; --d) xw[d] = xw[d - 1];
      xw[0] = x;
      Four pre = bias;
#pragma unroll
      for (int d = 0; d < KT; ++d) {
        pre.a = fma2(w[KT - 1 - d].a, xw[d].a, pre.a);
        pre.b = fma2(w[KT - 1 - d].b, xw[d].b, pre.b);
      }
      const f32x2 sa = sig(pre.a), sb = sig(pre.b);
      act = {mul2(pre.a, sa), mul2(pre.b, sb)};
      slope.a = mul2(sa, fma2(pre.a, fma2(sa, minus, one), one));
      slope.b = mul2(sb, fma2(pre.b, fma2(sb, minus, one), one));
    };
    auto dot = [](const Four& u, const Four& v) {
      const float2 s = parts(fma2(u.a, v.a, mul2(u.b, v.b)));
      return s.x + s.y;
    };
    // dy <- rn (dy - act rn^2 ad), f = -rn^2 ad
    auto through_norm = [](Four& dy, const Four& act, float rn, float f) {
      const f32x2 f2 = two(f, f), r2 = two(rn, rn);
      dy.a = mul2(r2, fma2(act.a, f2, dy.a));
      dy.b = mul2(r2, fma2(act.b, f2, dy.b));
    };
    auto enter = [&](const Four& dy, const Four& slope) {  // a token's dpre
#pragma unroll
      for (int d = KT - 1; d > 0; --d) dp[d] = dp[d - 1];
      dp[0] = {mul2(dy.a, slope.a), mul2(dy.b, slope.b)};
    };
    // one token: its input and output gradient in; the windows move on, dp[0] is its dpre
    auto token = [&](const Four& x, Four dy, int64_t t) {
      Four act, slope;
      activate(x, act, slope);
      if (any) {
        float ss = dot(act, act), ad = dot(act, dy);
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
          const float rn = rsqrtf(ss + P.eps);
          through_norm(dy, act, rn, -rn * rn * ad);
        }
      }
      enter(dy, slope);
    };
    auto count = [&]() {  // the token belongs to this range: its part of dw and dbias
      db.a = add2(db.a, dp[0].a);
      db.b = add2(db.b, dp[0].b);
#pragma unroll
      for (int d = 0; d < KT; ++d) {
        dw[KT - 1 - d].a = fma2(dp[0].a, xw[d].a, dw[KT - 1 - d].a);
        dw[KT - 1 - d].b = fma2(dp[0].b, xw[d].b, dw[KT - 1 - d].b);
      }
    };
    auto back = [&]() {  // the gradient of the input D places before dp[0]
      Four v = {mul2(w[0].a, dp[0].a), mul2(w[0].b, dp[0].b)};
#pragma unroll
      for (int i = 1; i < KT; ++i) {
        v.a = fma2(w[i].a, dp[i].a, v.a);
        v.b = fma2(w[i].b, dp[i].b, v.b);
      }
      return v;
    };
    int n = held ? min(__popc(__ballot_sync(0xffffffffu, (int64_t)mine <= r0)) - 1, P.N - 1)
                 : seq_of_token(P.cu, P.N, P.T, r0);
    if (n < 0) n = 0;
    for (; n < P.N; ++n) {
      int64_t s_beg, s_end;
      bound(n, s_beg, s_end);
      if (s_beg >= r1) break;
      const int64_t a = max(r0, s_beg), e = min(r1, s_end);
      if (a >= e) continue;
      const int64_t te = min(e + D, s_end);
      const int64_t cs = ((int64_t)n * P.C + c) * (K - 1);
#pragma unroll
      for (int d = 0; d < KT; ++d) {
        xw[d] = zero4();
        dp[d] = zero4();
      }
#pragma unroll
      for (int d = 1; d < KT; ++d) {  // the inputs before the first token
        const int64_t p = a - d;
        if (on && d < K) {
          if (p >= s_beg) {
            XIn<T, CK> xi;
            xi.load(P, p * P.C + c, p, xg);
            xw[d - 1] = xi.get();
          } else if (P.cs_in) {
            xw[d - 1] = hist(P.cs_in + cs + (K - 1) + (p - s_beg));
          }
        }
      }
      // place p: a token of this range, or one of the history if the sequence starts here
      auto emit = [&](int64_t p) {
        if (!on) return;
        Four v = back();
        const int64_t jo = p - (s_end - (K - 1));  // place in the history left behind
        if (P.dcs_out && jo >= 0 && jo < K - 1) {
          const Four o = hist(P.dcs_out + cs + jo);
          v.a = add2(v.a, o.a);
          v.b = add2(v.b, o.b);
        }
        if (p >= a) {
          if (p < e) put4((T*)P.dx + p * P.C + c, v);
        } else if (p < s_beg && a == s_beg && P.dcs_in) {
          const int64_t j = p - s_beg + (K - 1);
          if (j >= 0) {
            float* o = P.dcs_in + cs + j;
            const float2 x = parts(v.a), y = parts(v.b);
            o[0] = x.x;
            o[K - 1] = x.y;
            o[2 * (K - 1)] = y.x;
            o[3 * (K - 1)] = y.y;
          }
        }
      };
      unsigned char* rx = ring_x + tid * XS;
      unsigned char* ry = ring_y + tid * YS;
      // copies of the batch whose first element is `at`, as far as its tokens are needed
      const int64_t row = P.C;
      auto fetch = [&](int64_t u0, int slot) {
        const int64_t left = te - u0;
        if (on && left > 0) {
          const int64_t at = u0 * row + c;
          const int m = left < PF ? (int)left : PF;
#pragma unroll
          for (int u = 0; u < PF; ++u)
            if (u < m) {
              XIn<T, CK>::copy(rx + (slot + u) * CB_THREADS * XS, P, at + u * row, u0 + u, xg);
              ring_copy<YS>(ry + (slot + u) * CB_THREADS * YS, (const T*)P.dy + at + u * row);
            }
        }
        ring_commit();
      };
      auto x_at = [&](int k) {
        return on ? reinterpret_cast<const XIn<T, CK>*>(rx + k * CB_THREADS * XS)->get() : zero4();
      };
      auto y_at = [&](int k) {
        return on ? reinterpret_cast<const Raw4<T>*>(ry + k * CB_THREADS * YS)->get() : zero4();
      };
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) fetch(a + k * PF, k * PF);
      int slot = 0;
      int64_t t = a;
      auto slowly = [&]() {  // one batch with every condition
        fetch(t + AHEAD * PF, (slot + AHEAD * PF) % RING);
        ring_wait<AHEAD>();
#pragma unroll 1
        for (int u = 0; u < PF && t + u < te; ++u) {
          token(x_at(slot + u), y_at(slot + u), t + u);
          if (t + u < e) count();
          emit(t + u - D);
        }
        slot = (slot + PF) % RING;
        t += PF;
      };
      slowly();  // its tokens have nothing to store yet, or history
      static_assert(D <= PF || KT == 8, "the first batch covers the lag");
      if (D > PF && t < te) slowly();
#pragma unroll 1
      for (; t + PF <= e; t += PF) {
        fetch(t + AHEAD * PF, (slot + AHEAD * PF) % RING);
        ring_wait<AHEAD>();
        {
          T* out = (T*)P.dx + (t - D) * P.C + c;
#pragma unroll
          for (int u = 0; u < PF; u += 2) {
            if (G128) {
              // two tokens at once: lane halves take a token each, quarters a sum each, and the norm's
              // factors are computed for both in one go: 9 shuffles for what took 20
              Four act0, act1, sl0, sl1, dy0 = y_at(slot + u), dy1 = y_at(slot + u + 1);
              activate(x_at(slot + u), act0, sl0);
              const Four x3 = xw[KT - 1];  // leaves the window, but token t + u still needs it
              activate(x_at(slot + u + 1), act1, sl1);
              if (any) {
                const bool up = lane & 16, second = lane & 8;
                const float s0 = dot(act0, act0), s1 = dot(act1, act1);
                const float a0 = dot(act0, dy0), a1 = dot(act1, dy1);
                const float s = (up ? s1 : s0) + __shfl_xor_sync(0xffffffffu, up ? s0 : s1, 16);
                const float q = (up ? a1 : a0) + __shfl_xor_sync(0xffffffffu, up ? a0 : a1, 16);
                float v = (second ? q : s) + __shfl_xor_sync(0xffffffffu, second ? s : q, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                const float o = __shfl_xor_sync(0xffffffffu, v, 8);
                const float rn = rsqrtf((second ? o : v) + P.eps);
                const float f = -rn * rn * (second ? v : o);
                const float rno = __shfl_xor_sync(0xffffffffu, rn, 16);
                const float fo = __shfl_xor_sync(0xffffffffu, f, 16);
                if (norm) {
                  through_norm(dy0, act0, up ? rno : rn, up ? fo : f);
                  through_norm(dy1, act1, up ? rn : rno, up ? f : fo);
                }
              }
              enter(dy0, sl0);
              // xw is a token further than dp here
              db.a = add2(db.a, dp[0].a);
              db.b = add2(db.b, dp[0].b);
#pragma unroll
              for (int d = 0; d < KT; ++d) {
                const Four& x = d + 1 < KT ? xw[d + 1] : x3;
                dw[KT - 1 - d].a = fma2(dp[0].a, x.a, dw[KT - 1 - d].a);
                dw[KT - 1 - d].b = fma2(dp[0].b, x.b, dw[KT - 1 - d].b);
              }
              if (on) put4(out + (int64_t)u * P.C, back());
              enter(dy1, sl1);
              count();
              if (on) put4(out + (int64_t)(u + 1) * P.C, back());
            } else {
#pragma unroll
              for (int k = u; k < u + 2; ++k) {
                token(x_at(slot + k), y_at(slot + k), t + k);
                count();
                if (on) put4(out + (int64_t)k * P.C, back());
              }
            }
          }
        }
        slot = (slot + PF) % RING;
      }
#pragma unroll 1
      while (t < te) slowly();
      ring_wait<0>();
      if (te == s_end) {  // nothing follows the sequence
#pragma unroll 1
        for (int m = 1; m <= D; ++m) {
#pragma unroll
          for (int d = KT - 1; d > 0; --d) dp[d] = dp[d - 1];
          dp[0] = zero4();
          emit(s_end - 1 + m - D);
        }
      }
      if (gl == 64 && any) __syncthreads();  // the exchange starts over on the next sequence
    }
  }
  if (on) {
    float* row = P.part + (int64_t)blockIdx.y * P.C * (K + 1);
#pragma unroll
    for (int i = 0; i < KT; ++i)
      if (i >= pad) {
        const float2 x = parts(dw[i].a), y = parts(dw[i].b);
        float* o = row + (int64_t)c * K + i - pad;
        o[0] = x.x;
        o[K] = x.y;
        o[2 * K] = y.x;
        o[3 * K] = y.y;
      }
    const float2 x = parts(db.a), y = parts(db.b);
    *reinterpret_cast<float4*>(row + (int64_t)P.C * K + c) = make_float4(x.x, x.y, y.x, y.y);
  }
}

template <typename T, int KT, bool CK, bool G128>
cudaError_t run(ConvBwdArgs a, cudaStream_t s) {
  int dev = 0, sms = 148, per_sm = 1;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, conv_bwd_kernel<T, KT, CK, G128>, CB_THREADS, 0);
  const int64_t tiles = (a.C + CB_THREADS * CB_CH - 1) / (CB_THREADS * CB_CH);
  // four waves of blocks: the channels without a norm take less time, and the hardware's dispatch evens
  // that out; at least 32 tokens in a range (its ends cost about 8 more; 16 and 64 are slower)
  int64_t ranges = 4 * (int64_t)sms * (per_sm > 0 ? per_sm : 1) / tiles;
  if (ranges > (a.n_tok + 31) / 32) ranges = (a.n_tok + 31) / 32;
  if (ranges > a.max_parts) ranges = a.max_parts;
  if (ranges < 1) ranges = 1;
  conv_bwd_kernel<T, KT, CK, G128><<<dim3((unsigned)tiles, (unsigned)ranges), CB_THREADS, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t wk = (int64_t)a.C * a.K;
  return launch_sum_parts(a.part, ranges, a.dbias ? wk + a.C : wk, wk, a.dw, a.dbias, wk + a.C, s);
}

template <typename T, bool CK, bool G128>
cudaError_t taps(const ConvBwdArgs& a, cudaStream_t s) {
  return a.K <= 2   ? run<T, 2, CK, G128>(a, s)
         : a.K <= 4 ? run<T, 4, CK, G128>(a, s)
                    : run<T, 8, CK, G128>(a, s);
}
template <typename T, bool CK>
cudaError_t group(const ConvBwdArgs& a, cudaStream_t s) {
  return a.group == 128 ? taps<T, CK, true>(a, s) : taps<T, CK, false>(a, s);
}

}  // namespace

cudaError_t launch_conv_bwd(const ConvBwdArgs& a, gdn_dtype dt, cudaStream_t s) {
  if (dt == GDN_BF16)
    return a.xs ? group<__nv_bfloat16, true>(a, s) : group<__nv_bfloat16, false>(a, s);
  return a.xs ? group<float, true>(a, s) : group<float, false>(a, s);
}

}  // namespace gdn
