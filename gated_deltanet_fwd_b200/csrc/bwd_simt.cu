// bwd_simt.cu -- gradients of the chunked gated delta rule on CUDA cores (fp32 FFMA): the all-fp32
// mode and every shape the tensor-core path does not serve (dk, dv <= 128 in multiples of 16, chunk
// 16/32/64).
//
// With the chunk form of chunk_simt.cu (gamma the in-chunk cumulative log-decay, Gamma = e^gamma,
// d_s = e^{gamma_L - gamma_s}, E_rs = e^{gamma_r - gamma_s}, T' = (I + A)^{-1} diag(beta),
// P = E o Q K^T, W = V - Gamma K S0^T, U = T' W, dO' = scale dO), the gradient dS of the state leaving a
// chunk and dO give
//   dU  = P^T dO' + d K dS^T            dW = T'^T dU = dV
//   dS0 = Gamma_L dS + (Gamma dO')^T Q - (Gamma dW)^T K
//   dN  =  E o (dO' U^T)  (s < r)       p_r = dO'_r . U_r  (a token's own pair, which has no decay)
//   dM  = -E o (dW U^T)   (s < r)
//   dQ  = Gamma (dO' S0) + dN K + p k
//   dKe = dM K - Gamma (dW S0)          dKw = d (U dS) + dN^T Q + dM^T K       dK = dKe + dKw + p q
//   dgamma_r = q_r.(dQ_r - p_r k_r) + k_r.(dKe_r - dKw_r)
//   dg_t = sum_{r >= t} dgamma_r + Gamma_L <S0, dS> + sum_s k_s.(d U dS)_s
//   dbeta_r = (dW_r . U_r) / beta_r^2
// dgamma needs no product of its own: gamma only scales, so its gradient is what the scaled rows meet.
// The terms of a pair (r, s) cancel exactly between r and s for t <= s, both sides being sums of the
// same products.  dbeta follows from U = beta o (v - S k)  and  dW = beta o dR; a beta of magnitude
// below 2^-30 is replaced by +-2^-30 in T' so that the quotient exists (U, dW and all that follows
// move by less than 2^-30 of a beta = 1 token; dV is rescaled, so it is exactly 0 for beta = 0).
//
// Three kernels.  gprep, parallel over (chunk, k-head): T', P and the decay factors to the workspace.
// gwalk, one block per (sequence, v-head, 16 value rows) and direction: forward it leaves the entering
// states S0 and U, backward dS and dW.  (Neither walk needs the other, and value rows are independent in
// both, so the serial part is split over them.)  ggrad, parallel over (chunk, k-head): everything else; the
// v-heads that share the k-head are summed in registers in head order, so dq and dk do not depend on
// scheduling.  Cumulative log-decays are kept in 64 bits: their differences lose half the digits of an
// fp32 sum once |gamma| is in the hundreds.  The walks are bound by the latency of a chunk's few small
// products and barriers.
#include "bwd_internal.cuh"

namespace gdn {
namespace bwd {
namespace {

constexpr int THREADS = 256;
constexpr int DVS = 16;  // value rows per block of the two walks

// [slot][v-head] arrays after the header
struct SimtWs {
  float* tp;   // [C][C] T', then [C][C] P
  float* S;    // [dv][dk] state entering the chunk
  float* dS;   // [dv][dk] gradient of the state leaving it
  float* U;    // [C][dv]
  float* dW;   // [C][dv]
  float* rec;  // [5][C]: Gamma, d, beta (floored), gamma (64-bit, two places)
};

__host__ __device__ inline SimtWs simt_ws(void* ws, int64_t slots, int Hv, int dk, int dv, int C) {
  SimtWs w;
  const int64_t n = slots * Hv;
  w.tp = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(ws) + HEADER);
  w.S = w.tp + n * 2 * C * C;
  w.dS = w.S + n * dv * dk;
  w.U = w.dS + n * dv * dk;
  w.dW = w.U + n * C * dv;
  w.rec = w.dW + n * C * dv;
  return w;
}

struct SimtArgs {
  const void *q, *k, *v, *dout;
  TokStrides ts;
  const float *g, *beta, *S0, *dST;
  const int32_t* cu;
  void *dq, *dk_, *dv_, *dg, *dbeta;
  float* dS0;
  float scale;
  int64_t T, slots;
  int N, Hk, Hv, dk, dv, C;
  void* ws;
  int* status;
};

// This chunk's gates of one v-head, by one warp per call site: gam (64-bit cumulative log-decay, constant
// behind the end) and bet (as used in T').  C <= 64: lanes hold tokens lane and 32 + lane.
__device__ __forceinline__ void scan_gates(const SimtArgs& P, int64_t t0, int L, int h, int lane,
                                           double* gam, float* bet) {
  double x[2];
  float b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 32 * i + lane;
    x[i] = r < L ? (double)P.g[(t0 + r) * P.Hv + h] : 0.0;
    b[i] = r < L ? floor_beta(P.beta[(t0 + r) * P.Hv + h]) : 0.0f;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y0 = __shfl_up_sync(0xffffffffu, x[0], o), y1 = __shfl_up_sync(0xffffffffu, x[1], o);
    if (lane >= o) {
      x[0] += y0;
      x[1] += y1;
    }
  }
  x[1] += __shfl_sync(0xffffffffu, x[0], 31);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (32 * i + lane < P.C) {
      gam[32 * i + lane] = x[i];
      bet[32 * i + lane] = b[i];
    }
}

// rows [t0, t0 + L) of a token tensor into smem [C][ld], zeros behind
template <typename T>
__device__ __forceinline__ void load_rows(const T* src, int64_t stride, int64_t t0, int L, int C,
                                          int width, float* dst, int ld, float mul = 1.0f) {
  const int w4 = width / 4;
  for (int e = threadIdx.x; e < C * w4; e += THREADS) {
    const int r = e / w4, c = 4 * (e - r * w4);
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < L) load4(src + (t0 + r) * stride + c, f);
    *reinterpret_cast<float4*>(dst + r * ld + c) =
        make_float4(mul * f[0], mul * f[1], mul * f[2], mul * f[3]);
  }
}

__device__ __forceinline__ void load_rows_f(const float* src, int C, int width, float* dst, int ld) {
  load_rows<float>(src, width, 0, C, C, width, dst, ld);
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float acc) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, acc))));
}

// ------------------------------------------------------------------------------- gprep -----
template <typename T>
__global__ void __launch_bounds__(THREADS) gprep_kernel(const SimtArgs P) {
  extern __shared__ __align__(16) float sm[];
  const int C = P.C, ldk = P.dk + 4, ldc = C + 4;
  float* Ks = sm;
  float* Qs = Ks + C * ldk;
  float* KK = Qs + C * ldk;
  float* QK = KK + C * ldc;
  float* A = QK + C * ldc;
  float* Ti = A + C * ldc;
  float* bet = Ti + C * ldc;
  double* gam = reinterpret_cast<double*>(bet + C);
  Chunk ch;
  const int64_t slot = blockIdx.x / P.Hk;
  const int hk = (int)(blockIdx.x - slot * P.Hk);
  if (!find_chunk(P.cu, P.T, P.N, C, slot, ch, P.status)) return;
  const SimtWs w = simt_ws(P.ws, P.slots, P.Hv, P.dk, P.dv, C);
  load_rows((const T*)P.k + hk * P.dk, P.ts.k, ch.t0, ch.L, C, P.dk, Ks, ldk);
  load_rows((const T*)P.q + hk * P.dk, P.ts.q, ch.t0, ch.L, C, P.dk, Qs, ldk);
  __syncthreads();
  const int tid = threadIdx.x;
  for (int e = tid; e < C * C / 4; e += THREADS) {  // 1 row x 4 columns
    const int r = e / (C / 4), s = 4 * (e % (C / 4));
    if (s > r) continue;
    float a[4] = {}, b[4] = {};
    for (int i = 0; i < P.dk; i += 4) {
      const float4 kr = *reinterpret_cast<const float4*>(Ks + r * ldk + i);
      const float4 qr = *reinterpret_cast<const float4*>(Qs + r * ldk + i);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float4 ks = *reinterpret_cast<const float4*>(Ks + (s + x) * ldk + i);
        a[x] = dot4(kr, ks, a[x]);
        b[x] = dot4(qr, ks, b[x]);
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      KK[r * ldc + s + x] = a[x];
      QK[r * ldc + s + x] = b[x];
    }
  }
  const int G = P.Hv / P.Hk;
  for (int gi = 0; gi < G; ++gi) {
    const int h = hk * G + gi;
    __syncthreads();
    if (tid < 32) scan_gates(P, ch.t0, ch.L, h, tid, gam, bet);
    __syncthreads();
    float* tp = w.tp + (slot * P.Hv + h) * 2 * C * C;
    float* rec = w.rec + (slot * P.Hv + h) * 5 * C;
    if (tid < C) {
      rec[tid] = expf((float)gam[tid]);
      rec[C + tid] = expf((float)(gam[C - 1] - gam[tid]));
      rec[2 * C + tid] = bet[tid];
      reinterpret_cast<double*>(rec + 3 * C)[tid] = gam[tid];
    }
    for (int e = tid; e < C * C; e += THREADS) {
      const int r = e / C, s = e - r * C;
      const float ex = s <= r ? expf((float)(gam[r] - gam[s])) : 0.0f;
      A[r * ldc + s] = s < r ? bet[r] * ex * KK[r * ldc + s] : 0.0f;
      tp[C * C + e] = s <= r ? ex * QK[r * ldc + s] : 0.0f;
    }
    __syncthreads();
    // T = (I + A)^{-1}, one column per thread by forward substitution
    if (tid < C) {
      const int c = tid;
      for (int r = 0; r < C; ++r) {
        float x = r == c ? 1.0f : 0.0f;
        if (r > c) {
          float x1 = 0.0f, x2 = 0.0f, x3 = 0.0f;
          int s = c;
          for (; s + 3 < r; s += 4) {
            x = fmaf(-A[r * ldc + s], Ti[s * ldc + c], x);
            x1 = fmaf(-A[r * ldc + s + 1], Ti[(s + 1) * ldc + c], x1);
            x2 = fmaf(-A[r * ldc + s + 2], Ti[(s + 2) * ldc + c], x2);
            x3 = fmaf(-A[r * ldc + s + 3], Ti[(s + 3) * ldc + c], x3);
          }
          for (; s < r; ++s) x = fmaf(-A[r * ldc + s], Ti[s * ldc + c], x);
          x += (x1 + x2) + x3;
        }
        Ti[r * ldc + c] = x;
      }
    }
    __syncthreads();
    for (int e = tid; e < C * C; e += THREADS) {
      const int r = e / C, s = e - r * C;
      tp[e] = s <= r ? Ti[r * ldc + s] * bet[s] : 0.0f;
    }
  }
}

// ------------------------------------------------------------------------------- gwalk -----
// Block = (sequence, v-head, 16 value rows, direction).
struct Walk {
  int n, h, hk, j0;
  int64_t s_beg, s_end, slot0, nch;
};

__device__ __forceinline__ bool walk_of(const SimtArgs& P, Walk& W) {
  const int slices = P.dv / DVS, unit = blockIdx.x >> 1;
  W.j0 = (unit % slices) * DVS;
  W.h = (unit / slices) % P.Hv;
  W.n = unit / (slices * P.Hv);
  W.hk = W.h / (P.Hv / P.Hk);
  if (!seq_range(P.cu, P.T, W.n, P.C, W.s_beg, W.s_end, W.slot0)) {
    if (threadIdx.x == 0) report(P.status, GDN_ERR_DEVICE_ARG);
    return false;
  }
  W.nch = (W.s_end - W.s_beg + P.C - 1) / P.C;
  return true;
}

template <typename T>
__device__ __forceinline__ void walk_forward(const SimtArgs& P, const Walk& W, float* sm) {
  const int C = P.C, ldk = P.dk + 4, ldc = C + 4, tid = threadIdx.x;
  float* Ss = sm;                 // [DVS][ldk]
  float* Ks = Ss + DVS * ldk;     // [C][ldk]
  float* Ts = Ks + C * ldk;       // [C][ldc]
  float* Ws = Ts + C * ldc;       // [C][DVS]
  float* Us = Ws + C * DVS;       // [C][DVS]
  float* Gm = Us + C * DVS;
  float* dd = Gm + C;
  const SimtWs w = simt_ws(P.ws, P.slots, P.Hv, P.dk, P.dv, C);
  const int64_t sbase = ((int64_t)W.n * P.Hv + W.h) * P.dv * P.dk + (int64_t)W.j0 * P.dk;
  for (int e = tid; e < DVS * P.dk; e += THREADS)
    Ss[(e / P.dk) * ldk + e % P.dk] = P.S0 ? P.S0[sbase + e] : 0.0f;
  const int w4 = P.dk / 4, jst = THREADS / w4;
  for (int64_t c = 0; c < W.nch; ++c) {
    const int64_t t0 = W.s_beg + c * C, sh = (W.slot0 + c) * P.Hv + W.h;
    const int L = (int)min((int64_t)C, W.s_end - t0);
    __syncthreads();
    if (tid < 2 * C) Gm[tid] = w.rec[sh * 5 * C + tid];  // Gamma, d
    load_rows((const T*)P.k + W.hk * P.dk, P.ts.k, t0, L, C, P.dk, Ks, ldk);
    load_rows_f(w.tp + sh * 2 * C * C, C, C, Ts, ldc);
    load_rows((const T*)P.v + W.h * P.dv + W.j0, P.ts.v, t0, L, C, DVS, Ws, DVS);
    float* So = w.S + sh * P.dv * P.dk + W.j0 * P.dk;
    for (int e = tid; e < DVS * P.dk; e += THREADS) So[e] = Ss[(e / P.dk) * ldk + e % P.dk];
    __syncthreads();
    const int j = tid % DVS;
    for (int r = tid / DVS; r < C; r += THREADS / DVS) {  // W = V - Gamma K S^T
      float acc = 0.0f;
      for (int i = 0; i < P.dk; i += 4)
        acc = dot4(*reinterpret_cast<const float4*>(Ks + r * ldk + i),
                   *reinterpret_cast<const float4*>(Ss + j * ldk + i), acc);
      Ws[r * DVS + j] -= Gm[r] * acc;
    }
    __syncthreads();
    for (int r = tid / DVS; r < C; r += THREADS / DVS) {  // U = T' W
      float acc = 0.0f;
      for (int s = 0; s <= r; ++s) acc = fmaf(Ts[r * ldc + s], Ws[s * DVS + j], acc);
      Us[r * DVS + j] = acc * dd[r];
      w.U[sh * C * P.dv + r * P.dv + W.j0 + j] = acc;
    }
    __syncthreads();
    const float gl = Gm[C - 1];
    if (tid < jst * w4) {
      const int i = 4 * (tid % w4);
      for (int jj = tid / w4; jj < DVS; jj += jst) {
        float4 a = *reinterpret_cast<float4*>(Ss + jj * ldk + i);
        a.x *= gl; a.y *= gl; a.z *= gl; a.w *= gl;
        for (int s = 0; s < C; ++s) {
          const float u = Us[s * DVS + jj];
          const float4 kv = *reinterpret_cast<const float4*>(Ks + s * ldk + i);
          a.x = fmaf(u, kv.x, a.x); a.y = fmaf(u, kv.y, a.y);
          a.z = fmaf(u, kv.z, a.z); a.w = fmaf(u, kv.w, a.w);
        }
        *reinterpret_cast<float4*>(Ss + jj * ldk + i) = a;
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void walk_backward(const SimtArgs& P, const Walk& W, float* sm) {
  const int C = P.C, ldk = P.dk + 4, ldc = C + 4, tid = threadIdx.x;
  float* Ss = sm;              // [DVS][ldk] dS
  float* Ks = Ss + DVS * ldk;  // [C][ldk]
  float* Qs = Ks + C * ldk;    // [C][ldk]
  float* Ts = Qs + C * ldk;    // [C][ldc] T'
  float* Ps = Ts + C * ldc;    // [C][ldc] P
  float* Os = Ps + C * ldc;    // [C][DVS] dO'
  float* Us = Os + C * DVS;    // [C][DVS] dU
  float* Ws = Us + C * DVS;    // [C][DVS] Gamma dW
  float* Gm = Ws + C * DVS;
  float* dd = Gm + C;
  const SimtWs w = simt_ws(P.ws, P.slots, P.Hv, P.dk, P.dv, C);
  const int64_t sbase = ((int64_t)W.n * P.Hv + W.h) * P.dv * P.dk + (int64_t)W.j0 * P.dk;
  for (int e = tid; e < DVS * P.dk; e += THREADS)
    Ss[(e / P.dk) * ldk + e % P.dk] = P.dST ? P.dST[sbase + e] : 0.0f;
  const int w4 = P.dk / 4, jst = THREADS / w4;
  for (int64_t c = W.nch - 1; c >= 0; --c) {
    const int64_t t0 = W.s_beg + c * C, sh = (W.slot0 + c) * P.Hv + W.h;
    const int L = (int)min((int64_t)C, W.s_end - t0);
    __syncthreads();
    if (tid < 2 * C) Gm[tid] = w.rec[sh * 5 * C + tid];  // Gamma, d
    load_rows((const T*)P.k + W.hk * P.dk, P.ts.k, t0, L, C, P.dk, Ks, ldk);
    load_rows((const T*)P.q + W.hk * P.dk, P.ts.q, t0, L, C, P.dk, Qs, ldk);
    load_rows_f(w.tp + sh * 2 * C * C, C, C, Ts, ldc);
    load_rows_f(w.tp + sh * 2 * C * C + C * C, C, C, Ps, ldc);
    load_rows((const T*)P.dout + W.h * P.dv + W.j0, (int64_t)P.Hv * P.dv, t0, L, C, DVS, Os, DVS,
              P.scale);
    float* So = w.dS + sh * P.dv * P.dk + W.j0 * P.dk;
    for (int e = tid; e < DVS * P.dk; e += THREADS) So[e] = Ss[(e / P.dk) * ldk + e % P.dk];
    __syncthreads();
    const int j = tid % DVS;
    for (int s = tid / DVS; s < C; s += THREADS / DVS) {  // dU = P^T dO' + d K dS^T
      float acc = 0.0f;
      for (int i = 0; i < P.dk; i += 4)
        acc = dot4(*reinterpret_cast<const float4*>(Ks + s * ldk + i),
                   *reinterpret_cast<const float4*>(Ss + j * ldk + i), acc);
      acc *= dd[s];
      for (int r = s; r < C; ++r) acc = fmaf(Ps[r * ldc + s], Os[r * DVS + j], acc);
      Us[s * DVS + j] = acc;
    }
    __syncthreads();
    for (int s = tid / DVS; s < C; s += THREADS / DVS) {  // dW = T'^T dU
      float acc = 0.0f;
      for (int r = s; r < C; ++r) acc = fmaf(Ts[r * ldc + s], Us[r * DVS + j], acc);
      Ws[s * DVS + j] = Gm[s] * acc;
      w.dW[sh * C * P.dv + s * P.dv + W.j0 + j] = acc;
      if (s < L) {
        const float bf = w.rec[sh * 5 * C + 2 * C + s];
        float out = acc;
        if (fabsf(bf) == kBetaFloor) out *= P.beta[(t0 + s) * P.Hv + W.h] / bf;  // T' used the floor
        ((T*)P.dv_)[((t0 + s) * P.Hv + W.h) * P.dv + W.j0 + j] = from_f<T>(out);
      }
    }
    __syncthreads();
    const float gl = Gm[C - 1];
    if (tid < jst * w4) {
      const int i = 4 * (tid % w4);
      for (int jj = tid / w4; jj < DVS; jj += jst) {
        float4 a = *reinterpret_cast<float4*>(Ss + jj * ldk + i);
        a.x *= gl; a.y *= gl; a.z *= gl; a.w *= gl;
        for (int s = 0; s < C; ++s) {
          const float u = Os[s * DVS + jj] * Gm[s], x = -Ws[s * DVS + jj];
          const float4 qv = *reinterpret_cast<const float4*>(Qs + s * ldk + i);
          const float4 kv = *reinterpret_cast<const float4*>(Ks + s * ldk + i);
          a.x = fmaf(u, qv.x, fmaf(x, kv.x, a.x)); a.y = fmaf(u, qv.y, fmaf(x, kv.y, a.y));
          a.z = fmaf(u, qv.z, fmaf(x, kv.z, a.z)); a.w = fmaf(u, qv.w, fmaf(x, kv.w, a.w));
        }
        *reinterpret_cast<float4*>(Ss + jj * ldk + i) = a;
      }
    }
  }
  __syncthreads();
  if (P.dS0)
    for (int e = tid; e < DVS * P.dk; e += THREADS)
      P.dS0[sbase + e] = Ss[(e / P.dk) * ldk + e % P.dk];
}

template <typename T>
__global__ void __launch_bounds__(THREADS) gwalk_kernel(const SimtArgs P) {
  extern __shared__ __align__(16) float sm[];
  Walk W;
  if (!walk_of(P, W)) return;
  if (blockIdx.x & 1)
    walk_forward<T>(P, W, sm);
  else
    walk_backward<T>(P, W, sm);
}

// ------------------------------------------------------------------------------- ggrad -----
// Warp w holds rows 8w .. 8w + 7 of the chunk, lane l columns 4l .. 4l + 3 of dq, dKe and dKw.
template <typename T>
__global__ void __launch_bounds__(THREADS) ggrad_kernel(const SimtArgs P) {
  extern __shared__ __align__(16) float sm[];
  const int C = P.C, ldk = P.dk + 4, ldv = P.dv + 4, ldc = C + 4, tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  float* Ks = sm;                // [C][ldk]
  float* Qs = Ks + C * ldk;      // [C][ldk]
  float* Us = Qs + C * ldk;      // [C][ldv]
  float* Os = Us + C * ldv;      // [C][ldv] dO'
  float* Ws = Os + C * ldv;      // [C][ldv] dW
  float* Ns = Ws + C * ldv;      // [C][ldc] dN
  float* Ms = Ns + C * ldc;      // [C][ldc] dM
  float* Gm = Ms + C * ldc;
  float* dd = Gm + C;
  float* bet = dd + C;
  float* own = bet + C;   // p
  float* dgm = own + C;   // dgamma
  float* red = dgm + C;   // [8]
  float* kw = red + 8;    // [C] k.(d U dS)
  double* gam = reinterpret_cast<double*>(kw + C);
  Chunk ch;
  const int64_t slot = blockIdx.x / P.Hk;
  const int hk = (int)(blockIdx.x - slot * P.Hk);
  if (!find_chunk(P.cu, P.T, P.N, C, slot, ch, P.status)) return;
  const SimtWs w = simt_ws(P.ws, P.slots, P.Hv, P.dk, P.dv, C);
  const int G = P.Hv / P.Hk, L = ch.L;
  const int64_t t0 = ch.t0;
  load_rows((const T*)P.k + hk * P.dk, P.ts.k, t0, L, C, P.dk, Ks, ldk);
  load_rows((const T*)P.q + hk * P.dk, P.ts.q, t0, L, C, P.dk, Qs, ldk);
  const int r0 = 8 * warp, c0 = 4 * lane;
  const bool rows_on = r0 < C, on = rows_on && c0 < P.dk;
  float dq[8][4] = {}, dk[8][4] = {};  // summed over the v-heads
  for (int gi = 0; gi < G; ++gi) {
    const int h = hk * G + gi;
    const int64_t sh = slot * P.Hv + h;
    const float* S = w.S + sh * P.dv * P.dk;
    const float* dS = w.dS + sh * P.dv * P.dk;
    __syncthreads();
    for (int e = tid; e < 3 * C; e += THREADS) Gm[e] = w.rec[sh * 5 * C + e];  // Gamma, d, beta
    if (tid < C) gam[tid] = reinterpret_cast<const double*>(w.rec + sh * 5 * C + 3 * C)[tid];
    load_rows_f(w.U + sh * C * P.dv, C, P.dv, Us, ldv);
    load_rows_f(w.dW + sh * C * P.dv, C, P.dv, Ws, ldv);
    load_rows((const T*)P.dout + h * P.dv, (int64_t)P.Hv * P.dv, t0, L, C, P.dv, Os, ldv, P.scale);
    __syncthreads();
    float frob = 0.0f;
    for (int e = tid; e < P.dv * P.dk; e += THREADS) frob = fmaf(S[e], dS[e], frob);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) frob += __shfl_xor_sync(0xffffffffu, frob, o);
    if (lane == 0) red[warp] = frob;
    __syncthreads();
    // dN, dM and p: this warp's rows, columns lane and lane + 32
    if (rows_on) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int s = lane + 32 * half;
        if (s >= C) break;
        float on_[8] = {}, om[8] = {};
        for (int jx = 0; jx < P.dv; jx += 4) {
          const float4 u = *reinterpret_cast<const float4*>(Us + s * ldv + jx);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            on_[x] = dot4(*reinterpret_cast<const float4*>(Os + (r0 + x) * ldv + jx), u, on_[x]);
            om[x] = dot4(*reinterpret_cast<const float4*>(Ws + (r0 + x) * ldv + jx), u, om[x]);
          }
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int r = r0 + x;
          const float e = s < r ? expf((float)(gam[r] - gam[s])) : 0.0f;
          Ns[r * ldc + s] = e * on_[x];
          Ms[r * ldc + s] = -e * om[x];
          if (s == r) {
            own[r] = on_[x];
            if (r < L)
              ((T*)P.dbeta)[(t0 + r) * P.Hv + h] = from_f<T>(om[x] / bet[r] / bet[r]);
          }
        }
      }
    }
    __syncthreads();
    float aq[8][4] = {}, ae[8][4] = {}, aw[8][4] = {};
    if (on) {
      for (int jx = 0; jx < P.dv; ++jx) {
        const float4 s4 = *reinterpret_cast<const float4*>(S + jx * P.dk + c0);
        const float4 d4 = *reinterpret_cast<const float4*>(dS + jx * P.dk + c0);
        const float sv[4] = {s4.x, s4.y, s4.z, s4.w}, dv4[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float o = Os[(r0 + x) * ldv + jx], ww = Ws[(r0 + x) * ldv + jx],
                      u = Us[(r0 + x) * ldv + jx];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            aq[x][y] = fmaf(o, sv[y], aq[x][y]);
            ae[x][y] = fmaf(ww, sv[y], ae[x][y]);
            aw[x][y] = fmaf(u, dv4[y], aw[x][y]);
          }
        }
      }
#pragma unroll
      for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          aq[x][y] *= Gm[r0 + x];
          ae[x][y] *= -Gm[r0 + x];
          aw[x][y] *= dd[r0 + x];
        }
    }
    if (rows_on) {
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        float v = 0.0f;
        if (on)
#pragma unroll
          for (int y = 0; y < 4; ++y) v = fmaf(Ks[(r0 + x) * ldk + c0 + y], aw[x][y], v);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) kw[r0 + x] = v;
      }
    }
    if (on) {
      for (int s = 0; s < r0 + 8; ++s) {  // rows of this warp against earlier tokens
        const float4 k4 = *reinterpret_cast<const float4*>(Ks + s * ldk + c0);
        const float kv[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float nn = Ns[(r0 + x) * ldc + s], mm = Ms[(r0 + x) * ldc + s];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            aq[x][y] = fmaf(nn, kv[y], aq[x][y]);
            ae[x][y] = fmaf(mm, kv[y], ae[x][y]);
          }
        }
      }
      for (int r = r0; r < C; ++r) {  // and later tokens
        const float4 k4 = *reinterpret_cast<const float4*>(Ks + r * ldk + c0);
        const float4 q4 = *reinterpret_cast<const float4*>(Qs + r * ldk + c0);
        const float kv[4] = {k4.x, k4.y, k4.z, k4.w}, qv[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float nn = Ns[r * ldc + r0 + x], mm = Ms[r * ldc + r0 + x];
#pragma unroll
          for (int y = 0; y < 4; ++y) aw[x][y] = fmaf(nn, qv[y], fmaf(mm, kv[y], aw[x][y]));
        }
      }
    }
    if (rows_on) {
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int r = r0 + x;
        float v = 0.0f;
        if (on) {
          const float p = own[r];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float kv = Ks[r * ldk + c0 + y], qv = Qs[r * ldk + c0 + y];
            v = fmaf(qv, aq[x][y], fmaf(kv, ae[x][y] - aw[x][y], v));
            dq[x][y] += fmaf(p, kv, aq[x][y]);
            dk[x][y] += fmaf(p, qv, ae[x][y] + aw[x][y]);
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) dgm[r] = v;
      }
    }
    __syncthreads();
    if (tid == 0) {  // dg: suffix sums, and what leaves through the state
      float f = 0.0f, acc = 0.0f;
      for (int x = 0; x < THREADS / 32; ++x) f += red[x];
      f *= Gm[C - 1];
      for (int r = 0; r < L; ++r) f += kw[r];
      for (int r = L - 1; r >= 0; --r) {
        acc += dgm[r];
        ((T*)P.dg)[(t0 + r) * P.Hv + h] = from_f<T>(acc + f);
      }
    }
  }
  if (on) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int r = r0 + x;
      if (r >= L) break;
      T* oq = (T*)P.dq + ((t0 + r) * P.Hk + hk) * P.dk + c0;
      T* ok = (T*)P.dk_ + ((t0 + r) * P.Hk + hk) * P.dk + c0;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        oq[y] = from_f<T>(dq[x][y]);
        ok[y] = from_f<T>(dk[x][y]);
      }
    }
  }
}

template <typename T>
cudaError_t launch_t(const SimtArgs& P, cudaStream_t s) {
  const int C = P.C, ldk = P.dk + 4, ldv = P.dv + 4, ldc = C + 4;
  const size_t f = sizeof(float);
  const size_t sm_prep = (2 * (size_t)C * ldk + 4 * C * ldc + C) * f + C * 8;
  const size_t sm_walk =  // the backward walk's; the forward one needs less
      ((size_t)(DVS + 2 * C) * ldk + 2 * C * ldc + 3 * C * DVS + 2 * C) * f;
  const size_t sm_grad =
      (2 * (size_t)C * ldk + 3 * C * ldv + 2 * C * ldc + 6 * C + 8) * f + C * 8;
  auto set = [](auto kern, size_t bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  };
  cudaError_t e = set(gprep_kernel<T>, sm_prep);
  if (e == cudaSuccess) e = set(gwalk_kernel<T>, sm_walk);
  if (e == cudaSuccess) e = set(ggrad_kernel<T>, sm_grad);
  if (e != cudaSuccess) return e;
  const int64_t par = P.slots * P.Hk, walks = 2 * (int64_t)P.N * P.Hv * (P.dv / DVS);
  if (par > 0x7fffffff || walks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (par > 0) gprep_kernel<T><<<(unsigned)par, THREADS, sm_prep, s>>>(P);
  if (walks > 0) gwalk_kernel<T><<<(unsigned)walks, THREADS, sm_walk, s>>>(P);
  if (par > 0) ggrad_kernel<T><<<(unsigned)par, THREADS, sm_grad, s>>>(P);
  return cudaGetLastError();
}

}  // namespace

size_t simt_workspace_bytes(int N, int64_t n_tok, int Hv, int dk, int dv, int C) {
  const size_t n = (size_t)max_slots(N, n_tok, C) * Hv;
  return HEADER +
         n * (2 * (size_t)C * C + 2 * (size_t)dv * dk + 2 * (size_t)C * dv + 5 * (size_t)C) * sizeof(float);
}

cudaError_t launch_simt(const Args& a, cudaStream_t s) {
  SimtArgs p;
  p.q = a.q; p.k = a.k; p.v = a.v; p.dout = a.dout;
  p.ts = a.ts;
  p.g = a.g; p.beta = a.beta; p.S0 = a.S0; p.dST = a.dST;
  p.cu = a.cu;
  p.dq = a.dq; p.dk_ = a.dk_; p.dv_ = a.dv_; p.dg = a.dg; p.dbeta = a.dbeta;
  p.dS0 = a.dS0;
  p.scale = a.scale;
  p.T = a.T;
  p.slots = (int64_t)a.B * a.T > 0 ? max_slots(a.N, (int64_t)a.B * a.T, a.C) : 0;
  p.N = a.N; p.Hk = a.Hk; p.Hv = a.Hv; p.dk = a.dk; p.dv = a.dv; p.C = a.C;
  p.ws = a.ws;
  p.status = a.status;
  return a.dt == GDN_BF16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
}

}  // namespace bwd
}  // namespace gdn
