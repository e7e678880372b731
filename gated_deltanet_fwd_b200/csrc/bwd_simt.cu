// bwd_simt.cu -- gradients of the chunked gated delta rule on CUDA cores (fp32 FFMA): the all-fp32
// mode and every shape the tensor-core path does not serve (dk, dv <= 128 in multiples of 16, chunk
// 16 or 32; a caller's 64 runs as 32).
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
//   dgamma_r = q_r.(dQ_r - p_r k_r) + k_r.(dKe_r - dKw_r + (d U dS)_r),   kappa_s = k_s.(d U dS)_s
//   dg_t = sum_{r >= t} dgamma_r + Gamma_L <S0, dS> + sum_{s < t} kappa_s
//   dbeta_r = (dW_r . U_r) / beta_r^2
// dgamma needs no product of its own: gamma only scales, so its gradient is what the scaled rows meet.
// The terms of a pair (r, s) cancel exactly between r and s for t <= s, both sides being sums of the
// same products; and -kappa_r of a later token meets the +kappa_r of the state leaving, so neither is formed:
// under strong decay dg is smaller than their rounding errors.  dbeta follows from U = beta o (v - S k)  and  dW = beta o dR; a beta of magnitude
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
// products and barriers: 1034 tokens in four ragged sequences, 4 v-heads, dk 64, dv 96, chunk 32, fp32: gprep 11,
// gwalk 113, ggrad 36 us.  With each chunk's loads awaited before its products gwalk took 137; chunks of 64 are slower
// than of 32 at every size tried.
#include <type_traits>

#include "bwd_internal.cuh"
#include "ptx.cuh"

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
  int stages;  // of the walks (set at launch)
  void* ws;
  int* status;
};

// This chunk's gates of one v-head, by one warp per call site: gam (64-bit cumulative log-decay, constant
// behind the end) and bet (as used in T').  C <= 32: a lane a token.
__device__ __forceinline__ void scan_gates(const SimtArgs& P, int64_t t0, int L, int h, int lane,
                                           double* gam, float* bet) {
  double x = lane < L ? (double)floor_decay(P.g[(t0 + lane) * P.Hv + h]) : 0.0;
  const float b = lane < L ? floor_beta(P.beta[(t0 + lane) * P.Hv + h]) : 0.0f;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane < P.C) {
    gam[lane] = x;
    bet[lane] = b;
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

// load_rows without waiting where the source is fp32 (ptx::cp_async_wait_all does).
template <typename T>
__device__ __forceinline__ void fetch_rows(const T* src, int64_t stride, int64_t t0, int L, int C,
                                           int width, float* dst, int ld) {
  if constexpr (std::is_same<T, float>::value) {
    const int w4 = width / 4;
    for (int e = threadIdx.x; e < C * w4; e += THREADS) {
      const int r = e / w4, c = 4 * (e - r * w4);
      ptx::cp_async16_zfill(dst + r * ld + c, src + (t0 + (r < L ? r : 0)) * stride + c, r < L ? 16u : 0u);
    }
  } else {
    load_rows(src, stride, t0, L, C, width, dst, ld);
  }
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float acc) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, acc))));
}

// ------------------------------------------------------------------------------- gprep -----
// Thread tile of the C x C products: TS x TS entries, 16 x 16 threads.
template <typename T, int C>
__global__ void __launch_bounds__(THREADS) gprep_kernel(const SimtArgs P) {
  extern __shared__ __align__(16) float sm[];
  constexpr int ldc = C + 4, TS = C / 16, RG = C / 4;
  const int ldk = P.dk + 4;
  float* Ks = sm;
  float* Qs = Ks + C * ldk;
  float* KK = Qs + C * ldk;
  float* QK = KK + C * ldc;
  float* At = QK + C * ldc;      // A transposed
  float* line = At + C * ldc;    // [2][C]
  float* bet = line + 2 * C;
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
  {
    const int rb = TS * (tid / 16), sb = TS * (tid % 16);
    if (sb <= rb) {
      float a[TS][TS] = {}, b[TS][TS] = {};
      for (int i = 0; i < P.dk; i += 4) {
        float4 ks[TS];
#pragma unroll
        for (int y = 0; y < TS; ++y) ks[y] = *reinterpret_cast<const float4*>(Ks + (sb + y) * ldk + i);
#pragma unroll
        for (int x = 0; x < TS; ++x) {
          const float4 kr = *reinterpret_cast<const float4*>(Ks + (rb + x) * ldk + i);
          const float4 qr = *reinterpret_cast<const float4*>(Qs + (rb + x) * ldk + i);
#pragma unroll
          for (int y = 0; y < TS; ++y) {
            a[x][y] = dot4(kr, ks[y], a[x][y]);
            b[x][y] = dot4(qr, ks[y], b[x][y]);
          }
        }
      }
#pragma unroll
      for (int x = 0; x < TS; ++x)
#pragma unroll
        for (int y = 0; y < TS; ++y) {
          KK[(rb + x) * ldc + sb + y] = a[x][y];
          QK[(rb + x) * ldc + sb + y] = b[x][y];
        }
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
      const int r = e / C, s = e % C;
      const float ex = s <= r ? expf((float)(gam[r] - gam[s])) : 0.0f;
      At[s * ldc + r] = s < r ? bet[r] * ex * KK[r * ldc + s] : 0.0f;
      tp[C * C + e] = s <= r ? ex * QK[r * ldc + s] : 0.0f;
    }
    __syncthreads();
    // T = (I + A)^{-1} by right-looking substitution: a thread holds C / 4 consecutive rows of one column;
    // row s, once final, is handed to everybody and taken off the later rows
    const int g = tid / 64, c = tid % 64;
    const bool on = c < C;
    float x[RG];
#pragma unroll
    for (int q = 0; q < RG; ++q) x[q] = g * RG + q == c ? 1.0f : 0.0f;
    for (int og = 0; og < 4; ++og) {
#pragma unroll
      for (int q = 0; q < RG; ++q) {
        const int s = og * RG + q;
        float* ln = line + (s & 1) * C;
        if (g == og && on) ln[c] = x[q];
        __syncthreads();
        if (on && g >= og) {
          const float t = ln[c];
#pragma unroll
          for (int k = 0; k < RG; k += 4) {
            const float4 a = *reinterpret_cast<const float4*>(At + s * ldc + g * RG + k);
            x[k] = fmaf(-a.x, t, x[k]);  // A is zero on and above the diagonal
            x[k + 1] = fmaf(-a.y, t, x[k + 1]);
            x[k + 2] = fmaf(-a.z, t, x[k + 2]);
            x[k + 3] = fmaf(-a.w, t, x[k + 3]);
          }
        }
      }
    }
    if (on)
#pragma unroll
      for (int q = 0; q < RG; ++q) tp[(g * RG + q) * C + c] = c <= g * RG + q ? x[q] * bet[c] : 0.0f;
  }
}

// ------------------------------------------------------------------------------- gwalk -----
// Block = (sequence, v-head, 16 value rows, direction).  A chunk's inputs lie in one of `stages` buffers: with
// two, which fp32 inputs get where two blocks still fit an SM, the next chunk's copies run beside this one's
// products.
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

// Thread (j = tid % 16, rg = tid / 16) holds rows rg, rg + 16, .. of one value column j.
// acc[m] += sum_i A[rg + 16 m][i] B[i] over rows of A in shared memory (float4 steps)
template <int R>
__device__ __forceinline__ void rows_dot(const float* A, int lda, const float* b, int n, int rg,
                                         float (&acc)[R]) {
#pragma unroll 4
  for (int i = 0; i < n; i += 4) {
    const float4 v = *reinterpret_cast<const float4*>(b + i);
#pragma unroll
    for (int m = 0; m < R; ++m)
      acc[m] = dot4(*reinterpret_cast<const float4*>(A + (rg + 16 * m) * lda + i), v, acc[m]);
  }
}
// acc[m] += sum_s A[rg + 16 m][s] B[s][j]
template <int R, int C>
__device__ __forceinline__ void rows_mul(const float* A, const float* B, int rg, int j,
                                         float (&acc)[R]) {
#pragma unroll 4
  for (int s = 0; s < C; s += 4) {
    float b[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) b[q] = B[(s + q) * DVS + j];
#pragma unroll
    for (int m = 0; m < R; ++m) {
      const float4 a = *reinterpret_cast<const float4*>(A + (rg + 16 * m) * (C + 4) + s);
      acc[m] = fmaf(a.x, b[0], fmaf(a.y, b[1], fmaf(a.z, b[2], fmaf(a.w, b[3], acc[m]))));
    }
  }
}
// acc[m] += sum_r A[r][rg + 16 m] B[r][j]
template <int R, int C>
__device__ __forceinline__ void cols_mul(const float* A, const float* B, int rg, int j,
                                         float (&acc)[R]) {
#pragma unroll 8
  for (int r = 0; r < C; ++r) {
    const float b = B[r * DVS + j];
#pragma unroll
    for (int m = 0; m < R; ++m) acc[m] = fmaf(A[r * (C + 4) + rg + 16 * m], b, acc[m]);
  }
}

template <typename T, int C>
__device__ __forceinline__ void walk_forward(const SimtArgs& P, const Walk& W, float* sm) {
  constexpr int ldc = C + 4, R = C / 16;
  const int ldk = P.dk + 4, tid = threadIdx.x;
  float* Ss = sm;                 // [DVS][ldk]
  float* Us = Ss + DVS * ldk;     // [C][DVS]
  float* buf = Us + C * DVS;      // K [C][ldk], T' [C][ldc], V then W [C][DVS], Gamma and d [2][C]
  const int stage = C * (ldk + ldc + DVS + 2);
  const SimtWs w = simt_ws(P.ws, P.slots, P.Hv, P.dk, P.dv, C);
  const int64_t sbase = ((int64_t)W.n * P.Hv + W.h) * P.dv * P.dk + (int64_t)W.j0 * P.dk;
  const int w4 = P.dk / 4, jst = THREADS / w4, sj = tid / w4, si = 4 * (tid - sj * w4);
  const int j = tid % DVS, rg = tid / DVS;
  for (int jj = sj; sj < jst && jj < DVS; jj += jst)
    *reinterpret_cast<float4*>(Ss + jj * ldk + si) =
        P.S0 ? *reinterpret_cast<const float4*>(P.S0 + sbase + jj * P.dk + si)
             : make_float4(0.f, 0.f, 0.f, 0.f);
  auto fetch = [&](int64_t c) {
    const int64_t t0 = W.s_beg + c * C, sh = (W.slot0 + c) * P.Hv + W.h;
    const int L = (int)min((int64_t)C, W.s_end - t0);
    float* b = buf + (P.stages == 2 ? (c & 1) * stage : 0);
    fetch_rows((const T*)P.k + W.hk * P.dk, P.ts.k, t0, L, C, P.dk, b, ldk);
    b += C * ldk;
    fetch_rows<float>(w.tp + sh * 2 * C * C, C, 0, C, C, C, b, ldc);
    b += C * ldc;
    fetch_rows((const T*)P.v + W.h * P.dv + W.j0, P.ts.v, t0, L, C, DVS, b, DVS);
    fetch_rows<float>(w.rec + sh * 5 * C, 0, 0, 1, 1, 2 * C, b + C * DVS, 2 * C);
  };
  if (W.nch > 0) fetch(0);
  for (int64_t c = 0; c < W.nch; ++c) {
    const int64_t sh = (W.slot0 + c) * P.Hv + W.h;
    float* Ks = buf + (P.stages == 2 ? (c & 1) * stage : 0);
    float *Ts = Ks + C * ldk, *Ws = Ts + C * ldc, *Gm = Ws + C * DVS, *dd = Gm + C;
    if (P.stages == 1 && c > 0) {
      __syncthreads();
      fetch(c);
    }
    ptx::cp_async_wait_all();
    __syncthreads();
    if (P.stages == 2 && c + 1 < W.nch) fetch(c + 1);
    float* So = w.S + sh * P.dv * P.dk + W.j0 * P.dk;
    for (int jj = sj; sj < jst && jj < DVS; jj += jst)
      *reinterpret_cast<float4*>(So + jj * P.dk + si) = *reinterpret_cast<float4*>(Ss + jj * ldk + si);
    {  // W = V - Gamma K S^T
      float acc[R] = {};
      rows_dot<R>(Ks, ldk, Ss + j * ldk, P.dk, rg, acc);
#pragma unroll
      for (int m = 0; m < R; ++m) Ws[(rg + 16 * m) * DVS + j] -= Gm[rg + 16 * m] * acc[m];
    }
    __syncthreads();
    {  // U = T' W
      float acc[R] = {};
      rows_mul<R, C>(Ts, Ws, rg, j, acc);
#pragma unroll
      for (int m = 0; m < R; ++m) {
        const int r = rg + 16 * m;
        Us[r * DVS + j] = acc[m] * dd[r];
        w.U[sh * C * P.dv + r * P.dv + W.j0 + j] = acc[m];
      }
    }
    __syncthreads();
    const float gl = Gm[C - 1];
    for (int jj = sj; sj < jst && jj < DVS; jj += jst) {
      float4 a = *reinterpret_cast<float4*>(Ss + jj * ldk + si);
      a.x *= gl; a.y *= gl; a.z *= gl; a.w *= gl;
#pragma unroll 8
      for (int s = 0; s < C; ++s) {
        const float u = Us[s * DVS + jj];
        const float4 kv = *reinterpret_cast<const float4*>(Ks + s * ldk + si);
        a.x = fmaf(u, kv.x, a.x); a.y = fmaf(u, kv.y, a.y);
        a.z = fmaf(u, kv.z, a.z); a.w = fmaf(u, kv.w, a.w);
      }
      *reinterpret_cast<float4*>(Ss + jj * ldk + si) = a;
    }
  }
}

template <typename T, int C>
__device__ __forceinline__ void walk_backward(const SimtArgs& P, const Walk& W, float* sm) {
  constexpr int ldc = C + 4, R = C / 16;
  const int ldk = P.dk + 4, tid = threadIdx.x;
  float* Ss = sm;              // [DVS][ldk] dS
  float* Us = Ss + DVS * ldk;  // [C][DVS] dU
  float* Ws = Us + C * DVS;    // [C][DVS] -Gamma dW
  // K, Q [C][ldk], T', P [C][ldc], dO' then Gamma dO' [C][DVS], Gamma, d, beta [3][C]
  float* buf = Ws + C * DVS;
  const int stage = C * (2 * ldk + 2 * ldc + DVS + 3);
  const SimtWs w = simt_ws(P.ws, P.slots, P.Hv, P.dk, P.dv, C);
  const int64_t sbase = ((int64_t)W.n * P.Hv + W.h) * P.dv * P.dk + (int64_t)W.j0 * P.dk;
  const int w4 = P.dk / 4, jst = THREADS / w4, sj = tid / w4, si = 4 * (tid - sj * w4);
  const int j = tid % DVS, rg = tid / DVS;
  for (int jj = sj; sj < jst && jj < DVS; jj += jst)
    *reinterpret_cast<float4*>(Ss + jj * ldk + si) =
        P.dST ? *reinterpret_cast<const float4*>(P.dST + sbase + jj * P.dk + si)
              : make_float4(0.f, 0.f, 0.f, 0.f);
  auto fetch = [&](int64_t c) {
    const int64_t t0 = W.s_beg + c * C, sh = (W.slot0 + c) * P.Hv + W.h;
    const int L = (int)min((int64_t)C, W.s_end - t0);
    float* b = buf + (P.stages == 2 ? (c & 1) * stage : 0);
    fetch_rows((const T*)P.k + W.hk * P.dk, P.ts.k, t0, L, C, P.dk, b, ldk);
    b += C * ldk;
    fetch_rows((const T*)P.q + W.hk * P.dk, P.ts.q, t0, L, C, P.dk, b, ldk);
    b += C * ldk;
    fetch_rows<float>(w.tp + sh * 2 * C * C, C, 0, 2 * C, 2 * C, C, b, ldc);  // T', P
    b += 2 * C * ldc;
    fetch_rows((const T*)P.dout + W.h * P.dv + W.j0, (int64_t)P.Hv * P.dv, t0, L, C, DVS, b, DVS);
    fetch_rows<float>(w.rec + sh * 5 * C, 0, 0, 1, 1, 3 * C, b + C * DVS, 3 * C);
  };
  if (W.nch > 0) fetch(W.nch - 1);
  for (int64_t c = W.nch - 1; c >= 0; --c) {
    const int64_t t0 = W.s_beg + c * C, sh = (W.slot0 + c) * P.Hv + W.h;
    const int L = (int)min((int64_t)C, W.s_end - t0);
    float* Ks = buf + (P.stages == 2 ? (c & 1) * stage : 0);
    float *Qs = Ks + C * ldk, *Ts = Qs + C * ldk, *Ps = Ts + C * ldc, *Os = Ps + C * ldc;
    float *Gm = Os + C * DVS, *dd = Gm + C, *bet = dd + C;
    if (P.stages == 1 && c < W.nch - 1) {
      __syncthreads();
      fetch(c);
    }
    ptx::cp_async_wait_all();
    for (int e = 4 * tid; e < C * DVS; e += 4 * THREADS) {  // this thread's own part of dO
      float4 o = *reinterpret_cast<float4*>(Os + e);
      o.x *= P.scale; o.y *= P.scale; o.z *= P.scale; o.w *= P.scale;
      *reinterpret_cast<float4*>(Os + e) = o;
    }
    __syncthreads();
    if (P.stages == 2 && c > 0) fetch(c - 1);
    float* So = w.dS + sh * P.dv * P.dk + W.j0 * P.dk;
    for (int jj = sj; sj < jst && jj < DVS; jj += jst)
      *reinterpret_cast<float4*>(So + jj * P.dk + si) = *reinterpret_cast<float4*>(Ss + jj * ldk + si);
    {  // dU = P^T dO' + d K dS^T
      float acc[R] = {};
      rows_dot<R>(Ks, ldk, Ss + j * ldk, P.dk, rg, acc);
#pragma unroll
      for (int m = 0; m < R; ++m) acc[m] *= dd[rg + 16 * m];
      cols_mul<R, C>(Ps, Os, rg, j, acc);
#pragma unroll
      for (int m = 0; m < R; ++m) Us[(rg + 16 * m) * DVS + j] = acc[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < R; ++m) Os[(rg + 16 * m) * DVS + j] *= Gm[rg + 16 * m];
    {  // dW = T'^T dU
      float acc[R] = {};
      cols_mul<R, C>(Ts, Us, rg, j, acc);
#pragma unroll
      for (int m = 0; m < R; ++m) {
        const int s = rg + 16 * m;
        Ws[s * DVS + j] = -Gm[s] * acc[m];
        w.dW[sh * C * P.dv + s * P.dv + W.j0 + j] = acc[m];
        if (s < L) {
          const float bf = bet[s];
          float out = acc[m];
          if (fabsf(bf) == kBetaFloor) out *= P.beta[(t0 + s) * P.Hv + W.h] / bf;  // T' used the floor
          ((T*)P.dv_)[((t0 + s) * P.Hv + W.h) * P.dv + W.j0 + j] = from_f<T>(out);
        }
      }
    }
    __syncthreads();
    const float gl = Gm[C - 1];
    for (int jj = sj; sj < jst && jj < DVS; jj += jst) {
      float4 a = *reinterpret_cast<float4*>(Ss + jj * ldk + si);
      a.x *= gl; a.y *= gl; a.z *= gl; a.w *= gl;
#pragma unroll 8
      for (int s = 0; s < C; ++s) {
        const float u = Os[s * DVS + jj], x = Ws[s * DVS + jj];
        const float4 qv = *reinterpret_cast<const float4*>(Qs + s * ldk + si);
        const float4 kv = *reinterpret_cast<const float4*>(Ks + s * ldk + si);
        a.x = fmaf(u, qv.x, fmaf(x, kv.x, a.x)); a.y = fmaf(u, qv.y, fmaf(x, kv.y, a.y));
        a.z = fmaf(u, qv.z, fmaf(x, kv.z, a.z)); a.w = fmaf(u, qv.w, fmaf(x, kv.w, a.w));
      }
      *reinterpret_cast<float4*>(Ss + jj * ldk + si) = a;
    }
  }
  __syncthreads();
  if (P.dS0)
    for (int jj = sj; sj < jst && jj < DVS; jj += jst)
      *reinterpret_cast<float4*>(P.dS0 + sbase + jj * P.dk + si) =
          *reinterpret_cast<float4*>(Ss + jj * ldk + si);
}

template <typename T, int C>
__global__ void __launch_bounds__(THREADS) gwalk_kernel(const SimtArgs P) {
  extern __shared__ __align__(16) float sm[];
  Walk W;
  if (!walk_of(P, W)) return;
  if (blockIdx.x & 1)
    walk_forward<T, C>(P, W, sm);
  else
    walk_backward<T, C>(P, W, sm);
}

// ------------------------------------------------------------------------------- ggrad -----
// CW (a power of two >= dk / 4) neighbouring threads share RPT rows; each holds 4 columns of dq, dKe, dKw.
// Blocks an SM that the registers leave room for: with one row a thread (dk up to 32) three are 4 % of a call of
// 4096 tokens faster than two, with more rows one with all its registers is faster than two by 1 %.
template <typename T, int C, int RPT>
__global__ void __launch_bounds__(THREADS, C == 16 ? 2 : RPT == 1 ? 3 : 1) ggrad_kernel(const SimtArgs P, int CW) {
  extern __shared__ __align__(16) float sm[];
  constexpr int ldc = C + 4, TS = C / 16;
  const int ldk = P.dk + 4, ldv = P.dv + 4, tid = threadIdx.x;
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
  const int rg = tid / CW, r0 = RPT * rg, c0 = 4 * (tid - rg * CW);
  const bool rows_on = r0 < C, on = rows_on && c0 < P.dk;
  // sum over the threads that share a row (all lanes take part)
  auto row_sum = [&](float v) {
    for (int o = CW >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  float dq[RPT][4] = {}, dk[RPT][4] = {};  // summed over the v-heads
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
    float frob = 0.0f;
    for (int e = 4 * tid; e < P.dv * P.dk; e += 4 * THREADS)
      frob = dot4(*reinterpret_cast<const float4*>(S + e), *reinterpret_cast<const float4*>(dS + e),
                  frob);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) frob += __shfl_xor_sync(0xffffffffu, frob, o);
    if (lane == 0) red[warp] = frob;
    __syncthreads();
    // dN, dM (zero on and above the diagonal), p and dbeta: TS x TS entries a thread
    {
      const int rb = TS * (tid / 16), sb = TS * (tid % 16);
      float a[TS][TS] = {}, b[TS][TS] = {};
      if (sb <= rb) {
        for (int jx = 0; jx < P.dv; jx += 4) {
          float4 u[TS];
#pragma unroll
          for (int y = 0; y < TS; ++y) u[y] = *reinterpret_cast<const float4*>(Us + (sb + y) * ldv + jx);
#pragma unroll
          for (int x = 0; x < TS; ++x) {
            const float4 o = *reinterpret_cast<const float4*>(Os + (rb + x) * ldv + jx);
            const float4 d = *reinterpret_cast<const float4*>(Ws + (rb + x) * ldv + jx);
#pragma unroll
            for (int y = 0; y < TS; ++y) {
              a[x][y] = dot4(o, u[y], a[x][y]);
              b[x][y] = dot4(d, u[y], b[x][y]);
            }
          }
        }
      }
#pragma unroll
      for (int x = 0; x < TS; ++x)
#pragma unroll
        for (int y = 0; y < TS; ++y) {
          const int r = rb + x, s = sb + y;
          const float e = s < r ? expf((float)(gam[r] - gam[s])) : 0.0f;
          Ns[r * ldc + s] = e * a[x][y];
          Ms[r * ldc + s] = -e * b[x][y];
          if (s == r) {
            own[r] = a[x][y];
            if (r < L)
              ((T*)P.dbeta)[(t0 + r) * P.Hv + h] = from_f<T>(b[x][y] / bet[r] / bet[r]);
          }
        }
    }
    __syncthreads();
    float aq[RPT][4] = {}, ae[RPT][4] = {}, aw[RPT][4] = {};
    if (on) {
      // unrolled for the latency of the state loads (from L2), as far as registers allow
#pragma unroll(RPT <= 2 ? 4 : 1)
      for (int jx = 0; jx < P.dv; jx += 4) {
        float4 s4[4], d4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          s4[q] = *reinterpret_cast<const float4*>(S + (jx + q) * P.dk + c0);
          d4[q] = *reinterpret_cast<const float4*>(dS + (jx + q) * P.dk + c0);
        }
#pragma unroll
        for (int x = 0; x < RPT; ++x) {
          const float4 o4 = *reinterpret_cast<const float4*>(Os + (r0 + x) * ldv + jx);
          const float4 w4 = *reinterpret_cast<const float4*>(Ws + (r0 + x) * ldv + jx);
          const float4 u4 = *reinterpret_cast<const float4*>(Us + (r0 + x) * ldv + jx);
          const float o[4] = {o4.x, o4.y, o4.z, o4.w}, ww[4] = {w4.x, w4.y, w4.z, w4.w},
                      u[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float sv[4] = {s4[q].x, s4[q].y, s4[q].z, s4[q].w};
            const float dv[4] = {d4[q].x, d4[q].y, d4[q].z, d4[q].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              aq[x][y] = fmaf(o[q], sv[y], aq[x][y]);
              ae[x][y] = fmaf(ww[q], sv[y], ae[x][y]);
              aw[x][y] = fmaf(u[q], dv[y], aw[x][y]);
            }
          }
        }
      }
#pragma unroll
      for (int x = 0; x < RPT; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          aq[x][y] *= Gm[r0 + x];
          ae[x][y] *= -Gm[r0 + x];
          aw[x][y] *= dd[r0 + x];
        }
    }
#pragma unroll
    for (int x = 0; x < RPT; ++x) {
      float v = 0.0f;
      if (on)
        v = dot4(*reinterpret_cast<const float4*>(Ks + (r0 + x) * ldk + c0),
                 make_float4(aw[x][0], aw[x][1], aw[x][2], aw[x][3]), 0.0f);
      v = row_sum(v);
      if (rows_on && c0 == 0) kw[r0 + x] = v;
#pragma unroll
      for (int y = 0; y < 4; ++y) {  // the state's part stays out of dgamma
        dk[x][y] += aw[x][y];
        aw[x][y] = 0.0f;
      }
    }
    if (on) {
#pragma unroll 2
      for (int s = 0; s < r0 + RPT; s += 4) {  // these rows against earlier tokens (C is a multiple of 4)
        float4 k4[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) k4[q] = *reinterpret_cast<const float4*>(Ks + (s + q) * ldk + c0);
#pragma unroll
        for (int x = 0; x < RPT; ++x) {
          const float4 n4 = *reinterpret_cast<const float4*>(Ns + (r0 + x) * ldc + s);
          const float4 m4 = *reinterpret_cast<const float4*>(Ms + (r0 + x) * ldc + s);
          const float nn[4] = {n4.x, n4.y, n4.z, n4.w}, mm[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float kv[4] = {k4[q].x, k4[q].y, k4[q].z, k4[q].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              aq[x][y] = fmaf(nn[q], kv[y], aq[x][y]);
              ae[x][y] = fmaf(mm[q], kv[y], ae[x][y]);
            }
          }
        }
      }
#pragma unroll 4
      for (int r = r0; r < C; ++r) {  // and later tokens
        const float4 k4 = *reinterpret_cast<const float4*>(Ks + r * ldk + c0);
        const float4 q4 = *reinterpret_cast<const float4*>(Qs + r * ldk + c0);
        const float kv[4] = {k4.x, k4.y, k4.z, k4.w}, qv[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int x = 0; x < RPT; ++x) {
          const float nn = Ns[r * ldc + r0 + x], mm = Ms[r * ldc + r0 + x];
#pragma unroll
          for (int y = 0; y < 4; ++y) aw[x][y] = fmaf(nn, qv[y], fmaf(mm, kv[y], aw[x][y]));
        }
      }
    }
#pragma unroll
    for (int x = 0; x < RPT; ++x) {
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
      v = row_sum(v);
      if (rows_on && c0 == 0) dgm[r] = v;
    }
    __syncthreads();
    // dg: suffix sums, and what leaves through the state
    if (warp == 0) {
      float f = 0.0f;
      for (int x = 0; x < THREADS / 32; ++x) f += red[x];
      f *= Gm[C - 1];
      // kappa, summed over earlier tokens
      float k0 = lane < L ? kw[lane] : 0.0f;
      float a0 = lane < L ? dgm[lane] : 0.0f;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float l0 = __shfl_up_sync(0xffffffffu, k0, o);
        const float u0 = __shfl_down_sync(0xffffffffu, a0, o);
        if (lane >= o) k0 += l0;
        if (lane + o < 32) a0 += u0;
      }
      k0 = __shfl_up_sync(0xffffffffu, k0, 1);
      k0 = lane > 0 ? k0 : 0.0f;
      // the first token's decay multiplies the initial state: without one its gradient is zero, where the pairs
      // in a0 cancel only up to their rounding
      const bool none = ch.first && !P.S0 && lane == 0;
      if (lane < L) ((T*)P.dg)[(t0 + lane) * P.Hv + h] = from_f<T>(none ? 0.0f : a0 + f + k0);
    }
  }
  if (on) {
#pragma unroll
    for (int x = 0; x < RPT; ++x) {
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

template <typename T, int C, int RPT>
cudaError_t launch_grad(const SimtArgs& P, int cw, int64_t par, size_t bytes, cudaStream_t s) {
  const cudaError_t e = allow_smem(ggrad_kernel<T, C, RPT>, bytes);
  if (e != cudaSuccess) return e;
  ggrad_kernel<T, C, RPT><<<(unsigned)par, THREADS, bytes, s>>>(P, cw);
  return cudaGetLastError();
}

template <typename T, int C>
cudaError_t launch_c(SimtArgs P, cudaStream_t s) {
  const int ldk = P.dk + 4, ldv = P.dv + 4, ldc = C + 4;
  const size_t f = sizeof(float);
  const size_t sm_prep = (2 * (size_t)C * ldk + 3 * C * ldc + 3 * C) * f + C * 8;
  // the backward walk's; the forward one needs less
  const size_t stage = (size_t)C * (2 * ldk + 2 * ldc + DVS + 3) * f, rest = ((size_t)DVS * ldk + 2 * C * DVS) * f;
  const bool two = std::is_same<T, float>::value && rest + 2 * stage <= 113 * 1024;
  const size_t sm_walk = rest + (two ? 2 : 1) * stage;
  P.stages = two ? 2 : 1;
  const size_t sm_grad =
      (2 * (size_t)C * ldk + 3 * C * ldv + 2 * C * ldc + 6 * C + 8) * f + C * 8;
  cudaError_t e = allow_smem(gprep_kernel<T, C>, sm_prep);
  if (e == cudaSuccess) e = allow_smem(gwalk_kernel<T, C>, sm_walk);
  if (e != cudaSuccess) return e;
  const int64_t par = P.slots * P.Hk, walks = 2 * (int64_t)P.N * P.Hv * (P.dv / DVS);
  if (par > 0x7fffffff || walks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (par > 0) gprep_kernel<T, C><<<(unsigned)par, THREADS, sm_prep, s>>>(P);
  if (walks > 0) gwalk_kernel<T, C><<<(unsigned)walks, THREADS, sm_walk, s>>>(P);
  e = cudaGetLastError();
  if (par == 0 || e != cudaSuccess) return e;
  int cw = 4;
  while (4 * cw < P.dk) cw *= 2;
  switch (C * cw / THREADS) {  // rows a thread
    case 4: return launch_grad<T, C, C == 32 ? 4 : 1>(P, cw, par, sm_grad, s);
    case 2: return launch_grad<T, C, 2>(P, cw, par, sm_grad, s);
    default: return launch_grad<T, C, 1>(P, cw, par, sm_grad, s);
  }
}

template <typename T>
cudaError_t launch_t(const SimtArgs& P, cudaStream_t s) {
  return P.C == 32 ? launch_c<T, 32>(P, s) : launch_c<T, 16>(P, s);
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
