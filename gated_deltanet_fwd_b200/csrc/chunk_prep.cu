// chunk_prep.cu -- the state-independent half of the tensor-core prefill (bf16, dk = dv = 128,
// chunks of 64 tokens), fully parallel over (chunk, k-head).
//
// Method: the chunked parallel mode of "解密Qwen3-Next的Gated DeltaNet：如何用75%混合层实现长文本
// 高效推理" §2.2 applied to the gated delta rule.  Inside a chunk of L <= 64 tokens with in-chunk
// cumulative log-decays gamma_r, everything that does not depend on the state entering the chunk
// is fixed by the chunk's own keys, queries and gates:
//   A[r,s] = beta_r e^{gamma_r - gamma_s} k_r.k_s   (s < r),     T' = (I + A)^{-1} diag(beta)
//   P[r,s] = e^{gamma_r - gamma_s} q_r.k_s          (s <= r)
//   Gamma_r = e^{gamma_r},   d_s = e^{gamma_63 - gamma_s}
// so that, for a chunk entering with state S0, the corrected values are U = T'(V - diag(Gamma) K
// S0^T), the outputs scale (diag(Gamma) Q S0^T + P U) and the leaving state Gamma_63 S0 +
// U^T diag(d) K -- the chain kernel (chunk_chain.cu) evaluates those.  Only differences of
// cumulative log-decays are exponentiated, so nothing over- or underflows; rows past a sequence
// end read zero keys, queries, log-decay and beta, which makes their rows of T' and P zero.
//
// One CTA per (chunk slot, k-head): K and Q are loaded once and [K; Q] K^T is one tcgen05 MMA
// (M = 128, N = 64, K-dim 128, fp32 in tensor memory); the Hv/Hk v-heads that share the k-head
// then take their own gates: the decay masks are applied straight out of tensor memory, and
// I + A is inverted in fp32 by two warpgroups at once (one v-head each: forward substitution on
// the four 16 x 16 diagonal blocks, one column per lane, then the off-diagonal blocks by distance
// with tf32 mma.sync block products).  T', P, Gamma and d go to the workspace (layout in
// chunk_tm.cuh).
//
// For the backward pass (BWD; bwd_tc.cuh) the same inverse is written as T' = diag(beta) T~ with
// T~ = (I + A~)^{-1}, A~[r,s] = e^{gamma_r - gamma_s} beta_s k_r.k_s: T~ has an exact unit diagonal, so
// its bf16 copy loses only what the small off-diagonal entries lose, and beta is applied in fp32 by
// whoever uses it.  The record then holds Gamma, d, beta and gamma log2 e, P carries the
// output scale, and scale Gamma Q goes out next to it (operands of the backward chain, where scaling Q
// cost 1400 cycles of a chunk).  8192 (chunk, k-head) items of two v-heads: 250 us, some 14000 cycles an
// item beside another one on the SM -- a third the solve, then masks, scale Gamma Q and T~ -- where its 0.8 GB
// would take 123 us.
#include "bwd_internal.cuh"
#include "chunk_tm.cuh"
#include "gdn_internal.cuh"
#include "ptx.cuh"

namespace gdn {
namespace {

using namespace ptx;

constexpr int PP_THREADS = 256;  // two warpgroups
constexpr int AS = 68;           // fp32 row stride of the A and T matrices
constexpr int PS = 144;          // byte stride of P's rows on their way out (BWD; in T's place)
constexpr int MS = 20;           // fp32 row stride of the 16 x 16 block-product scratch
constexpr int PAIR = 2;          // v-heads solved side by side (one per warpgroup)

constexpr uint32_t PP_KQ = 0;                                 // [K; Q]: 2 halves x 128 x 128 B
constexpr uint32_t PP_A = 32768;                              // PAIR x fp32 [64][AS]
constexpr uint32_t PP_T = PP_A + PAIR * 64 * AS * 4;          // PAIR x fp32 [64][AS]
constexpr uint32_t PP_MB = PP_T + PAIR * 64 * AS * 4;         // PAIR x 4 x fp32 [16][MS]
constexpr uint32_t PP_GB = PP_MB + PAIR * 4 * 16 * MS * 4;    // PAIR x (gamma log2e [64], beta [64])
constexpr uint32_t PP_BAR = PP_GB + PAIR * 128 * 4;           // mbarrier, tensor-memory slot
constexpr uint32_t PP_SMEM = PP_BAR + 64 + 1024;              // + slack for 1024-byte alignment
// two CTAs per SM: the SM's 228 KB of shared memory less 1 KB the hardware reserves per CTA
static_assert(PP_SMEM <= 228 * 1024 / 2 - 1024, "two prep CTAs per SM");

constexpr float kLog2e = 1.4426950408889634f;

// Optional phase timing, compiled in only with -DGDN_PREP_TRACE: globaltimer stamps (ns) of every
// work item, 8 slots per item, written to PrepParams::trace.
#ifdef GDN_PREP_TRACE
#define PP_TS(k)                                                                   \
  do {                                                                             \
    if (P.trace && tid == 0) P.trace[(size_t)cur.it * 8 + (k)] = globaltimer_ns(); \
  } while (0)
#else
#define PP_TS(k) \
  do {           \
  } while (0)
#endif

struct PrepParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const float* g;
  const float* beta;
  const int32_t* cu;
  unsigned char* ws;  // workspace base
  int* status;
  int64_t q_stride, k_stride;  // elements between consecutive tokens
  int64_t T;
  int64_t gd_off;  // byte offset of the GD array
  int N, Hk, Hv;
  unsigned long long* trace;  // phase timing (trace builds only), else unused
  int debug_thread;  // failure-test builds only: this thread's first wait counts as run out
  // fused gates: g and beta computed here from a, b (bf16) when a is set
  const __nv_bfloat16* a;
  const __nv_bfloat16* b;
  const float* A_log;
  const float* dt_bias;
  // backward: byte offset of the scale Gamma Q tiles
  int64_t qg_off;
  float scale;
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// T = (I + A)^{-1} for the unit lower-triangular I + A (A strictly lower, fp32 [64][AS]) by one
// warpgroup (w4 = warp within the group, bar = its named barrier).  Tf receives the lower triangle
// and the unit diagonal; above the diagonal it is left unwritten.
__device__ __forceinline__ void solve64(int bar, const float* Af, float* Tf, float* Mb, int w4, int lane) {
  // diagonal 16 x 16 blocks: right-looking forward substitution, one column per lane
  if (w4 < 2) {
    const int blk = 2 * w4 + (lane >> 4), jj = lane & 15, col = 16 * blk + jj;
    const float* ab = Af + 16 * blk * AS + 16 * blk;
    float x[16], a[16], an[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) x[r] = (r == jj) ? 1.0f : 0.0f;
#pragma unroll
    for (int t = 1; t < 16; ++t) a[t] = ab[t * AS];
#pragma unroll
    for (int r = 0; r < 15; ++r) {
#pragma unroll
      for (int t = r + 2; t < 16; ++t) an[t] = ab[t * AS + r + 1];  // next column, early
#pragma unroll
      for (int t = r + 1; t < 16; ++t) x[t] = fmaf(-a[t], x[r], x[t]);
#pragma unroll
      for (int t = r + 2; t < 16; ++t) a[t] = an[t];
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) Tf[(16 * blk + r) * AS + col] = x[r];
  }
  named_bar(bar, 128);
  // off-diagonal blocks by distance:  T_ij = -T_ii sum_{k=j}^{i-1} A_ik T_kj
  if (w4 >= 1) {  // distance 1: block (w4, w4 - 1)
    const int i = w4, j = w4 - 1;
    float acc[2][4] = {};
    warp_mm16(Af + 16 * i * AS + 16 * j, AS, Tf + 16 * j * AS + 16 * j, AS, acc, lane);
    float* Mi = Mb + i * 16 * MS;
    warp_store16(Mi, MS, acc, 1.0f, lane);
    __syncwarp();
    float t2[2][4] = {};
    warp_mm16(Tf + 16 * i * AS + 16 * i, AS, Mi, MS, t2, lane);
    warp_store16(Tf + 16 * i * AS + 16 * j, AS, t2, -1.0f, lane);
  }
  named_bar(bar, 128);
  if (w4 >= 2) {  // distance 2: blocks (2,0), (3,1)
    const int i = w4, j = w4 - 2;
    float acc[2][4] = {};
    warp_mm16(Af + 16 * i * AS + 16 * j, AS, Tf + 16 * j * AS + 16 * j, AS, acc, lane);
    warp_mm16(Af + 16 * i * AS + 16 * (j + 1), AS, Tf + 16 * (j + 1) * AS + 16 * j, AS, acc,
              lane);
    float* Mi = Mb + i * 16 * MS;
    warp_store16(Mi, MS, acc, 1.0f, lane);
    __syncwarp();
    float t2[2][4] = {};
    warp_mm16(Tf + 16 * i * AS + 16 * i, AS, Mi, MS, t2, lane);
    warp_store16(Tf + 16 * i * AS + 16 * j, AS, t2, -1.0f, lane);
  } else if (w4 == 0) {  // meanwhile the known part of block (3,0): A_30 T_00 + A_31 T_10
    float acc[2][4] = {};
    warp_mm16(Af + 48 * AS + 0, AS, Tf + 0 * AS + 0, AS, acc, lane);
    warp_mm16(Af + 48 * AS + 16, AS, Tf + 16 * AS + 0, AS, acc, lane);
    warp_store16(Mb, MS, acc, 1.0f, lane);
  }
  named_bar(bar, 128);
  if (w4 == 3) {  // distance 3: block (3,0)
    float acc[2][4];
    {
      const int g = lane >> 2, t = lane & 3;
#pragma unroll
      for (int nn = 0; nn < 2; ++nn) {
        acc[nn][0] = Mb[g * MS + 8 * nn + 2 * t];
        acc[nn][1] = Mb[g * MS + 8 * nn + 2 * t + 1];
        acc[nn][2] = Mb[(g + 8) * MS + 8 * nn + 2 * t];
        acc[nn][3] = Mb[(g + 8) * MS + 8 * nn + 2 * t + 1];
      }
    }
    warp_mm16(Af + 48 * AS + 32, AS, Tf + 32 * AS + 0, AS, acc, lane);
    float* Mi = Mb + 3 * 16 * MS;
    warp_store16(Mi, MS, acc, 1.0f, lane);
    __syncwarp();
    float t2[2][4] = {};
    warp_mm16(Tf + 48 * AS + 48, AS, Mi, MS, t2, lane);
    warp_store16(Tf + 48 * AS + 0, AS, t2, -1.0f, lane);
  }
  named_bar(bar, 128);
}

template <bool BWD>
__global__ void __launch_bounds__(PP_THREADS, 2) chunk_prep_kernel(
    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_q,  // BWD
    const PrepParams P) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + PP_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + PP_BAR + 8);
  uint64_t* lbar = reinterpret_cast<uint64_t*>(smem + PP_BAR + 16);  // BWD: K and Q of a whole chunk

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = P.Hv / P.Hk;
  // BWD: the header's status word and item counter start at zero, without a launch of their own.  What another
  // block reports earlier than this is a malformed cu_seqlens, which the chains meet and report again.
  if (BWD && blockIdx.x == 0 && tid == 0) {
    *P.status = GDN_OK;
    *reinterpret_cast<int*>(P.ws + bwd::COUNTER) = 0;
  }

  // ---- work items (slot, k-head), item = slot * Hk + hk, strided over the persistent CTAs
  struct Item {
    int64_t it, slot, t0, s_end;
    int hk, L;
  };
  // 1: `I` is a chunk; 0: past the last chunk (so is every later item); -1: malformed cu_seqlens
  // (reported; nothing may be read through it).  Uniform across the CTA.
  bwd::ChunkCursor cursor;
  auto locate = [&](int64_t it, Item& I) -> int {
    I.it = it;
    if (BWD) {  // items fit 32 bits (launch_tc); the cursor reads each entry of cu_seqlens once
      I.slot = (uint32_t)it / (uint32_t)P.Hk;
      I.hk = (int)((uint32_t)it - (uint32_t)I.slot * (uint32_t)P.Hk);
      bwd::Chunk ch;
      if (!cursor.find(P.cu, P.T, P.N, tm::C, I.slot, ch, P.status)) return cursor.bad ? -1 : 0;
      I.t0 = ch.t0;
      I.s_end = ch.t0 + ch.L;
      I.L = ch.L;
      return 1;
    }
    I.slot = it / P.Hk;
    I.hk = (int)(it - I.slot * P.Hk);
    int n = -1;
    int64_t s_beg = 0;
    if (!P.cu) {
      const int64_t per = (P.T + tm::C - 1) / tm::C;
      if (per > 0 && I.slot < per * P.N) {
        n = (int)(I.slot / per);
        s_beg = (int64_t)n * P.T;
        I.s_end = s_beg + P.T;
        I.t0 = s_beg + (I.slot - (int64_t)n * per) * tm::C;
      }
    } else {
      int64_t base = 0;
      for (int m = 0; m < P.N; ++m) {
        const int64_t a = P.cu[m], b = P.cu[m + 1];
        if (a < 0 || b < a || b > P.T) {
          if (tid == 0) report(P.status, GDN_ERR_DEVICE_ARG);
          return -1;
        }
        const int64_t nch = (b - a + tm::C - 1) / tm::C;
        if (I.slot < base + nch) {
          n = m;
          I.s_end = b;
          I.t0 = a + (I.slot - base) * tm::C;
          break;
        }
        base += nch;
      }
    }
    if (n < 0) return 0;
    I.L = (int)min((int64_t)tm::C, I.s_end - I.t0);
    return 1;
  };
  // K and Q of an item into the 128-byte-swizzled [K; Q] operand, rows >= L zero-filled:
  // asynchronous per-thread copies (cp.async), waited for before the item's MMA
  auto issue_loads = [&](const Item& I) {
    constexpr int PER = 2 * 64 * 16 / PP_THREADS;
#pragma unroll(BWD ? 1 : PER)
    for (int i = 0; i < PER; ++i) {
      const int e = tid + i * PP_THREADS;
      const int which = e >> 10, r = (e >> 4) & 63, ch = e & 15;
      const int half = ch >> 3, c8 = ch & 7;
      const __nv_bfloat16* src = (which ? P.q + (I.t0 + (r < I.L ? r : 0)) * P.q_stride
                                        : P.k + (I.t0 + (r < I.L ? r : 0)) * P.k_stride) +
                                 I.hk * tm::D + ch * 8;
      cp_async16_zfill(smem + PP_KQ + half * 16384 + which * 8192 + sw128(r, c8 * 8), src,
                       r < I.L ? 16u : 0u);
    }
  };

  // this lane's gate values (tokens lane, 32 + lane) of a v-head
  auto gates = [&](const Item& I, int h, float& x0, float& x1, float& b0, float& b1) {
    const int64_t t0 = I.t0;
    const int L = I.L;
    x0 = x1 = b0 = b1 = 0.f;
    if (!BWD && P.a) {
      // the gates of the layer: beta = sigmoid(b), g = -exp(A_log) softplus(a + dt_bias)
      const float ea = expf(__ldg(P.A_log + h)), db = __ldg(P.dt_bias + h);
      if (lane < L) {
        x0 = -ea * softplusf_(__bfloat162float(P.a[(t0 + lane) * P.Hv + h]) + db);
        b0 = sigmoidf_(__bfloat162float(P.b[(t0 + lane) * P.Hv + h]));
      }
      if (32 + lane < L) {
        x1 = -ea * softplusf_(__bfloat162float(P.a[(t0 + 32 + lane) * P.Hv + h]) + db);
        b1 = sigmoidf_(__bfloat162float(P.b[(t0 + 32 + lane) * P.Hv + h]));
      }
    } else {
      if (lane < L) {
        x0 = P.g[(t0 + lane) * P.Hv + h];
        b0 = P.beta[(t0 + lane) * P.Hv + h];
      }
      if (32 + lane < L) {
        x1 = P.g[(t0 + 32 + lane) * P.Hv + h];
        b1 = P.beta[(t0 + 32 + lane) * P.Hv + h];
      }
    }
    x0 = floor_decay(x0);
    x1 = floor_decay(x1);
  };

  // BWD: a whole chunk comes as boxes of tensor maps, which cost the warps no instructions; the rows behind
  // a partial chunk have to read as zeros, so it goes through issue_loads
  auto load_item = [&](const Item& I) {
    if (!BWD || I.L < tm::C) {
      issue_loads(I);
    } else if (warp == 1 && elect_one()) {
      const int32_t t = (int32_t)I.t0;
      mbar_arrive_expect_tx(lbar, 32768);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        tma_load_3d(smem + PP_KQ + half * 16384, &map_k, lbar, 64 * half, I.hk, t);
        tma_load_3d(smem + PP_KQ + half * 16384 + 8192, &map_q, lbar, 64 * half, I.hk, t);
      }
    }
  };

  Item cur;
  int st = locate(blockIdx.x, cur);
  if (st <= 0) return;  // nothing allocated yet
  PP_TS(0);
  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(lbar, 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 64);
    tmem_relinquish();
  }
  if (!BWD) issue_loads(cur);
  // Once this thread's copies have landed: every thread's copies visible to the tensor core, then
  // D1 = [K; Q] K^T of the item in shared memory (rows 0..63 K K^T, rows 64..127 Q K^T; M = 128,
  // N = 64, K-dim 128) into tensor memory, completion signalled on `bar`.
  uint32_t load_phase = 0;
  auto loads_then_mma = [&](uint32_t tmem, int L) {
    if (!BWD || L < tm::C) {
      cp_async_wait_all();
      fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (BWD && L == tm::C) {
      if (warp == 0 && !mbar_wait(lbar, load_phase)) {
        report(P.status, GDN_ERR_TIMEOUT);
        mbar_wait(lbar, load_phase);  // its copies may still be under way
      }
      __syncwarp();
      load_phase ^= 1;
    }
    // under elect.sync the MMAs are issued some ten cycles apart, under a plain lane test 134
    if (BWD ? warp == 0 && elect_one() : tid == 0) {
      const uint32_t id = idesc_bf16(128, 64, 0, 0);
      const uint64_t d0 = sdesc_sw128(sbase + PP_KQ, 16, 1024);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint64_t d = d0 + (uint64_t)(((ks >> 2) * 16384 + (ks & 3) * 32) >> 4);
        mma_bf16_ss(tmem, d, d, id, ks > 0);
      }
      mma_commit(bar);
    }
  };
  // the tensor-memory address is visible after the barrier in the first call
  cp_async_wait_all();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (BWD) load_item(cur);  // the barriers are initialised
  loads_then_mma(tmem, cur.L);
  PP_TS(1);
  uint32_t mma_phase = 0;
  bool ok = true;
  float nx0 = 0.f, nx1 = 0.f, nb0 = 0.f, nb1 = 0.f;  // BWD: gates of this warp's next head
  if (BWD && warp < min(PAIR, G)) gates(cur, cur.hk * G + warp, nx0, nx1, nb0, nb1);
  while (st > 0 && ok) {
    const int64_t slot = cur.slot;
    const int hk = cur.hk, L = cur.L;
    Item nxt;
    const int nst = locate(cur.it + gridDim.x, nxt);
    float* gl2_all = reinterpret_cast<float*>(smem + PP_GB);
  for (int h0 = 0; h0 < G; h0 += PAIR) {
    const int npair = min(PAIR, G - h0);
    // ---- cumulative log-decays (x log2 e) and betas of the pair's v-heads (warp gi: head gi)
    if (warp < npair) {
      const int h = hk * G + h0 + warp;
      float* gl2 = gl2_all + warp * 128;
      float x0, x1, b0, b1;
      if (BWD)
        x0 = nx0, x1 = nx1, b0 = nb0, b1 = nb1;  // fetched an item ahead
      else
        gates(cur, h, x0, x1, b0, b1);
      if (BWD) {
        if (lane < L) b0 = bwd::floor_beta(b0);
        if (32 + lane < L) b1 = bwd::floor_beta(b1);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y0 = __shfl_up_sync(0xffffffffu, x0, o);
        const float y1 = __shfl_up_sync(0xffffffffu, x1, o);
        if (lane >= o) {
          x0 += y0;
          x1 += y1;
        }
      }
      x1 += __shfl_sync(0xffffffffu, x0, 31);
      gl2[lane] = x0 * kLog2e;
      gl2[32 + lane] = x1 * kLog2e;
      gl2[64 + lane] = b0;
      gl2[96 + lane] = b1;
    }
    if (h0 == 0) {
      ok = mbar_wait(bar, mma_phase);
#ifdef GDN_FAULT_INJECTION
      if (tid == P.debug_thread) ok = false;
#endif
      mma_phase ^= 1;
      if (!ok) report(P.status, GDN_ERR_TIMEOUT);
    }
    tc_fence_before();
    // one answer for the CTA: a thread that went on alone would wait at barriers the others never reach
    ok = __syncthreads_and(ok) != 0;
    if (!ok) break;
    tc_fence_after();
    // scale Gamma Q of the pair as the swizzled image of two 64-column halves
    if (BWD) {
      uint4 w[4];
      const int ch = tid & 15;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (tid >> 4) + 16 * i;
        w[i] = *reinterpret_cast<const uint4*>(smem + PP_KQ + (ch >> 3) * 16384 + 8192 +
                                               sw128(r, (ch & 7) * 8));
      }
      for (int gi = 0; gi < npair; ++gi) {
        unsigned char* out = P.ws + P.qg_off + ((size_t)slot * P.Hv + hk * G + h0 + gi) * 16384 +
                             (ch >> 3) * 8192;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (tid >> 4) + 16 * i;
          const float f = P.scale * ex2f(gl2_all[gi * 128 + r]);
          const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          uint32_t y[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            y[q] = pack_bf16x2(f * __uint_as_float(x[q] << 16), f * __uint_as_float(x[q] & 0xffff0000u));
          *reinterpret_cast<uint4*>(out + sw128(r, (ch & 7) * 8)) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      // the next head's gates, while this pair is worked on
      if (h0 + PAIR < G) {
        if (warp < min(PAIR, G - h0 - PAIR))
          gates(cur, hk * G + h0 + PAIR + warp, nx0, nx1, nb0, nb1);
      } else if (nst > 0 && warp < min(PAIR, G)) {
        gates(nxt, nxt.hk * G + warp, nx0, nx1, nb0, nb1);
      }
    }
    // the MMA has read [K; Q]: the next item's K and Q may land there while this one is worked on (BWD:
    // after the last pair's masks)
    if (!BWD && h0 == 0 && nst > 0) issue_loads(nxt);
    PP_TS(2);
    // ---- decay masks straight out of tensor memory.  Thread: row R = 32 (warp & 3) + lane of
    // [K; Q], columns 32 (warp >> 2) .. + 31.  Rows 0..63 -> A (fp32, smem), 64..127 -> P (bf16,
    // workspace).  e^{gamma_r - gamma_s} = 2^{(gamma_r - gamma_s) log2 e}, never above 1.
    if constexpr (BWD) {
      // The same masks with the gates read four at a time, blocks above the diagonal skipped by whole warps,
      // and P by way of shared memory (where T will be), to leave in whole rows: 16 bytes a lane, 128 apart,
      // took most of this phase's 7500 cycles.
      const int R = 32 * (warp & 3) + lane, r = R & 63, cb = 32 * (warp >> 2);
      const bool keys = (warp & 3) < 2, above = cb > 0 && (warp & 1) == 0;
      const int last = keys ? r - 1 : r;
      float d[32];
      if (!above) {
        tmem_ld16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + cb, *reinterpret_cast<float(*)[16]>(d));
        tmem_ld16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + cb + 16,
                  *reinterpret_cast<float(*)[16]>(d + 16));
        tmem_ld_wait();
      }
      for (int gi = 0; gi < npair; ++gi) {
        const float* gl2 = gl2_all + gi * 128;
        const float gr = gl2[r];
        float* Af = reinterpret_cast<float*>(smem + PP_A) + gi * 64 * AS + r * AS + cb;
        unsigned char* Pf = smem + PP_T + gi * 64 * AS * 4 + r * PS + cb * 2;
#pragma unroll
        for (int q8 = 0; q8 < 4; ++q8) {
          float v[8] = {};
          if (!above) {
#pragma unroll
            for (int q4 = 0; q4 < 2; ++q4) {
              const int s0 = cb + 8 * q8 + 4 * q4;
              const float4 g4 = *reinterpret_cast<const float4*>(gl2 + s0);
              const float4 b4 = keys ? *reinterpret_cast<const float4*>(gl2 + 64 + s0)
                                     : make_float4(P.scale, P.scale, P.scale, P.scale);
              const float gs[4] = {g4.x, g4.y, g4.z, g4.w}, bs[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float x = bs[e] * ex2f(gr - gs[e]) * d[8 * q8 + 4 * q4 + e];
                v[4 * q4 + e] = s0 + e <= last ? x : 0.0f;
              }
            }
          }
          if (keys) {
            *reinterpret_cast<float4*>(Af + 8 * q8) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(Af + 8 * q8 + 4) = make_float4(v[4], v[5], v[6], v[7]);
          } else {
            *reinterpret_cast<uint4*>(Pf + 16 * q8) = pack8(v);
          }
        }
      }
    } else {
      const int R = 32 * (warp & 3) + lane, r = R & 63, cb = 32 * (warp >> 2);
      float d[32];
      tmem_ld16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + cb, *reinterpret_cast<float(*)[16]>(d));
      tmem_ld16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + cb + 16,
                *reinterpret_cast<float(*)[16]>(d + 16));
      tmem_ld_wait();
      for (int gi = 0; gi < npair; ++gi) {
        const int h = hk * G + h0 + gi;
        const float* gl2 = gl2_all + gi * 128;
        const float gr = gl2[r];
        const float br = R < 64 ? gl2[64 + r] : 1.0f;
        float v[32];
#pragma unroll
        for (int b16 = 0; b16 < 2; ++b16) {
          if (cb + 16 * b16 <= r) {
#pragma unroll
            for (int q = 16 * b16; q < 16 * b16 + 16; ++q) {
              const int s = cb + q;
              const bool keep = R < 64 ? (s < r) : (s <= r);
              v[q] = keep ? br * ex2f(gr - gl2[s]) * d[q] : 0.0f;
            }
          } else {  // the 16 columns lie above the diagonal
#pragma unroll
            for (int q = 16 * b16; q < 16 * b16 + 16; ++q) v[q] = 0.0f;
          }
        }
        if (R < 64) {
          float* Af = reinterpret_cast<float*>(smem + PP_A) + gi * 64 * AS;
#pragma unroll
          for (int q4 = 0; q4 < 8; ++q4)
            *reinterpret_cast<float4*>(Af + r * AS + cb + 4 * q4) =
                make_float4(v[4 * q4], v[4 * q4 + 1], v[4 * q4 + 2], v[4 * q4 + 3]);
        } else {
          unsigned char* tp = P.ws + tm::tp_offset() + ((size_t)slot * P.Hv + h) * tm::TP_BYTES;
          uint4* dst = reinterpret_cast<uint4*>(tp + (size_t)(64 + r) * 128 + cb * 2);
#pragma unroll
          for (int q8 = 0; q8 < 4; ++q8) dst[q8] = pack8(v + 8 * q8);
        }
      }
    }
    __syncthreads();  // A of every head of the pair complete
    if (BWD) {
      if (h0 + PAIR >= G && nst > 0) load_item(nxt);  // Q was read before the barrier
      const int c8 = tid & 7;
      for (int gi = 0; gi < npair; ++gi) {
        unsigned char* tp = P.ws + tm::tp_offset() + ((size_t)slot * P.Hv + hk * G + h0 + gi) * tm::TP_BYTES;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = (tid >> 3) + 32 * i;
          *reinterpret_cast<uint4*>(tp + (64 + r) * 128 + c8 * 16) =
              *reinterpret_cast<const uint4*>(smem + PP_T + gi * 64 * AS * 4 + r * PS + c8 * 16);
        }
      }
      __syncthreads();  // T may be written
    }
    // after the last pair's masks D1 is free: the next item's MMA runs during this item's solve
    if (!BWD && h0 + PAIR >= G && nst > 0) loads_then_mma(tmem, tm::C);
    PP_TS(3);
    // ---- T = (I + A)^{-1}: warpgroup gi solves head gi
    const int gi = warp >> 2, w4 = warp & 3, t4 = tid & 127;
    if (gi < npair) {
      const int h = hk * G + h0 + gi;
      const float* Af = reinterpret_cast<const float*>(smem + PP_A) + gi * 64 * AS;
      float* Tf = reinterpret_cast<float*>(smem + PP_T) + gi * 64 * AS;
      float* Mb = reinterpret_cast<float*>(smem + PP_MB) + gi * 4 * 16 * MS;
      const float* gl2 = gl2_all + gi * 128;
      solve64(1 + gi, Af, Tf, Mb, w4, lane);
      PP_TS(4);
      // T' = T diag(beta), zero above the diagonal -> rows 0..63 of the [T'; P] tile
      unsigned char* tp = P.ws + tm::tp_offset() + ((size_t)slot * P.Hv + h) * tm::TP_BYTES;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // a warp writes whole rows
        const int r = (t4 >> 3) + 16 * i, s0 = 8 * (t4 & 7);
        float tv[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int s = s0 + q;
          tv[q] = (s <= r) ? (BWD ? Tf[r * AS + s] : Tf[r * AS + s] * gl2[64 + s]) : 0.0f;
        }
        *reinterpret_cast<uint4*>(tp + (size_t)r * 128 + s0 * 2) = pack8(tv);
      }
      // Gamma_r and d_s (gamma is constant past the sequence end, so gamma_63 is the chunk's total)
      if (t4 < 64) {
        constexpr size_t gd_bytes = BWD ? bwd::GD_BYTES : tm::GD_BYTES;
        float* gd = reinterpret_cast<float*>(P.ws + P.gd_off +
                                             ((size_t)slot * P.Hv + h) * gd_bytes);
        gd[t4] = ex2f(gl2[t4]);
        gd[64 + t4] = ex2f(gl2[63] - gl2[t4]);
        if (BWD) {
          gd[128 + t4] = gl2[64 + t4];
          gd[192 + t4] = gl2[t4];
        }
      }
    }
    if (BWD && h0 + PAIR >= G && nst > 0)
      loads_then_mma(tmem, nxt.L);  // with the barrier below
    else
      __syncthreads();  // gates / A / T buffers free for the next pair
    PP_TS(5);
  }
    cur = nxt;
    st = nst;
  }
  cp_async_wait_all();  // nothing lands in shared memory after the CTA ends
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
}

}  // namespace

unsigned long long* g_prep_trace = nullptr;  // trace builds: device buffer of 8 stamps per CTA
int g_debug_prep_thread = -1;                // failure-test builds: see PrepParams::debug_thread

namespace {

template <bool BWD>
cudaError_t launch_prep_t(const PrepParams& p, int64_t slots, cudaStream_t s, const CUtensorMap& mk,
                          const CUtensorMap& mq) {
  int sms = 0;
  cudaError_t e = sm_count(sms);
  if (e == cudaSuccess) e = allow_smem(chunk_prep_kernel<BWD>, PP_SMEM);
  // all of the unified L1 / shared-memory space as shared memory: two CTAs per SM
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(chunk_prep_kernel<BWD>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e != cudaSuccess) return e;
  // persistent: two CTAs per SM, each taking every grid-th (slot, k-head) item
  const int64_t items = slots * p.Hk;
  const int64_t grid = items < 2 * (int64_t)sms ? items : 2 * (int64_t)sms;
  chunk_prep_kernel<BWD><<<(unsigned)grid, PP_THREADS, PP_SMEM, s>>>(mk, mq, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk_prep(const void* q, const void* k, TokStrides ts, const float* g,
                              const float* beta, const int32_t* cu, int N, int B, int64_t T,
                              int Hk, int Hv, void* ws, int* status, cudaStream_t s,
                              const ChunkFusion& fuse) {
  const int64_t n_tok = (int64_t)B * T;
  const int64_t slots = tm::max_slots(N, n_tok);
  if (slots <= 0 || n_tok == 0) return cudaSuccess;
  if (slots > 0x7fffffff / 64) return cudaErrorInvalidConfiguration;
  PrepParams p;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.k = reinterpret_cast<const __nv_bfloat16*>(k);
  p.g = g;
  p.beta = beta;
  p.cu = cu;
  p.ws = reinterpret_cast<unsigned char*>(ws);
  p.status = status;
  p.q_stride = ts.q;
  p.k_stride = ts.k;
  p.T = T;
  p.gd_off = (int64_t)(fuse.bwd_gd_off ? fuse.bwd_gd_off : tm::gd_offset(N, n_tok, Hv));
  p.N = N;
  p.Hk = Hk;
  p.Hv = Hv;
  p.trace = g_prep_trace;
  p.debug_thread = g_debug_prep_thread;
  p.a = fuse.a;
  p.b = fuse.b;
  p.A_log = fuse.A_log;
  p.dt_bias = fuse.dt_bias;
  p.qg_off = (int64_t)fuse.bwd_qg_off;
  p.scale = fuse.scale;
  const CUtensorMap none = {};
  return fuse.bwd_gd_off ? launch_prep_t<true>(p, slots, s, *fuse.bwd_k, *fuse.bwd_q)
                         : launch_prep_t<false>(p, slots, s, none, none);
}

}  // namespace gdn

#ifdef GDN_FAULT_INJECTION
// Failure-test builds only: in the next prefills and backward passes on the tensor-core path the wait of thread
// `t` of every preparation CTA counts as run out (-1: none), the other threads' do not.
extern "C" void gdn_debug_set_prep_thread(int t) { gdn::g_debug_prep_thread = t; }
#endif

#ifdef GDN_PREP_TRACE
// Trace builds only: device buffer (8 stamps of 8 bytes per prep CTA) for the phase stamps.
extern "C" void gdn_debug_set_prep_trace(void* buf) {
  gdn::g_prep_trace = reinterpret_cast<unsigned long long*>(buf);
}
#endif
