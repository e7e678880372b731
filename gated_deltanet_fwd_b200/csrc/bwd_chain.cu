// bwd_chain.cu -- the two serial walks of the tensor-core backward pass (bwd_tc.cuh): one CTA per
// (sequence, v-head) carries the fp32 state S (forward) or its gradient dS (backward) through the
// chunks in tensor memory.
//
// Tensor-memory lane j is value row j, as in chunk_chain.cu, so the carried matrix and the epilogue
// results are A operands from tensor memory and every B operand is a TMA-loaded tile:
//   forward, chunk by chunk from the first (X' = -(S K^T) Gamma):
//     D  = S_bf16 K^T          N 64,  K 128   critical
//     E  = V^T T~^T            N 64,  K 64    while X' is formed
//     E += X' T~^T             N 64,  K 64    critical
//     S  = Gamma_63 S + (beta d E) K      N 128, K 64   critical
//   backward, from the last chunk (X = beta (D2 + d D)):
//     D  = dS_bf16 K^T         N 64,  K 128   critical
//     D2 = dO^T (scale P)              N 64,  K 64    early
//     W  = X T~                N 64,  K 64    critical: dW^T = dV^T
//     dS = Gamma_63 dS + dO^T (scale Gamma Q) - (Gamma W) K     N 128, K 64 twice, the second critical
// Warp roles (512 threads): warps 0-7 the critical epilogues (warps w and w + 4 share 32 lanes and split the
// columns) and, while the first product of a chunk runs, the carried matrix scaled by Gamma_63; warps
// 8-11 its bf16 copy, and U or dv, to memory; warp 12 the TMA producer; warp 13 the MMA issuer.  What bounds
// it is the latency of the critical sequence of one chunk, 3400 cycles forward and 3800 backward, not
// traffic (32 v-heads, sequences of 16384, 8192, 6144 and 2048 tokens: 568 us for 2.8 GB).  Three things
// that shorten it, by clock stamps of a 64-chunk run:
//   - MMAs are issued under elect.sync, which tells the compiler that one thread is active, with
//     descriptors that are loop-invariant but for constants (the stage is a template argument): about 10
//     cycles apart, against 134 under a plain lane test and 45 with descriptors computed in the loop;
//   - the bf16 copy, U and dv leave through shared memory and bulk copies: stores of 32 bytes a lane, 256
//     bytes apart, held up every warp of the SM for 1300 of a chunk's 6300 cycles;
//   - two warps per lane quarter halve each epilogue's columns.
//
// A chunk that ends inside a tile: rows of K, Q, V, dO behind the sequence end hold whatever follows in
// memory, so the producer waits for that chunk's copies itself, clears those rows and only then
// publishes the stage.  Waits are bounded: one that runs out records GDN_ERR_TIMEOUT, and from
// then on every role skips its work but keeps the barrier sequence, so the CTA leaves together with
// nothing in flight.
#include <type_traits>

#include "bwd_tc.cuh"
#include "ptx.cuh"

namespace gdn {
namespace bwd {
namespace {

using namespace ptx;

// Four warpgroups: critical (two), side, and producer + issuer (two warps idle).  The launch gives
// every thread 128 registers.  The backward walk's critical groups need more and take them from the other
// two (2 x 144 + 120 + 104 = 4 x 128): spills cost twice here, since shared memory leaves almost no L1
// (a backward chunk took 3.2 us with 140 spilled bytes against 2.6 us without).
constexpr int THREADS = 512;
constexpr int MAX_SORTED = 256;  // sequences that are put in order of length
constexpr int W_SIDE = 8, W_PROD = 12, W_MMA = 13;

// shared memory, from a 1024-aligned base; a stage holds one chunk's tiles: K, [Q,] V or dO, T~ [and P],
// the record.  64-row tiles are two 64-column halves 8192 bytes apart.
template <bool BACK>
struct Sm {
  static constexpr uint32_t K = 0, Q = 16384, X = BACK ? 32768 : 16384, TP = X + 16384,
                            GD = TP + (BACK ? 16384 : 8192), STAGE = GD + 1024;
  static constexpr uint32_t TX = GD + GD_BYTES;  // bytes of a full stage
  static constexpr int STAGES = BACK ? 2 : 3;
  static constexpr uint32_t COPY = STAGES * STAGE;     // bf16 copies of the carried matrix on their way out
  static constexpr uint32_t OUT = COPY + 2 * 32768;    // U^T (forward) or dv (backward) on its way out
  static constexpr uint32_t BAR = OUT + 16384, BYTES = BAR + 256 + 1024;
  static_assert(STAGE % 1024 == 0 && BYTES <= 232448, "stage layout");
};

enum { B_FULL0 = 0, B_EMPTY0 = 3, B_FIX = 6, B_K = 7, B_U = 8, B_S = 9, B_DRAIN = 10, B_N = 11 };

// named barriers: hand-offs to the MMA issuer and between the two groups
enum { NB_X = 1, NB_U = 2, NB_S = 3, NB_COPY = 4, NB_SIDE = 5 };
constexpr int NB_CSI = 416;   // both groups + issuer warp
constexpr int NB_CI = 288;    // critical group + issuer warp
constexpr int NB_CS = 384;    // both groups

// tensor-memory columns
constexpr uint32_t TM_S = 0, TM_D = 128, TM_D2 = 192, TM_U = 256, TM_SB = 320, TM_X = 384,
                   TM_UD = 416;

struct ChainParams {
  const float* S0;     // initial state; null: zero
  const float* dS_T;   // gradient of the final one; null: zero
  float* dS0;          // gradient of the initial state; null: not wanted
  const int32_t* cu;
  unsigned char* ws;
  __nv_bfloat16* dv;
  int* status;
  int64_t T;
  TcLayout at;
  int N, Hk, Hv;
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint64_t dadd(uint64_t d, uint32_t bytes) {
  return d + (uint64_t)(bytes >> 4);
}
// 32 fp32 columns of this warp's lanes (no wait)
__device__ __forceinline__ void ld32(uint32_t taddr, float* v) {
  tmem_ld16(taddr, *reinterpret_cast<float(*)[16]>(v));
  tmem_ld16(taddr + 16, *reinterpret_cast<float(*)[16]>(v + 16));
}
__device__ __forceinline__ void ld64(uint32_t taddr, float* v) {
  ld32(taddr, v);
  ld32(taddr + 32, v + 32);
}

// One walk: sequence n, its tokens [s_beg, s_end), chunks from slot0 on; v-head h.  map_x: V forward, dO
// backward; map_tp: boxes of T~, backward of [T~; P].
template <bool BACK>
__device__ __forceinline__ void chain(const CUtensorMap* map_k, const CUtensorMap* map_x,
                                      const CUtensorMap* map_tp, const CUtensorMap* map_dv,
                                      const ChainParams& P, unsigned char* smem, int n, int h,
                                      int64_t s_beg, int64_t s_end, int64_t slot0) {
  using L_ = Sm<BACK>;
  const float* S_in = BACK ? P.dS_T : P.S0;
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L_::BAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L_::BAR + B_N * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L_::BAR + B_N * 8 + 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hk = h / (P.Hv / P.Hk);
  const size_t sidx = ((size_t)n * P.Hv + h) * tm::STATE_FLOATS;
  const int nch = (int)((s_end - s_beg + tm::C - 1) / tm::C);
  if (nch == 0) {  // empty sequence: the gradient passes through
    if (BACK && P.dS0)
      for (int e = tid; e < tm::D * tm::D; e += THREADS)
        P.dS0[sidx + e] = S_in ? S_in[sidx + e] : 0.0f;
    return;
  }
  // step i works on chunk chunk_of(i)
  auto chunk_of = [&](int i) { return BACK ? nch - 1 - i : i; };
  auto rows_of = [&](int c) { return (int)min((int64_t)tm::C, s_end - s_beg - (int64_t)tm::C * c); };

  if (tid == 0) {
    for (int i = 0; i < L_::STAGES; ++i) {
      mbar_init(&bars[B_FULL0 + i], 1);
      // the MMAs that read a stage and, forward, the side group's last look at its record
      mbar_init(&bars[B_EMPTY0 + i], BACK ? 1 : 2);
    }
    for (int i = B_FIX; i < B_N; ++i) mbar_init(&bars[i], 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto fail = [&](int code) {
    report(P.status, code);
    *abort_flag = 1;
  };
  // A bounded wait that gives up early once the CTA is aborting.  The flag and the timer are looked at
  // only in long waits: both take longer than the waits of a chunk.
  auto wait = [&](int b, uint32_t parity) -> bool {
    uint64_t t0 = 0;
#pragma unroll 1  // many inlined copies
    for (uint32_t k = 1; k < kSpinLimit; ++k) {
      if (mbar_try_wait(&bars[b], parity)) return true;
      if ((k & 255) == 0) {
        if (*abort_flag) return false;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitLimitNs) break;
      }
    }
    fail(GDN_ERR_TIMEOUT);
    return false;
  };
  // the same for a whole warp: one answer, so that its lanes stay together
  auto wait_w = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
  auto wait_full = [&](int i) {
    return wait_w(B_FULL0 + i % L_::STAGES, (uint32_t)(i / L_::STAGES) & 1);
  };
  auto record = [&](int i) {
    return reinterpret_cast<const float*>(smem + (i % L_::STAGES) * L_::STAGE + L_::GD);
  };

  if (warp < W_SIDE) {
    if (BACK) asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    // -------------------------------------------------------------- critical epilogues -------
    const int half = warp >> 2;
    const int j = 32 * (warp & 3) + lane;  // value row = tensor-memory lane
    const uint32_t lo = (uint32_t)(32 * (warp & 3)) << 16;
    // The carried matrix entering step i (this thread's 64 columns, in v): its bf16 copy is the next
    // product's operand; then, while that product runs, the matrix is scaled by Gamma_63.
    auto enter = [&](float* v, float gl, bool ok) {
      if (ok) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t pk[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) pk[q] = pack2(v[32 * hh + 2 * q], v[32 * hh + 2 * q + 1]);
          tmem_st16u(tmem + lo + TM_SB + 32 * half + 16 * hh, pk);
        }
        tmem_st_wait();
      }
      tc_fence_before();
      named_bar_arrive(NB_S, NB_CSI);
      named_bar_arrive(NB_COPY, NB_CS);
      if (ok) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[16 * q + e] *= gl;
          tmem_st16(tmem + lo + TM_S + 64 * half + 16 * q,
                    *reinterpret_cast<float(*)[16]>(v + 16 * q));
        }
        tmem_st_wait();
      }
    };
    {
      const float* src = S_in ? S_in + sidx + (size_t)j * tm::D + 64 * half : nullptr;
      float v[64];
#pragma unroll
      for (int q4 = 0; q4 < 16; ++q4) {
        const float4 f = src ? __ldg(reinterpret_cast<const float4*>(src) + q4)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
        v[4 * q4] = f.x;
        v[4 * q4 + 1] = f.y;
        v[4 * q4 + 2] = f.z;
        v[4 * q4 + 3] = f.w;
      }
      const bool ok = wait_full(0);
      enter(v, ok ? record(0)[63] : 0.0f, true);
    }
    for (int i = 0; i < nch; ++i) {
      const float* gd = record(i) + 32 * half;
      const uint32_t tm_u = tmem + lo + TM_U + 32 * half;
      // ---- X'.  The record's values are read before the waits, not after them, where registers allow.
      float4 ra[8];
#pragma unroll
      for (int q4 = 0; q4 < 8; ++q4)  // d, or Gamma
        ra[q4] = *reinterpret_cast<const float4*>(gd + (BACK ? 64 : 0) + 4 * q4);
      if (wait_w(B_K, i & 1)) {
        tc_fence_after();
        uint32_t pk[16];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float d[16], d2[16];
          tmem_ld16(tmem + lo + TM_D + 32 * half + 16 * hh, d);
          if (BACK) tmem_ld16(tmem + lo + TM_D2 + 32 * half + 16 * hh, d2);
          tmem_ld_wait();
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            const float* x = d + 4 * q4;
            const float4 a = ra[4 * hh + q4];
            uint32_t* o = pk + 8 * hh + 2 * q4;
            if (!BACK) {
              o[0] = pack2(-a.x * x[0], -a.y * x[1]);
              o[1] = pack2(-a.z * x[2], -a.w * x[3]);
            } else {
              const float* y = d2 + 4 * q4;
              const float4 be = *reinterpret_cast<const float4*>(gd + 128 + 16 * hh + 4 * q4);
              o[0] = pack2(be.x * fmaf(a.x, x[0], y[0]), be.y * fmaf(a.y, x[1], y[1]));
              o[1] = pack2(be.z * fmaf(a.z, x[2], y[2]), be.w * fmaf(a.w, x[3], y[3]));
            }
          }
        }
        tmem_st16u(tmem + lo + TM_X + 16 * half, pk);
        tmem_st_wait();
      }
      tc_fence_before();
      named_bar_arrive(NB_X, NB_CI);
      // ---- the update's operand: beta d E, or -Gamma dW
#pragma unroll
      for (int q4 = 0; q4 < 8; ++q4) {
        if (!BACK) {
          const float4 dd = *reinterpret_cast<const float4*>(gd + 64 + 4 * q4);
          const float4 be = *reinterpret_cast<const float4*>(gd + 128 + 4 * q4);
          ra[q4] = make_float4(be.x * dd.x, be.y * dd.y, be.z * dd.z, be.w * dd.w);
        } else {
          const float4 gm = *reinterpret_cast<const float4*>(gd + 4 * q4);
          ra[q4] = make_float4(-gm.x, -gm.y, -gm.z, -gm.w);
        }
      }
      if (wait_w(B_U, i & 1)) {
        tc_fence_after();
        float u[32];
        ld32(tm_u, u);
        tmem_ld_wait();
        uint32_t pd[16];
#pragma unroll
        for (int q4 = 0; q4 < 8; ++q4) {
          const float* x = u + 4 * q4;
          pd[2 * q4] = pack2(ra[q4].x * x[0], ra[q4].y * x[1]);
          pd[2 * q4 + 1] = pack2(ra[q4].z * x[2], ra[q4].w * x[3]);
        }
        tmem_st16u(tmem + lo + TM_UD + 16 * half, pd);
        tmem_st_wait();
      }
      tc_fence_before();
      // a full barrier, not an arrival: the group then never runs a barrier instance ahead of the
      // issuer, even when an abort makes it skip its waits
      named_bar(NB_U, NB_CSI);
      // ---- the updated matrix (not after the last chunk)
      float gl = 0.0f;
      if (i + 1 < nch && wait_full(i + 1)) gl = record(i + 1)[63];
      const bool s_ok = wait_w(B_S, i & 1);
      if (i + 1 < nch) {
        float v[64];
        if (s_ok) {
          tc_fence_after();
          ld64(tmem + lo + TM_S + 64 * half, v);
          tmem_ld_wait();
        }
        enter(v, gl, s_ok);
      } else if (BACK && P.dS0 && s_ok) {  // the gradient of the initial state
        tc_fence_after();
        float v[64];
        ld64(tmem + lo + TM_S + 64 * half, v);
        tmem_ld_wait();
        float4* dst = reinterpret_cast<float4*>(P.dS0 + sidx + (size_t)j * tm::D + 64 * half);
#pragma unroll
        for (int q4 = 0; q4 < 16; ++q4)
          dst[q4] = make_float4(v[4 * q4], v[4 * q4 + 1], v[4 * q4 + 2], v[4 * q4 + 3]);
      }
    }
  } else if (warp < W_PROD) {
    // -------------------------------------------------------------- side group (warps 8-11) --
    if (BACK) asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    const int quad = warp & 3, t4 = tid - 32 * W_SIDE;
    const int j = 32 * quad + lane;
    const uint32_t lo = (uint32_t)(32 * quad) << 16;
    // The bf16 copy of the matrix entering step i, from tensor memory to shared memory: the swizzled image
    // that the MMAs of the parallel kernel read (row j, 16-byte piece c at c ^ j % 8).
    // Two buffers in turn: a copy takes most of a chunk's time to leave.
    auto stage_copy = [&](int i) {
      named_bar(NB_COPY, NB_CS);
      tc_fence_after();
      unsigned char* row = smem + L_::COPY + (i & 1) * 32768 + j * 128;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float t[32];
        ld32(tmem + lo + TM_SB + 32 * hh, t);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<float4*>(row + hh * 16384 + ((q ^ (j & 7)) << 4)) =
              make_float4(t[4 * q], t[4 * q + 1], t[4 * q + 2], t[4 * q + 3]);
      }
      tc_fence_before();
    };
    auto send_copy = [&](int i) {
      const size_t sh = (size_t)(slot0 + chunk_of(i)) * P.Hv + h;
      bulk_store(P.ws + (BACK ? P.at.ds : P.at.s) + sh * 32768, smem + L_::COPY + (i & 1) * 32768, 32768);
      bulk_commit();
    };
    named_bar_arrive(NB_S, NB_CSI);
    stage_copy(0);
    fence_proxy_async_smem();
    named_bar(NB_SIDE, 128);
    if (t4 == 0) send_copy(0);
    __syncwarp();
    for (int i = 0; i < nch; ++i) {
      // all that was sent has left shared memory, except perhaps the copy entering this step
      if (t4 == 0) bulk_wait_read<1>();
      __syncwarp();
      named_bar(NB_U, NB_CSI);  // a full barrier (see the other group)
      const int c = chunk_of(i);
      // E^T or dW^T: complete since the critical group has waited for it
      bool ok = wait_w(B_U, i & 1);
      if (!BACK) ok = wait_full(i) && ok;  // the record is visible to this thread
      uint32_t ob[32];  // tokens 2q, 2q + 1 of value row j
      if (ok) {
        tc_fence_after();
        const float* be = record(i) + 128;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float t[32];
          ld32(tmem + lo + TM_U + 32 * hh, t);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            if (!BACK) {
              const float2 b2 = *reinterpret_cast<const float2*>(be + 32 * hh + 2 * q);
              t[2 * q] *= b2.x;
              t[2 * q + 1] *= b2.y;
            }
            ob[16 * hh + q] = pack2(t[2 * q], t[2 * q + 1]);
          }
        }
      }
      tc_fence_before();
      if (i + 1 < nch) named_bar_arrive(NB_S, NB_CSI);  // U / dW read
      const int L = rows_of(c);
      if (ok && !BACK) {  // U^T, the same kind of image
        unsigned char* row = smem + L_::OUT + j * 128;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<uint4*>(row + ((q ^ (j & 7)) << 4)) =
              make_uint4(ob[4 * q], ob[4 * q + 1], ob[4 * q + 2], ob[4 * q + 3]);
      }
      if (ok && BACK) {
        // dv, [token][channel], two bytes at a time: a warp's 32 channels are 64 consecutive bytes.  (Swapping
        // halves between lanes for 4-byte stores took 3700 cycles a chunk against 400.)  A whole chunk
        // goes out as the box of a tensor map, a partial one row by row.
        if (L == tm::C) {
          unsigned char* tile = smem + L_::OUT + (j >> 6) * 8192 + (j & 7) * 2;
          const uint32_t c8 = (uint32_t)(j & 63) >> 3;
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            const uint32_t r = 2 * q;
            *reinterpret_cast<uint16_t*>(tile + r * 128 + ((c8 ^ (r & 7)) << 4)) = (uint16_t)ob[q];
            *reinterpret_cast<uint16_t*>(tile + (r + 1) * 128 + ((c8 ^ ((r + 1) & 7)) << 4)) =
                (uint16_t)(ob[q] >> 16);
          }
        } else {
          const int64_t rs = (int64_t)P.Hv * tm::D;
          uint16_t* dst = reinterpret_cast<uint16_t*>(P.dv + (s_beg + (int64_t)tm::C * c) * rs +
                                                      h * tm::D + j);
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            if (2 * q < L) dst[(int64_t)(2 * q) * rs] = (uint16_t)ob[q];
            if (2 * q + 1 < L) dst[(int64_t)(2 * q + 1) * rs] = (uint16_t)(ob[q] >> 16);
          }
        }
      }
      const bool more = i + 1 < nch;
      if (more) stage_copy(i + 1);
      fence_proxy_async_smem();
      named_bar(NB_SIDE, 128);
      if (t4 == 0) {
        if (!BACK) mbar_arrive(&bars[B_EMPTY0 + i % L_::STAGES]);
        if (ok && !BACK) {
          const size_t sh = (size_t)(slot0 + c) * P.Hv + h;
          bulk_store(P.ws + P.at.u + sh * 16384, smem + L_::OUT, 16384);
          bulk_commit();
        }
        if (ok && BACK && L == tm::C) {
          const int32_t t0 = (int32_t)(s_beg + (int64_t)tm::C * c);
          tma_store_3d(map_dv, smem + L_::OUT, 0, h, t0);
          tma_store_3d(map_dv, smem + L_::OUT + 8192, 64, h, t0);
          bulk_commit();
        }
        if (more && !*abort_flag) send_copy(i + 1);
      }
      __syncwarp();
    }
    if (t4 == 0) bulk_wait<0>();  // nothing on its way out of shared memory
  } else {
    if (BACK) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == W_PROD) {
      // -------------------------------------------------------------- TMA producer -------------
      if (elect_one()) {
        prefetch_tensormap(map_k);
        prefetch_tensormap(map_x);
        prefetch_tensormap(map_tp);
      }
      int issued = 0;
      for (int i = 0; i < nch; ++i) {
        const int st = i % L_::STAGES, c = chunk_of(i), L = rows_of(c);
        bool go = true;
        if (lane == 0) {
          if (i >= L_::STAGES) go = wait(B_EMPTY0 + st, ((uint32_t)(i / L_::STAGES) & 1) ^ 1);
          go = go && !*abort_flag;
        }
        if (!__shfl_sync(0xffffffffu, (int)go, 0)) break;
        unsigned char* sp = smem + st * L_::STAGE;
        // a partial chunk's copies are awaited here, on a barrier of their own
        const bool part = L < tm::C;
        uint64_t* fb = part ? &bars[B_FIX] : &bars[B_FULL0 + st];
        if (elect_one()) {
          const int32_t t0 = (int32_t)(s_beg + (int64_t)tm::C * c);
          const size_t sh = (size_t)(slot0 + c) * P.Hv + h;
          mbar_arrive_expect_tx(fb, L_::TX);
          tma_load_3d(sp + L_::K, map_k, fb, 0, hk, t0);
          tma_load_3d(sp + L_::K + 8192, map_k, fb, 64, hk, t0);
          if (BACK) {
            bulk_load(sp + L_::Q, P.ws + P.at.qg + sh * 16384, 16384, fb);
          }
          tma_load_3d(sp + L_::X, map_x, fb, 0, h, t0);
          tma_load_3d(sp + L_::X + 8192, map_x, fb, 64, h, t0);
          tma_load_2d(sp + L_::TP, map_tp, fb, 0, (int32_t)(sh * 128));
          bulk_load(sp + L_::GD, P.ws + P.at.gd + sh * GD_BYTES, GD_BYTES, fb);
        }
        if (part) {  // once per sequence: its last chunk
          bool ok = mbar_wait(fb, 0);
          if (!ok && lane == 0) fail(GDN_ERR_TIMEOUT);
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            constexpr int TILES = BACK ? 6 : 4;  // 64-row half tiles of K, [Q,] X, one after the other
            clear_rows(sp, TILES, L, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_FULL0 + st]);
          } else {
            mbar_wait(fb, 0);  // its copies may still be under way
            break;
          }
        }
        issued = i + 1;
      }
      // never leave the CTA with copies still landing in shared memory (each wait bounded)
      if (lane == 0)
        for (int i = issued > L_::STAGES ? issued - L_::STAGES : 0; i < issued; ++i)
          if (!mbar_wait(&bars[B_FULL0 + i % L_::STAGES], (uint32_t)(i / L_::STAGES) & 1))
            report(P.status, GDN_ERR_TIMEOUT);
    } else if (warp == W_MMA) {
      // -------------------------------------------------------------- MMA issuer ---------------
      const uint32_t id_k = idesc_bf16(128, 64, 0, 0);             // A tensor memory, B K-major
      const uint32_t id_e = idesc_bf16(128, 64, 1, BACK ? 1 : 0);  // A smem MN-major
      const uint32_t id_u = idesc_bf16(128, 64, 0, BACK ? 1 : 0);  // T~^T forward, T~ backward
      const uint32_t id_s = idesc_bf16(128, 128, 0, 1);            // B = K, MN-major
      const uint32_t id_q = idesc_bf16(128, 128, 1, 1);            // A = dO^T, B = scale Gamma Q
      const uint64_t dK0 = sdesc_sw128(sbase + L_::K, 16, 1024);       // K as K-major B
      const uint64_t dKn0 = sdesc_sw128(sbase + L_::K, 8192, 1024);    // K as MN-major B
      const uint64_t dQn0 = sdesc_sw128(sbase + L_::Q, 8192, 1024);    // scale Gamma Q as MN-major B
      const uint64_t dXt0 = sdesc_sw128(sbase + L_::X, 8192, 1024);    // V^T / dO^T as MN-major A
      const uint64_t dT0 = BACK ? sdesc_sw128(sbase + L_::TP, 8192, 1024)   // T~ as MN-major B
                                : sdesc_sw128(sbase + L_::TP, 16, 1024);    // T~ as K-major B
      const uint64_t dP0 = sdesc_sw128(sbase + L_::TP + 8192, 8192, 1024);  // P as MN-major B
      constexpr uint32_t t_step = BACK ? 2048 : 32;
      auto step = [&](auto stage, int i) {
        constexpr uint32_t o = decltype(stage)::value * L_::STAGE;
        // the chunk's tiles have landed and nothing failed so far; a failure later in the chunk leaves its
        // MMAs to run on whatever is there, in bounds all the same
        const bool go = wait_full(i) && __all_sync(0xffffffffu, !*abort_flag);
        if (BACK && go) {  // state-independent; D2 was read before the previous chunk's NB_U
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_bf16_ss(tmem + TM_D2, dadd(dXt0, o + ks * 2048), dadd(dP0, o + ks * 2048), id_e,
                          ks > 0);
          }
        }
        __syncwarp();
        named_bar(NB_S, NB_CSI);  // bf16 copy in place, U / dW of the previous chunk read
        if (go) {
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_bf16_ts(tmem + TM_D, tmem + TM_SB + 8 * ks,
                          dadd(dK0, o + (ks >> 2) * 8192 + (ks & 3) * 32), id_k, ks > 0);
            mma_commit(&bars[B_K]);
            if (!BACK) {  // state-independent, while X' is formed
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_bf16_ss(tmem + TM_U, dadd(dXt0, o + ks * 2048), dadd(dT0, o + ks * 32), id_e,
                            ks > 0);
            }
          }
        }
        __syncwarp();
        named_bar(NB_X, NB_CI);  // X' written, matrix scaled
        if (go) {
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_bf16_ts(tmem + TM_U, tmem + TM_X + 8 * ks, dadd(dT0, o + ks * t_step), id_u,
                          !BACK || ks > 0);
            mma_commit(&bars[B_U]);
            if (BACK) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_bf16_ss(tmem + TM_S, dadd(dXt0, o + ks * 2048), dadd(dQn0, o + ks * 2048), id_q,
                            1);
            }
          }
        }
        __syncwarp();
        named_bar(NB_U, NB_CSI);  // the update's operand written
        if (go) {
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_bf16_ts(tmem + TM_S, tmem + TM_UD + 8 * ks, dadd(dKn0, o + ks * 2048), id_s, 1);
            mma_commit(&bars[B_S]);
            mma_commit(&bars[B_EMPTY0 + decltype(stage)::value]);
          }
        }
        __syncwarp();
      };
      for (int i = 0; i < nch; i += L_::STAGES) {
        step(std::integral_constant<int, 0>(), i);
        if (i + 1 < nch) step(std::integral_constant<int, 1>(), i + 1);
        if (L_::STAGES > 2 && i + 2 < nch) step(std::integral_constant<int, L_::STAGES - 1>(), i + 2);
      }
      // every MMA has completed before tensor memory is read back or released
      if (elect_one()) {
        mma_commit(&bars[B_DRAIN]);
        if (!mbar_wait(&bars[B_DRAIN], 0)) fail(GDN_ERR_TIMEOUT);
      }
      __syncwarp();
    }
  }

  // the issuer's drain is over for every thread after this barrier
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The two walks of a (sequence, v-head) do not depend on one another, so all of both are units of one
// launch, the longest sequences first: with 32 heads and sequences of 16384, 8192, 6144 and 2048 tokens the
// walks one after the other took 475 + 535 us, half of it with most SMs idle, together 568 us.
__global__ void __launch_bounds__(THREADS, 1) bwd_chain_kernel(
    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
    const __grid_constant__ CUtensorMap map_do, const __grid_constant__ CUtensorMap map_t,
    const __grid_constant__ CUtensorMap map_tp, const __grid_constant__ CUtensorMap map_dv,
    const ChainParams P) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int h = blockIdx.x % P.Hv;
  const bool back = (blockIdx.x / P.Hv) % 2 == 0;  // first: its chunks take longer
  int n = blockIdx.x / (2 * P.Hv);
  // the n-th longest sequence; many sequences balance without
  if (P.cu && P.N > 1 && P.N <= MAX_SORTED) {
    __shared__ int pick, len[MAX_SORTED];
    const int i = threadIdx.x;
    if (i < P.N) len[i] = P.cu[i + 1] - P.cu[i];
    __syncthreads();
    if (i < P.N) {
      int rank = 0;
      for (int m = 0; m < P.N; ++m) rank += len[m] > len[i] || (len[m] == len[i] && m < i);
      if (rank == n) pick = i;  // ranks are a permutation whatever cu_seqlens holds
    }
    __syncthreads();
    n = pick;
  }
  int64_t s_beg, s_end, slot0;
  if (!seq_range(P.cu, P.T, n, tm::C, s_beg, s_end, slot0)) {
    if (threadIdx.x == 0) report(P.status, GDN_ERR_DEVICE_ARG);
    return;  // nothing allocated yet
  }
  if (back)
    chain<true>(&map_k, &map_do, &map_tp, &map_dv, P, smem, n, h, s_beg, s_end, slot0);
  else
    chain<false>(&map_k, &map_v, &map_t, &map_dv, P, smem, n, h, s_beg, s_end, slot0);
}

}  // namespace

cudaError_t launch_bwd_chain(const Args& a, const TcMaps& m, cudaStream_t s) {
  const int64_t n_tok = (int64_t)a.B * a.T, units = 2 * (int64_t)a.N * a.Hv;
  if (units > 0x7fffffff) return cudaErrorInvalidConfiguration;
  ChainParams p;
  unsigned char* ws = reinterpret_cast<unsigned char*>(a.ws);
  p.S0 = a.S0;
  p.dS_T = a.dST;
  p.dS0 = a.dS0;
  p.cu = a.cu;
  p.ws = ws;
  p.dv = reinterpret_cast<__nv_bfloat16*>(a.dv_);
  p.status = a.status;
  p.T = a.T;
  p.at = tc_layout(max_slots(a.N, n_tok, tm::C), a.Hv);
  p.N = a.N;
  p.Hk = a.Hk;
  p.Hv = a.Hv;
  constexpr uint32_t bytes = Sm<true>::BYTES > Sm<false>::BYTES ? Sm<true>::BYTES : Sm<false>::BYTES;
  const cudaError_t e = allow_smem(bwd_chain_kernel, bytes);
  if (e != cudaSuccess) return e;
  bwd_chain_kernel<<<(unsigned)units, THREADS, bytes, s>>>(m.k, m.v, m.dout, m.t, m.tp, m.dv, p);
  return cudaGetLastError();
}

}  // namespace bwd
}  // namespace gdn
