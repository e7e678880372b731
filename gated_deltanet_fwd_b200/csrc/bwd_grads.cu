// bwd_grads.cu -- the parallel half of the tensor-core backward pass (bwd_tc.cuh): dq, dk, dg and dbeta of
// every chunk from the chains' states S, dS, U and dv.  Formulas in bwd_simt.cu.
//
// Work item = (chunk, k-head); an item runs through the v-heads that share the k-head.  Persistent CTAs, which
// take their items from a counter (the first one is the CTA's own number): the SMs finish equal work up
// to a fifth apart, by their way to memory.  Which CTA does an item changes none of its results.
// Everything is computed transposed -- lane i of tensor memory is channel i of q and k, columns are
// tokens -- so that every product has M = 128 and the sums over the shared heads stay in registers of
// the thread that owns the channel:
//   MMA_p  D2 = [dO; dW] U^T            M 128 (tokens), N 64, K 128
//   MMA_s  D1 = S^T [dO; dW]^T          M 128, N 128, K 128        (raw dQ | raw dKe)
//          D3 = dS^T U^T                M 128, N 64,  K 128        (raw dKw)
//   MMA_n  D4 = K^T [dN; dM]^T          M 128, N 128, K 64
//          D5 = Q^T dN + K^T dM         M 128, N 64,  K 64 twice
// Epilogue A (token rows): decay masks on D2 -> [dN; dM], strictly lower, in shared memory as bf16; from the
// diagonals p (a token's own pair, which has no decay: added to dq and dk in fp32 and kept out of dgamma,
// where only rounding errors would be left of it) and dbeta; and <S, dS> from shared memory.  Epilogue B
// (channel rows): Gamma and d applied in fp32, dq and dk summed over the heads, dgamma = q.dq +
// k.(dKe - D5) and kappa = k.(d D3) reduced over channels (bwd_simt.cu); two tokens per instruction
// (fp32x2).
// MMA_p of the next head runs beside epilogue B of this one.  [dO; dW] and U have two buffers; S and dS have one,
// free again before epilogue B; dq and dk leave through the [dO; dW] buffer of the item's last step.  So the
// loads of a step run beside the epilogues of the step before.
//
// Warp roles (384 threads): warps 0-7 the epilogues (lane quarter warp % 4; columns, in epilogue B tokens,
// split in two by warp / 4), warp 8 the TMA producer, warp 9 the MMA issuer, warp 10 sends dq and dk out.
// Bounds: 144 KB of tiles per (chunk, v-head) at two v-heads a k-head against about 6 units of
// 64 x 128 x 128 products: the epilogues' instructions, with HBM close behind.  16384 (chunk, v-head) pairs:
// 533 us for 2.6 GB, 4.9 TB/s (75 % of a copy).  The kernel is 100 KB of code and warps wait for instructions
// (a stall in six), so polling loops are kept rolled and an item's chunk is searched once, by the producer:
// 143 KB took 576 us.
// Bounded waits and the abort protocol as in bwd_chain.cu.
#include "bwd_tc.cuh"
#include "f32x2.cuh"
#include "ptx.cuh"

namespace gdn {
namespace bwd {
namespace {

using namespace ptx;

// Three warpgroups: epilogues (two), and producer, issuer and sender (one warp idle).  168 registers a thread at
// launch; 2 x 184 + 136 = 3 x 168 (the issuer keeps its loop-invariant descriptors in registers).
constexpr int THREADS = 384;
constexpr int W_PROD = 8, W_MMA = 9, W_OUT = 10;

// shared memory, from a 1024-aligned base
constexpr uint32_t SM_KQ = 0;               // [K; Q]: two 64-column halves x 128 rows x 128 B
constexpr uint32_t SM_OW = SM_KQ + 32768;   // [dO; dW]: two buffers of the same form; at the end of an
                                            // item dq, dk: each two halves x 64 x 128 B
constexpr uint32_t SM_U = SM_OW + 2 * 32768;  // U^T: two buffers of 128 rows x 128 B
constexpr uint32_t SM_S = SM_U + 2 * 16384;   // S: two halves x 128 rows x 128 B
constexpr uint32_t SM_DS = SM_S + 32768;      // dS: the same
constexpr uint32_t SM_NM = SM_DS + 32768;     // [dN; dM]: 128 rows x 128 B
constexpr uint32_t SM_GD = SM_NM + 16384;     // four records: one is read until its step ends
constexpr uint32_t SM_RED = SM_GD + 4 * GD_BYTES;  // 2 x (dgamma and kappa parts, each [4][64], sums [8])
constexpr uint32_t RED_FLOATS = 2 * 4 * 64 + 8;
constexpr uint32_t SM_OWN = SM_RED + 2 * RED_FLOATS * 4;  // p [64], summed over the heads
constexpr uint32_t SM_BAR = SM_OWN + 256;
constexpr uint32_t SM_ITEM = SM_BAR + 160;  // four steps' and two items' records
constexpr uint32_t SM_BYTES = SM_ITEM + 96 + 1024;
static_assert(SM_BYTES <= 232448, "shared memory budget");
constexpr uint32_t TX_KQ = 32768, TX_HEAD = 32768 + 16384 + GD_BYTES, TX_STATE = 65536;

// B_H, B_HE: two of each, by the step's parity; B_O: by the item's
enum { B_KQ, B_KQE, B_H, B_HE = B_H + 2, B_O = B_HE + 2, B_S = B_O + 2, B_SE, B_P, B_NM, B_N, B_D, B_FIX, B_DRAIN, B_COUNT };
static_assert(B_COUNT * 8 + 8 <= 160, "barriers");
constexpr int NB_E = 1, NB_EPI = 256;  // named barrier of the epilogues

// tensor-memory columns
constexpr uint32_t TM_D2 = 0, TM_D1 = 64, TM_D4 = 192, TM_D3 = 320, TM_D5 = 384;

struct GradParams {
  const float* beta;
  const float* S0;  // only whether there is one
  const int32_t* cu;
  const unsigned char* ws;
  int* next;  // items handed out beyond the CTAs' first ones
  __nv_bfloat16 *dq, *dk, *dv, *dg, *dbeta;
  int* status;
  int64_t T, items;
  TcLayout at;
  float scale;
  int N, Hk, Hv;
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint64_t dadd(uint64_t d, uint32_t bytes) {
  return d + (uint64_t)(bytes >> 4);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// acc + the products of eight bf16 pairs, in fp32
__device__ __forceinline__ float dot8(uint4 a, uint4 b, float acc) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 al, ah, bl, bh;\n\t"
        "mov.b32 {al, ah}, %1;\n\t"
        "mov.b32 {bl, bh}, %2;\n\t"
        "fma.rn.f32.bf16 %0, al, bl, %0;\n\t"
        "fma.rn.f32.bf16 %0, ah, bh, %0;\n\t}"
        : "+f"(acc)
        : "r"(x[i]), "r"(y[i]));
  return acc;
}

// Named barrier of `count` threads that tells whether `ok` holds for all of them.
__device__ __forceinline__ bool bar_all(int id, int count, bool ok) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(count), "r"((int)ok)
      : "memory");
  return r != 0;
}

__global__ void __launch_bounds__(THREADS, 1) bwd_grads_kernel(
    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_q,
    const __grid_constant__ CUtensorMap map_do, const __grid_constant__ CUtensorMap map_dv,
    const __grid_constant__ CUtensorMap map_dq, const __grid_constant__ CUtensorMap map_dk,
    const GradParams P) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM_BAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM_BAR + B_COUNT * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM_BAR + B_COUNT * 8 + 4);
  // a chunk and k-head as (tokens, 0 behind the last item; whether first of its sequence; k-head; first token):
  // of a step, published with its tiles, and of dq, dk on their way out
  int4* step_item = reinterpret_cast<int4*>(smem + SM_ITEM);
  int4* out_item = step_item + 4;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = P.Hv / P.Hk;

  // item -> chunk and k-head; false past the last one or for a malformed cu_seqlens
  ChunkCursor cursor;
  auto locate = [&](int64_t it, Chunk& ch, int64_t& slot, int& hk) {
    slot = (uint32_t)it / (uint32_t)P.Hk;  // items fit 32 bits (launch_tc)
    hk = (int)((uint32_t)it - (uint32_t)slot * (uint32_t)P.Hk);
    return it < P.items && cursor.find(P.cu, P.T, P.N, tm::C, slot, ch, P.status);
  };
  {
    Chunk ch;
    int64_t slot;
    int hk;
    if (!locate(blockIdx.x, ch, slot, hk)) return;  // nothing allocated yet
  }
  if (tid == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      const bool all = i == B_HE || i == B_HE + 1 || i == B_SE || i == B_KQE;
      const bool epi = i == B_NM || i == B_D || i == B_O || i == B_O + 1;
      mbar_init(&bars[i], all ? 9 : epi ? 8 : 1);  // 8 epilogue warps, one commit
    }
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
  auto wait = [&](int b, uint32_t parity) -> bool {
    uint64_t t0 = 0;
#pragma unroll 1  // a dozen inlined copies
    for (uint32_t k = 1; k < kSpinLimit; ++k) {
      if (mbar_try_wait(&bars[b], parity)) return true;
      if ((k & 255) == 0) {  // long waits only: the flag and the timer are slow to read
        if (*abort_flag) return false;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitLimitNs) break;
      }
    }
    fail(GDN_ERR_TIMEOUT);
    return false;
  };
  auto wait_w = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };

  // `x` counts this CTA's (item, v-head) steps, `y` its items
  int x = 0, y = 0;
  if (warp < 8) {
    // ------------------------------------------------------------------ epilogues ------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int quad = warp & 3, half = warp >> 2;
    const int row = 32 * quad + lane;  // epilogue A: row of [dO; dW]; epilogue B: channel
    const uint32_t lo = (uint32_t)(32 * quad) << 16;
    for (;; ++y) {
      // all warps leave together: the named barriers need every one of them
      const bool got = wait_w(B_H + (x & 1), (x >> 1) & 1);
      if (!bar_all(NB_E, NB_EPI, got)) break;
      const int4 item = step_item[x & 3];
      const int L = item.x, hk = item.z;
      const int64_t t0 = item.w;
      if (L == 0) break;
      // tokens 32 half + 2 q, + 1 of channel `row`: dq, dk summed over the heads, and q, k
      f32x2 aq[16], ak[16];
      uint32_t qv[16], kv[16];
      float* own = reinterpret_cast<float*>(smem + SM_OWN);
      float own_sum = 0.0f;  // p of this thread's row, over the heads
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        aq[q] = ak[q] = 0ull;
        qv[q] = kv[q] = 0u;
      }
      for (int gi = 0; gi < G; ++gi, ++x) {
        const int h = hk * G + gi;
        float* red = reinterpret_cast<float*>(smem + SM_RED) + (x & 1) * RED_FLOATS;
        float* sums = red + 512;  // <S, dS>
        const float* gd = reinterpret_cast<const float*>(smem + SM_GD + (x & 3) * GD_BYTES);
        const bool in = wait_w(B_H + (x & 1), (x >> 1) & 1);
        // seen: the next use may be published; at the end of an item dq and dk go through the buffer first
        if (lane == 0 && gi < G - 1) mbar_arrive(&bars[B_HE + (x & 1)]);
        // ---- epilogue A
        const int r = row & 63;
        float diag = 0.0f;
        if (wait_w(B_P, x & 1) && in) {
          tc_fence_after();
          float d[32];
          tmem_ld32(tmem + lo + TM_D2 + 32 * half, d);
          const float gr = gd[192 + r], mul = row < 64 ? P.scale : -1.0f;
          uint32_t pk[16];
          if (half > (quad & 1)) {  // above the diagonal
#pragma unroll
            for (int q = 0; q < 16; ++q) pk[q] = 0u;
          } else {
            const bool tri = half == (quad & 1);  // the block on the diagonal
#pragma unroll
            for (int q4 = 0; q4 < 8; ++q4) {
              const float4 gs = *reinterpret_cast<const float4*>(gd + 192 + 32 * half + 4 * q4);
              float v[4] = {ex2(gr - gs.x), ex2(gr - gs.y), ex2(gr - gs.z), ex2(gr - gs.w)};
              if (tri) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (4 * q4 + e >= lane) v[e] = 0.0f;
              }
              pk[2 * q4] = pack2(mul * v[0] * d[4 * q4], mul * v[1] * d[4 * q4 + 1]);
              pk[2 * q4 + 1] = pack2(mul * v[2] * d[4 * q4 + 2], mul * v[3] * d[4 * q4 + 3]);
            }
            if (tri) {  // dO_r . U_r or dW_r . U_r: column `lane` of this block, by halving
#pragma unroll
              for (int w = 16; w > 0; w >>= 1)
#pragma unroll
                for (int q = 0; q < 16; ++q)
                  if (q < w) d[q] = lane & w ? d[q + w] : d[q];
              diag = d[0];
            }
          }
          own_sum += P.scale * diag;
          if (quad < 2 && half == quad && gi == G - 1) own[row] = own_sum;
          unsigned char* nm = smem + SM_NM;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(nm + sw128(row, 32 * half + 8 * q)) =
                make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_NM]);  // [dN; dM] written, D2 read
        // ---- <S, dS>, dbeta; q and k of the item
        float fr = 0.0f;
        if (wait_w(B_S, x & 1)) {
          const uint4* s = reinterpret_cast<const uint4*>(smem + SM_S) + tid;
          const uint4* ds = reinterpret_cast<const uint4*>(smem + SM_DS) + tid;
          float f[4] = {};
#pragma unroll
          for (int q = 0; q < 8; ++q) f[q & 3] = dot8(s[q * 256], ds[q * 256], f[q & 3]);
          fr = (f[0] + f[1]) + (f[2] + f[3]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_SE]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) fr += __shfl_xor_sync(0xffffffffu, fr, o);
        if (lane == 0) sums[warp] = fr;
        if (quad >= 2 && half == (quad & 1) && in && r < L) {
          const float b = gd[128 + r], t = diag / b / b;
          P.dbeta[(t0 + r) * P.Hv + h] = __float2bfloat16_rn(t);
        }
        if (gi == 0) {
          if (wait_w(B_KQ, y & 1)) {
            // token t has t % 8 fixed per unrolled step: so is the swizzle of this thread's column
            const unsigned char* kt = smem + SM_KQ + (row >> 6) * 16384 + half * 4096 + (row & 7) * 2;
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const uint32_t c8 = ((uint32_t)row & 63) >> 3;
              const unsigned char* p0 = kt + 2 * q * 128 + ((c8 ^ ((2 * q) & 7)) << 4);
              const unsigned char* p1 = kt + (2 * q + 1) * 128 + ((c8 ^ ((2 * q + 1) & 7)) << 4);
              kv[q] = *reinterpret_cast<const uint16_t*>(p0) |
                      (uint32_t) * reinterpret_cast<const uint16_t*>(p1) << 16;
              qv[q] = *reinterpret_cast<const uint16_t*>(p0 + 8192) |
                      (uint32_t) * reinterpret_cast<const uint16_t*>(p1 + 8192) << 16;
            }
          }
        }
        if (gi == 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[B_KQE]);  // this warp needs K and Q no more
        }
        // ---- epilogue B
        if (wait_w(B_N, x & 1)) {
          tc_fence_after();
          float keep = 0.0f, keepk = 0.0f;
#pragma unroll
          for (int b = 0; b < 4; ++b) {  // 8 tokens at a time
            const int tb = 32 * half + 8 * b;
            float d1a[8], d1b[8], d4a[8], d4b[8], d3[8], d5[8], v[8], kap[8];
            tmem_ld8(tmem + lo + TM_D1 + tb, d1a);
            tmem_ld8(tmem + lo + TM_D4 + tb, d4a);
            tmem_ld8(tmem + lo + TM_D1 + 64 + tb, d1b);
            tmem_ld8(tmem + lo + TM_D4 + 64 + tb, d4b);
            tmem_ld8(tmem + lo + TM_D3 + tb, d3);
            tmem_ld8(tmem + lo + TM_D5 + tb, d5);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const int p = 4 * b + e / 2;
              const f32x2 k2 = widen(kv[p]), q2 = widen(qv[p]);
              const float2 g1 = *reinterpret_cast<const float2*>(gd + tb + e);
              const float2 dd = *reinterpret_cast<const float2*>(gd + 64 + tb + e);
              const f32x2 g2 = two(g1.x, g1.y), neg = two(-1.0f, -1.0f);
              const f32x2 fq = fma2(mul2(two(P.scale, P.scale), g2), two(d1a[e], d1a[e + 1]),
                                    two(d4a[e], d4a[e + 1]));
              const f32x2 fe = fma2(mul2(neg, g2), two(d1b[e], d1b[e + 1]),
                                    two(d4b[e], d4b[e + 1]));
              const f32x2 w1 = mul2(two(dd.x, dd.y), two(d3[e], d3[e + 1]));
              const f32x2 fw = add2(w1, two(d5[e], d5[e + 1]));
              const float2 vv = parts(fma2(q2, fq, mul2(k2, fma2(neg, two(d5[e], d5[e + 1]), fe))));
              v[e] = vv.x;
              v[e + 1] = vv.y;
              const float2 kk = parts(mul2(k2, w1));
              kap[e] = kk.x;
              kap[e + 1] = kk.y;
              aq[p] = add2(aq[p], fq);
              ak[p] = add2(ak[p], add2(fe, fw));
            }
            // sum over the warp's 32 channels: halve the tokens a lane holds three times, then add the
            // four lanes that are left with the same token: token tb + (lane >> 2)
#pragma unroll
            for (int w = 4; w > 0; w >>= 1) {
              const bool up = lane & (4 * w);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (e < w) {
                  const float give = up ? v[e] : v[e + w], stay = up ? v[e + w] : v[e];
                  v[e] = stay + __shfl_xor_sync(0xffffffffu, give, 4 * w);
                  const float givek = up ? kap[e] : kap[e + w], stayk = up ? kap[e + w] : kap[e];
                  kap[e] = stayk + __shfl_xor_sync(0xffffffffu, givek, 4 * w);
                }
              }
            }
            // the last two steps for both sums at once: odd lanes go on with kappa
            float o = lane & 1 ? kap[0] : v[0];
            o += __shfl_xor_sync(0xffffffffu, lane & 1 ? v[0] : kap[0], 1);
            o += __shfl_xor_sync(0xffffffffu, o, 2);
            const float p = __shfl_xor_sync(0xffffffffu, o, 1);
            if ((lane & 3) == b) {  // lane 4 k + b ends up with token 8 b + k
              keep = lane & 1 ? p : o;
              keepk = lane & 1 ? o : p;
            }
          }
          const int at = quad * 64 + 32 * half + 8 * (lane & 3) + (lane >> 2);
          red[at] = keep;
          red[256 + at] = keepk;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_D]);  // D1, D3, D4, D5 read
        named_bar(NB_E, NB_EPI);         // dgamma parts and sums of all warps
        // ---- dg: suffix sums over the chunk, and what leaves through the state
        const bool live = __all_sync(0xffffffffu, !*abort_flag) != 0;
        if (warp == (x & 7) && live) {
          float f = 0.0f;
#pragma unroll
          for (int q = 0; q < 8; ++q) f += sums[q];
          f *= gd[63];
          float a0 = 0.0f, a1 = 0.0f, k0 = 0.0f, k1 = 0.0f;  // tokens lane and 32 + lane
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            a0 += red[q * 64 + lane];
            a1 += red[q * 64 + 32 + lane];
            k0 += red[256 + q * 64 + lane];
            k1 += red[256 + q * 64 + 32 + lane];
          }
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float u0 = __shfl_down_sync(0xffffffffu, a0, o);
            const float u1 = __shfl_down_sync(0xffffffffu, a1, o);
            const float l0 = __shfl_up_sync(0xffffffffu, k0, o);
            const float l1 = __shfl_up_sync(0xffffffffu, k1, o);
            if (lane + o < 32) {
              a0 += u0;
              a1 += u1;
            }
            if (lane >= o) {
              k0 += l0;
              k1 += l1;
            }
          }
          a0 += __shfl_sync(0xffffffffu, a1, 0);
          const float all0 = __shfl_sync(0xffffffffu, k0, 31);  // kappa of earlier tokens
          k0 = __shfl_up_sync(0xffffffffu, k0, 1);
          k1 = __shfl_up_sync(0xffffffffu, k1, 1);
          k0 = lane > 0 ? k0 : 0.0f;
          k1 = lane > 0 ? all0 + k1 : all0;
          // the first token's decay multiplies the initial state: without one its gradient is zero
          const bool none = item.y && !P.S0;
          __nv_bfloat16* dst = P.dg + t0 * P.Hv + h;
          if (lane < L)
            dst[(int64_t)lane * P.Hv] = __float2bfloat16_rn(lane == 0 && none ? 0.0f : a0 + f + k0);
          if (32 + lane < L) dst[(int64_t)(32 + lane) * P.Hv] = __float2bfloat16_rn(a1 + f + k1);
        }
        // ---- dv rows whose beta was floored: T' used the floored value
        if (tid < L && live && fabsf(gd[128 + tid]) == kBetaFloor) {
          const int64_t at = (t0 + tid) * P.Hv + h;
          const float ratio = P.beta[at] / gd[128 + tid];
          __nv_bfloat16* dv = P.dv + at * tm::D;
#pragma unroll 1
          for (int e = 0; e < tm::D; ++e)
            dv[e] = __float2bfloat16_rn(__bfloat162float(dv[e]) * ratio);
        }
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) {  // the tokens' own pairs
        const f32x2 o2 = *reinterpret_cast<const f32x2*>(own + 32 * half + 2 * q);
        aq[q] = fma2(o2, widen(kv[q]), aq[q]);
        ak[q] = fma2(o2, widen(qv[q]), ak[q]);
      }
      // ---- dq, dk: two bytes at a time into shared memory (a warp's 32 channels are 64 consecutive
      // bytes) where dO and dW were, out as boxes of tensor maps; a partial chunk row by row
      if (L == tm::C) {
        unsigned char* tile = smem + SM_OW + ((x - 1) & 1) * 32768 + (row >> 6) * 8192 + half * 4096 + (row & 7) * 2;
        const uint32_t c8 = ((uint32_t)row & 63) >> 3;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const float2 fq = parts(aq[q]), fk = parts(ak[q]);
          const uint32_t wq = pack2(fq.x, fq.y), wk = pack2(fk.x, fk.y);
          unsigned char* p0 = tile + 2 * q * 128 + ((c8 ^ ((2 * q) & 7)) << 4);
          unsigned char* p1 = tile + (2 * q + 1) * 128 + ((c8 ^ ((2 * q + 1) & 7)) << 4);
          *reinterpret_cast<uint16_t*>(p0) = (uint16_t)wq;
          *reinterpret_cast<uint16_t*>(p1) = (uint16_t)(wq >> 16);
          *reinterpret_cast<uint16_t*>(p0 + 16384) = (uint16_t)wk;
          *reinterpret_cast<uint16_t*>(p1 + 16384) = (uint16_t)(wk >> 16);
        }
        fence_proxy_async_smem();
      } else if (__all_sync(0xffffffffu, !*abort_flag)) {
        const int64_t rs = (int64_t)P.Hk * tm::D;
        const int64_t base = (t0 + 32 * half) * rs + hk * tm::D + row;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const float2 fq = parts(aq[q]), fk = parts(ak[q]);
          const int t = 32 * half + 2 * q;
          if (t < L) {
            P.dq[base + 2 * q * rs] = __float2bfloat16_rn(fq.x);
            P.dk[base + 2 * q * rs] = __float2bfloat16_rn(fk.x);
          }
          if (t + 1 < L) {
            P.dq[base + (2 * q + 1) * rs] = __float2bfloat16_rn(fq.y);
            P.dk[base + (2 * q + 1) * rs] = __float2bfloat16_rn(fk.y);
          }
        }
      }
      __syncwarp();
      if (tid == 0) out_item[y & 1] = item;
      if (lane == 0) mbar_arrive(&bars[B_O + (y & 1)]);
    }
    if (tid == 0) out_item[y & 1] = make_int4(0, 0, 0, 0);
    if (lane == 0) mbar_arrive(&bars[B_O + (y & 1)]);
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 136;");
    if (warp == W_PROD) {
      // ------------------------------------------------------------------ TMA producer ---------
      if (elect_one()) {
        prefetch_tensormap(&map_k);
        prefetch_tensormap(&map_q);
        prefetch_tensormap(&map_do);
        prefetch_tensormap(&map_dv);
      }
      uint32_t fix = 0;
      bool stop = false;
      int z = 0;  // copies of S and dS
      // Copies of one group of tiles, published on `full`.  Rows behind the sequence end hold whatever
      // follows in memory: a partial chunk's copies are awaited here and those rows cleared (`tiles`
      // 64-row half tiles one after the other from `clear`) before the group is published.
      auto group = [&](int full, uint32_t bytes, int L, unsigned char* clear, int tiles, auto&& copy) {
        const bool part = L < tm::C;
        uint64_t* fb = &bars[part ? B_FIX : full];
        if (elect_one()) {
          mbar_arrive_expect_tx(fb, bytes);
          copy(fb);
        }
        if (!part) return true;
        bool ok = __all_sync(0xffffffffu, mbar_wait(fb, fix)) != 0;
        fix ^= 1;
        if (!ok) {
          if (lane == 0) fail(GDN_ERR_TIMEOUT);
          mbar_wait(fb, fix ^ 1);  // its copies may still be under way
          return false;
        }
        clear_rows(clear, tiles, L, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[full]);
        return true;
      };
      auto may = [&](int b, int k) {  // the k-th use of a buffer: after its use k - 1 was released
        bool go = true;
        if (lane == 0) {
          if (k > 0) go = wait(b, (uint32_t)(k - 1) & 1);
          go = go && !*abort_flag;
        }
        return __shfl_sync(0xffffffffu, (int)go, 0) != 0;
      };
      for (int it = blockIdx.x, next = 0;; it = next) {
        if (lane == 0) next = (int)gridDim.x + atomicAdd(P.next, 1);  // used an item later
        Chunk ch;
        int64_t slot;
        int hk;
        if (!locate(it, ch, slot, hk)) break;
        const int32_t t0 = (int32_t)ch.t0;
        for (int gi = 0; gi < G; ++gi) {
          const int h = hk * G + gi;
          const size_t sh = (size_t)slot * P.Hv + h;
          unsigned char* ow = smem + SM_OW + (x & 1) * 32768;
          const bool go = may(B_HE + (x & 1), x >> 1);
          if (go && lane == 0) step_item[x & 3] = make_int4(ch.L, ch.first, hk, t0);
          __syncwarp();
          if (!go ||
              !group(B_H + (x & 1), TX_HEAD, ch.L, ow, 4, [&](uint64_t* fb) {
                tma_load_3d(ow, &map_do, fb, 0, h, t0);
                tma_load_3d(ow + 8192, &map_dv, fb, 0, h, t0);
                tma_load_3d(ow + 16384, &map_do, fb, 64, h, t0);
                tma_load_3d(ow + 24576, &map_dv, fb, 64, h, t0);
                bulk_load(smem + SM_U + (x & 1) * 16384, P.ws + P.at.u + sh * 16384, 16384, fb);
                bulk_load(smem + SM_GD + (x & 3) * GD_BYTES, P.ws + P.at.gd + sh * GD_BYTES, GD_BYTES,
                          fb);
              })) {
            stop = true;
            break;
          }
          ++x;
          if (!may(B_SE, z) ||
              !group(B_S, TX_STATE, tm::C, nullptr, 0, [&](uint64_t* fb) {
                bulk_load(smem + SM_S, P.ws + P.at.s + sh * 32768, 32768, fb);
                bulk_load(smem + SM_DS, P.ws + P.at.ds + sh * 32768, 32768, fb);
              })) {
            stop = true;
            break;
          }
          ++z;
          if (gi == 0) {  // needed last: after the head's own tiles
            if (!may(B_KQE, y) ||
                !group(B_KQ, TX_KQ, ch.L, smem + SM_KQ, 4, [&](uint64_t* fb) {
                  tma_load_3d(smem + SM_KQ, &map_k, fb, 0, hk, t0);
                  tma_load_3d(smem + SM_KQ + 8192, &map_q, fb, 0, hk, t0);
                  tma_load_3d(smem + SM_KQ + 16384, &map_k, fb, 64, hk, t0);
                  tma_load_3d(smem + SM_KQ + 24576, &map_q, fb, 64, hk, t0);
                })) {
              stop = true;
              break;
            }
            ++y;
          }
        }
        if (stop) break;
        next = __shfl_sync(0xffffffffu, next, 0);
      }
      // never leave the CTA with copies still landing in shared memory (each wait bounded)
      if (lane == 0) {
        bool ok = true;
        for (int b = 0; b < 2; ++b)  // uses b, b + 2, ... of each buffer
          if (x > b) ok = mbar_wait(&bars[B_H + b], (uint32_t)((x - 1 - b) >> 1) & 1) && ok;
        if (z > 0) ok = mbar_wait(&bars[B_S], (uint32_t)(z - 1) & 1) && ok;
        if (y > 0) ok = mbar_wait(&bars[B_KQ], (uint32_t)(y - 1) & 1) && ok;
        if (!ok) report(P.status, GDN_ERR_TIMEOUT);
      }
      __syncwarp();
      // the end of the items, after the wait above: it is one more phase of the same barrier
      if (!stop && may(B_HE + (x & 1), x >> 1) && lane == 0) {
        step_item[x & 3] = make_int4(0, 0, 0, 0);
        mbar_arrive(&bars[B_H + (x & 1)]);
      }
      __syncwarp();
    } else if (warp == W_MMA) {
      // ------------------------------------------------------------------ MMA issuer -----------
      const uint32_t id_p = idesc_bf16(128, 64, 0, 1);    // A = [dO; dW] K-major, B = U^T MN-major
      const uint32_t id_d1 = idesc_bf16(128, 128, 1, 0);  // A = S^T MN-major, B = [dO; dW] K-major
      const uint32_t id_d3 = idesc_bf16(128, 64, 1, 1);   // A = dS^T, B = U^T; also Q^T, K^T with dN, dM
      const uint64_t dOW = sdesc_sw128(sbase + SM_OW, 16, 1024);
      const uint64_t dU = sdesc_sw128(sbase + SM_U, 16384, 1024);
      const uint64_t dSt = sdesc_sw128(sbase + SM_S, 16384, 1024);
      const uint64_t dDSt = sdesc_sw128(sbase + SM_DS, 16384, 1024);
      const uint64_t dKt = sdesc_sw128(sbase + SM_KQ, 16384, 1024);
      const uint64_t dQt = sdesc_sw128(sbase + SM_KQ + 8192, 16384, 1024);
      const uint64_t dNM = sdesc_sw128(sbase + SM_NM, 16, 1024);
      const uint64_t dNn = sdesc_sw128(sbase + SM_NM, 8192, 1024);
      const uint64_t dMn = sdesc_sw128(sbase + SM_NM + 8192, 8192, 1024);
      auto live = [&]() { return __all_sync(0xffffffffu, !*abort_flag) != 0; };
      auto products_p = [&](int k) {  // MMA_p of step k: the previous step's B_NM said that D2 is read
        const bool have = wait_w(B_H + (k & 1), (k >> 1) & 1) && step_item[k & 3].x > 0 && live();
        if (have) {
          tc_fence_after();
          const uint64_t ow = dadd(dOW, (k & 1) * 32768), u = dadd(dU, (k & 1) * 16384);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_bf16_ss(tmem + TM_D2, dadd(ow, (ks >> 2) * 16384 + (ks & 3) * 32),
                          dadd(u, ks * 2048), id_p, ks > 0);
            mma_commit(&bars[B_P]);
          }
        }
        __syncwarp();
        return have;
      };
      for (bool have = products_p(0); have; ++y) {
        for (int gi = 0; gi < G; ++gi, ++x) {
          const bool st = wait_w(B_S, x & 1);
          const bool d = x == 0 || wait_w(B_D, (x - 1) & 1);  // the previous step's D1, D3, D4, D5 are read
          have = have && st && d;
          if (have && live()) {
            tc_fence_after();
            const uint64_t ow = dadd(dOW, (x & 1) * 32768), u = dadd(dU, (x & 1) * 16384);
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                mma_bf16_ss(tmem + TM_D1, dadd(dSt, ks * 2048),
                            dadd(ow, (ks >> 2) * 16384 + (ks & 3) * 32), id_d1, ks > 0);
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                mma_bf16_ss(tmem + TM_D3, dadd(dDSt, ks * 2048), dadd(u, ks * 2048), id_d3, ks > 0);
              mma_commit(&bars[B_SE]);
              mma_commit(&bars[B_HE + (x & 1)]);
            }
          }
          __syncwarp();
          const bool kq = wait_w(B_KQ, y & 1);
          const bool nm = wait_w(B_NM, x & 1);  // [dN; dM] written
          if (have && kq && nm && live()) {
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_bf16_ss(tmem + TM_D4, dadd(dKt, ks * 2048), dadd(dNM, ks * 32), id_d1, ks > 0);
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_bf16_ss(tmem + TM_D5, dadd(dQt, ks * 2048), dadd(dNn, ks * 2048), id_d3, ks > 0);
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_bf16_ss(tmem + TM_D5, dadd(dKt, ks * 2048), dadd(dMn, ks * 2048), id_d3, 1);
              mma_commit(&bars[B_N]);
              if (gi == G - 1) mma_commit(&bars[B_KQE]);
            }
          }
          __syncwarp();
          have = have && products_p(x + 1);
        }
      }
      if (elect_one()) {
        mma_commit(&bars[B_DRAIN]);
        if (!mbar_wait(&bars[B_DRAIN], 0)) fail(GDN_ERR_TIMEOUT);
      }
      __syncwarp();
    } else if (warp == W_OUT) {
      // ------------------------------------------------------------------ dq, dk ---------------
      for (;; ++y) {
        if (!wait_w(B_O + (y & 1), (y >> 1) & 1)) break;
        const int4 item = out_item[y & 1];
        if (item.x == 0) break;
        x += G;
        const int b = (x - 1) & 1;
        if (lane == 0 && item.x == tm::C && !*abort_flag) {
          const unsigned char* out = smem + SM_OW + b * 32768;
          const int32_t t0 = item.w, hk = item.z;
          tma_store_3d(&map_dq, out, 0, hk, t0);
          tma_store_3d(&map_dq, out + 8192, 64, hk, t0);
          tma_store_3d(&map_dk, out + 16384, 0, hk, t0);
          tma_store_3d(&map_dk, out + 24576, 64, hk, t0);
          bulk_commit();
          bulk_wait_read<0>();
        }
        __syncwarp();
        if (lane < 8) mbar_arrive(&bars[B_HE + b]);  // in place of the epilogue warps
      }
      if (lane == 0) bulk_wait<0>();  // nothing on its way out of shared memory
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_bwd_grads(const Args& a, const TcMaps& m, cudaStream_t s) {
  const int64_t n_tok = (int64_t)a.B * a.T, slots = max_slots(a.N, n_tok, tm::C);
  unsigned char* ws = reinterpret_cast<unsigned char*>(a.ws);
  GradParams p;
  p.beta = a.beta;
  p.S0 = a.S0;
  p.cu = a.cu;
  p.ws = ws;
  p.next = reinterpret_cast<int*>(ws + COUNTER);
  p.dq = (__nv_bfloat16*)a.dq;
  p.dk = (__nv_bfloat16*)a.dk_;
  p.dv = (__nv_bfloat16*)a.dv_;
  p.dg = (__nv_bfloat16*)a.dg;
  p.dbeta = (__nv_bfloat16*)a.dbeta;
  p.status = a.status;
  p.T = a.T;
  p.items = slots * a.Hk;
  p.at = tc_layout(slots, a.Hv);
  p.scale = a.scale;
  p.N = a.N;
  p.Hk = a.Hk;
  p.Hv = a.Hv;
  int sms = 0;
  cudaError_t e = sm_count(sms);
  if (e == cudaSuccess) e = allow_smem(bwd_grads_kernel, SM_BYTES);
  if (e != cudaSuccess) return e;
  const int64_t grid = p.items < sms ? p.items : sms;
  bwd_grads_kernel<<<(unsigned)grid, THREADS, SM_BYTES, s>>>(m.k, m.q, m.dout, m.dv, m.dq, m.dk, p);
  return cudaGetLastError();
}

size_t tc_workspace_bytes(int N, int64_t n_tok, int Hv) {
  return tc_layout(max_slots(N, n_tok, tm::C), Hv).end;
}

cudaError_t launch_tc(const Args& a, cudaStream_t s) {
  ChunkFusion f;
  const int64_t slots = max_slots(a.N, (int64_t)a.B * a.T, tm::C);
  // rows of the [T~; P] tiles are TMA coordinates; all three kernels count in 32 bits
  if (slots > 0x7fffffff / 128 / a.Hv || (int64_t)a.B * a.T > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const TcLayout at = tc_layout(slots, a.Hv);
  const int64_t n_tok = (int64_t)a.B * a.T, rows = slots * a.Hv * 128;
  const int64_t hk = (int64_t)a.Hk * tm::D, hv = (int64_t)a.Hv * tm::D;
  const unsigned char* tp = reinterpret_cast<const unsigned char*>(a.ws) + at.tp;
  TcMaps m;
  if (!make_tok_map(&m.q, a.q, a.Hk, n_tok, a.ts.q) || !make_tok_map(&m.k, a.k, a.Hk, n_tok, a.ts.k) ||
      !make_tok_map(&m.v, a.v, a.Hv, n_tok, a.ts.v) || !make_tok_map(&m.dout, a.dout, a.Hv, n_tok, hv) ||
      !make_tok_map(&m.dq, a.dq, a.Hk, n_tok, hk) || !make_tok_map(&m.dk, a.dk_, a.Hk, n_tok, hk) ||
      !make_tok_map(&m.dv, a.dv_, a.Hv, n_tok, hv) || !make_rows64_map(&m.t, tp, rows, 64) ||
      !make_rows64_map(&m.tp, tp, rows, 128))
    return cudaErrorInvalidValue;
  f.bwd_k = &m.k;
  f.bwd_q = &m.q;
  f.bwd_gd_off = at.gd;
  f.bwd_qg_off = at.qg;
  f.scale = a.scale;
  cudaError_t e = launch_chunk_prep(a.q, a.k, a.ts, a.g, a.beta, a.cu, a.N, a.B, a.T, a.Hk, a.Hv,
                                    a.ws, a.status, s, f);
  if (e == cudaSuccess) e = launch_bwd_chain(a, m, s);
  if (e == cudaSuccess) e = launch_bwd_grads(a, m, s);
  return e;
}

}  // namespace bwd
}  // namespace gdn
