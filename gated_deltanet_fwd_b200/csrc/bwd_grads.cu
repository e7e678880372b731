// bwd_grads.cu -- the parallel half of the tensor-core backward pass (bwd_tc.cuh): dq, dk, dg and dbeta of
// every chunk from the chains' states S, dS, U and dv.  Formulas in bwd_simt.cu.
//
// Work item = (chunk, k-head), persistent CTAs; an item runs through the v-heads that share the k-head.
// Everything is computed transposed -- lane i of tensor memory is channel i of q and k, columns are
// tokens -- so that every product has M = 128 and the sums over the shared heads stay in registers of
// the thread that owns the channel:
//   MMA_p  D2 = [dO; dW] U^T            M 128 (tokens), N 64, K 128
//   MMA_s  D1 = S^T [dO; dW]^T          M 128, N 128, K 128        (raw dQ | raw dKe)
//          D3 = dS^T U^T                M 128, N 64,  K 128        (raw dKw)
//   MMA_n  D4 = K^T [dN; dM]^T          M 128, N 128, K 64
//          D5 = Q^T dN + K^T dM         M 128, N 64,  K 64 twice
// Epilogue A (token rows): decay masks on D2 -> [dN; dM] in shared memory as bf16; the diagonals are a
// token's own pair p and dbeta; <S, dS> from shared memory.  Epilogue B (channel rows): Gamma and d applied
// in fp32, dq and dk summed over the heads, dgamma = q.dq + k.(dKe - dKw) reduced over channels.
// MMA_s does not wait for epilogue A, and a head's tiles are refilled as soon as MMA_s is done with them,
// while MMA_n and epilogue B of that head still run.
//
// Warp roles (320 threads): warps 0-7 the epilogues (lane quarter warp % 4; columns, in epilogue B tokens,
// split in two by warp / 4), warp 8 the TMA producer, warp 9 the MMA issuer.  Bounds: 144 KB of tiles per
// (chunk, v-head) at two v-heads a k-head against about 6 units of 64 x 128 x 128 products: HBM.
// Bounded waits and the abort protocol as in bwd_chain.cu.
#include "bwd_tc.cuh"
#include "ptx.cuh"

namespace gdn {
namespace bwd {
namespace {

using namespace ptx;

constexpr int THREADS = 320;
constexpr int W_PROD = 8;  // warp 9 issues the MMAs

// shared memory, from a 1024-aligned base
constexpr uint32_t SM_KQ = 0;               // [K; Q]: two 64-column halves x 128 rows x 128 B
constexpr uint32_t SM_OW = SM_KQ + 32768;   // [dO; dW]: the same
constexpr uint32_t SM_U = SM_OW + 32768;    // U^T: 128 rows x 128 B
constexpr uint32_t SM_S = SM_U + 16384;     // S: two halves x 128 rows x 128 B
constexpr uint32_t SM_DS = SM_S + 32768;    // dS: the same
constexpr uint32_t SM_NM = SM_DS + 32768;   // [dN; dM]: 128 rows x 128 B
constexpr uint32_t SM_GD = SM_NM + 16384;   // two records
constexpr uint32_t SM_RED = SM_GD + 2 * GD_BYTES;  // 2 x (dgamma parts [4][64], p [64], sums [8] + [8])
constexpr uint32_t RED_FLOATS = 4 * 64 + 64 + 16;
constexpr uint32_t SM_BAR = SM_RED + 2 * RED_FLOATS * 4;
constexpr uint32_t SM_BYTES = SM_BAR + 128 + 1024;
static_assert(SM_BYTES <= 232448, "shared memory budget");
constexpr uint32_t TX_KQ = 32768, TX_HEAD = 32768 + 16384 + 65536 + GD_BYTES;

enum { B_KQ = 0, B_KQE = 1, B_H = 2, B_HE = 3, B_P = 4, B_N = 5, B_FIX = 6, B_DRAIN = 7, B_COUNT = 8 };
enum { NB_NM = 1, NB_D = 2, NB_E = 3 };
constexpr int NB_ALL = 288;  // epilogue warps + issuer
constexpr int NB_EPI = 256;

// tensor-memory columns
constexpr uint32_t TM_D2 = 0, TM_D1 = 64, TM_D4 = 192, TM_D3 = 320, TM_D5 = 384;

struct GradParams {
  const float* beta;
  const int32_t* cu;
  const unsigned char* ws;
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
__device__ __forceinline__ float bf_at(const unsigned char* p) {
  return __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t*>(p) << 16);
}
// sum of the products of eight bf16 pairs
__device__ __forceinline__ float dot8(uint4 a, uint4 b, float acc) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), acc);
    acc = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), acc);
  }
  return acc;
}

__global__ void __launch_bounds__(THREADS, 1) bwd_grads_kernel(
    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_q,
    const __grid_constant__ CUtensorMap map_do, const __grid_constant__ CUtensorMap map_dv,
    const GradParams P) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM_BAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SM_BAR + B_COUNT * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM_BAR + B_COUNT * 8 + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = P.Hv / P.Hk;

  // item -> chunk and k-head; false past the last one or for a malformed cu_seqlens
  auto locate = [&](int64_t it, Chunk& ch, int64_t& slot, int& hk) {
    slot = it / P.Hk;
    hk = (int)(it - slot * P.Hk);
    return it < P.items && find_chunk(P.cu, P.T, P.N, tm::C, slot, ch, P.status);
  };
  {
    Chunk ch;
    int64_t slot;
    int hk;
    if (!locate(blockIdx.x, ch, slot, hk)) return;  // nothing allocated yet
  }
  if (tid == 0) {
    for (int i = 0; i < B_COUNT; ++i) mbar_init(&bars[i], i == B_KQE ? 8 : i == B_HE ? 9 : 1);
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
    if (*abort_flag) return false;
    if (mbar_wait(&bars[b], parity)) return true;
    fail(GDN_ERR_TIMEOUT);
    return false;
  };
  auto wait_w = [&](int b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };

  // `x` counts this CTA's (item, v-head) steps, `y` its items
  int x = 0, y = 0;
  if (warp < 8) {
    // ------------------------------------------------------------------ epilogues ------------
    const int quad = warp & 3, half = warp >> 2;
    const int row = 32 * quad + lane;  // epilogue A: row of [dO; dW]; epilogue B: channel
    const uint32_t lo = (uint32_t)(32 * quad) << 16;
    for (int64_t it = blockIdx.x;; it += gridDim.x, ++y) {
      Chunk ch;
      int64_t slot;
      int hk;
      if (!locate(it, ch, slot, hk)) break;
      const int L = ch.L;
      float aq[32], ak[32];  // dq, dk of channel `row`, tokens 32 half ..; summed over the heads
#pragma unroll
      for (int q = 0; q < 32; ++q) aq[q] = ak[q] = 0.0f;
      for (int gi = 0; gi < G; ++gi, ++x) {
        const int h = hk * G + gi;
        float* red = reinterpret_cast<float*>(smem + SM_RED) + (x & 1) * RED_FLOATS;
        float* own = red + 256;
        float* sums = own + 64;  // [8] <S, dS>, [8] k.dKw of the state part
        const float* gd = reinterpret_cast<const float*>(smem + SM_GD + (x & 1) * GD_BYTES);
        const bool in = wait_w(B_H, x & 1);
        // ---- epilogue A
        if (wait_w(B_P, x & 1) && in) {
          tc_fence_after();
          float d[32];
          tmem_ld32(tmem + lo + TM_D2 + 32 * half, d);
          const int r = row & 63;
          const float gr = gd[192 + r], mul = row < 64 ? P.scale : -1.0f;
          float diag = 0.0f;
          uint32_t pk[16];
#pragma unroll
          for (int q4 = 0; q4 < 8; ++q4) {
            const float4 gs = *reinterpret_cast<const float4*>(gd + 192 + 32 * half + 4 * q4);
            const float gv[4] = {gs.x, gs.y, gs.z, gs.w};
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int s = 32 * half + 4 * q4 + e;
              const float w = d[4 * q4 + e];
              if (s == r) diag = w;
              v[e] = s < r ? mul * ex2(gr - gv[e]) * w : 0.0f;
            }
            pk[2 * q4] = pack2(v[0], v[1]);
            pk[2 * q4 + 1] = pack2(v[2], v[3]);
          }
          unsigned char* nm = smem + SM_NM;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(nm + sw128(row, 32 * half + 8 * q)) =
                make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
          if ((r >> 5) == half) {  // this thread held the diagonal of its row
            if (row < 64) {
              own[r] = P.scale * diag;
            } else if (r < L) {
              const float b = gd[128 + r], t = diag / b / b;
              P.dbeta[(ch.t0 + r) * P.Hv + h] = __float2bfloat16_rn(t);
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        named_bar(NB_NM, NB_ALL);  // [dN; dM] written, D2 read; p visible to every epilogue warp
        // ---- <S, dS>
        float fr = 0.0f;
        if (in) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint32_t o = (uint32_t)(q * 256 + tid) * 16;
            fr = dot8(*reinterpret_cast<const uint4*>(smem + SM_S + o),
                      *reinterpret_cast<const uint4*>(smem + SM_DS + o), fr);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[B_HE]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) fr += __shfl_xor_sync(0xffffffffu, fr, o);
        if (lane == 0) sums[warp] = fr;
        // ---- epilogue B
        if (wait_w(B_N, x & 1)) {
          tc_fence_after();
          float kw = 0.0f, keep = 0.0f;
          const unsigned char* kt = smem + SM_KQ + (row >> 6) * 16384;
#pragma unroll
          for (int b = 0; b < 4; ++b) {  // 8 tokens at a time
            const int t0 = 32 * half + 8 * b;
            float d1a[8], d1b[8], d4a[8], d4b[8], d3[8], d5[8], v[8];
            tmem_ld8(tmem + lo + TM_D1 + t0, d1a);
            tmem_ld8(tmem + lo + TM_D4 + t0, d4a);
            tmem_ld8(tmem + lo + TM_D1 + 64 + t0, d1b);
            tmem_ld8(tmem + lo + TM_D4 + 64 + t0, d4b);
            tmem_ld8(tmem + lo + TM_D3 + t0, d3);
            tmem_ld8(tmem + lo + TM_D5 + t0, d5);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int t = t0 + e;
              // token t0 + e has t % 8 == e: the swizzle of this thread's column is fixed per e
              const uint32_t off = (uint32_t)t * 128 + (((((uint32_t)row & 63) >> 3) ^ e) << 4) +
                                   ((uint32_t)row & 7) * 2;
              const float kv = bf_at(kt + off), qv = bf_at(kt + 8192 + off);
              const float gm = gd[t], dd = gd[64 + t], p = own[t];
              const float fq = fmaf(P.scale * gm, d1a[e], d4a[e]);
              const float fe = fmaf(-gm, d1b[e], d4b[e]);
              const float w1 = dd * d3[e], fw = w1 + d5[e];
              v[e] = fmaf(qv, fq, kv * (fe - fw));
              kw = fmaf(kv, w1, kw);
              aq[8 * b + e] += fmaf(p, kv, fq);
              ak[8 * b + e] += fmaf(p, qv, fe + fw);
            }
            // sum over the warp's 32 channels: halve the tokens a lane holds three times, then add the
            // four lanes that are left with the same token: token t0 + (lane >> 2)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool up = lane & 16;
              const float give = up ? v[e] : v[e + 4], stay = up ? v[e + 4] : v[e];
              v[e] = stay + __shfl_xor_sync(0xffffffffu, give, 16);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const bool up = lane & 8;
              const float give = up ? v[e] : v[e + 2], stay = up ? v[e + 2] : v[e];
              v[e] = stay + __shfl_xor_sync(0xffffffffu, give, 8);
            }
            {
              const bool up = lane & 4;
              const float give = up ? v[0] : v[1], stay = up ? v[1] : v[0];
              v[0] = stay + __shfl_xor_sync(0xffffffffu, give, 4);
            }
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
            if ((lane & 3) == b) keep = v[0];  // lane 4 k + b ends up with token 8 b + k
          }
          red[quad * 64 + 32 * half + 8 * (lane & 3) + (lane >> 2)] = keep;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) kw += __shfl_xor_sync(0xffffffffu, kw, o);
          if (lane == 0) sums[8 + warp] = kw;
        }
        tc_fence_before();
        named_bar_arrive(NB_D, NB_ALL);  // D1, D3, D4, D5 read
        named_bar(NB_E, NB_EPI);         // dgamma parts and sums of all warps
        // ---- dg: suffix sums over the chunk, and what leaves through the state
        const bool live = __all_sync(0xffffffffu, !*abort_flag) != 0;
        if (warp == (x & 7) && live) {
          float f = 0.0f, k2 = 0.0f;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            f += sums[q];
            k2 += sums[8 + q];
          }
          f = fmaf(gd[63], f, k2);
          float a0 = 0.0f, a1 = 0.0f;  // tokens lane and 32 + lane
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            a0 += red[q * 64 + lane];
            a1 += red[q * 64 + 32 + lane];
          }
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float u0 = __shfl_down_sync(0xffffffffu, a0, o);
            const float u1 = __shfl_down_sync(0xffffffffu, a1, o);
            if (lane + o < 32) {
              a0 += u0;
              a1 += u1;
            }
          }
          a0 += __shfl_sync(0xffffffffu, a1, 0);
          __nv_bfloat16* dst = P.dg + ch.t0 * P.Hv + h;
          if (lane < L) dst[(int64_t)lane * P.Hv] = __float2bfloat16_rn(a0 + f);
          if (32 + lane < L) dst[(int64_t)(32 + lane) * P.Hv] = __float2bfloat16_rn(a1 + f);
        }
        // ---- dv rows whose beta was floored: T' used the floored value
        if (tid < L && live) {
          const int64_t at = (ch.t0 + tid) * P.Hv + h;
          const float b = P.beta[at], bf = gd[128 + tid];
          if (b != bf) {
            __nv_bfloat16* dv = P.dv + at * tm::D;
            for (int e = 0; e < tm::D; ++e)
              dv[e] = __float2bfloat16_rn(__bfloat162float(dv[e]) * (b / bf));
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[B_KQE]);  // K and Q of this item read
      // ---- dq, dk: lanes row, row ^ 1 swap, so that a store is a pair of channels
      if (__all_sync(0xffffffffu, !*abort_flag)) {
        const int odd = row & 1;
        const int64_t rs = (int64_t)P.Hk * tm::D;
        const int64_t base = (ch.t0 + 32 * half + odd) * rs + hk * tm::D + (row & ~1);
        uint32_t* oq = reinterpret_cast<uint32_t*>(P.dq + base);
        uint32_t* ok = reinterpret_cast<uint32_t*>(P.dk + base);
        const uint32_t sel = odd ? 0x7632u : 0x5410u;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const uint32_t mq = pack2(aq[2 * q], aq[2 * q + 1]), mk = pack2(ak[2 * q], ak[2 * q + 1]);
          const uint32_t nq = __shfl_xor_sync(0xffffffffu, mq, 1);
          const uint32_t nk = __shfl_xor_sync(0xffffffffu, mk, 1);
          if (32 * half + 2 * q + odd < L) {
            oq[(int64_t)q * rs] = odd ? __byte_perm(nq, mq, sel) : __byte_perm(mq, nq, sel);
            ok[(int64_t)q * rs] = odd ? __byte_perm(nk, mk, sel) : __byte_perm(mk, nk, sel);
          }
        }
      }
    }
  } else if (warp == W_PROD) {
    // ------------------------------------------------------------------ TMA producer ---------
    if (elect_one()) {
      prefetch_tensormap(&map_k);
      prefetch_tensormap(&map_q);
      prefetch_tensormap(&map_do);
      prefetch_tensormap(&map_dv);
    }
    uint32_t fix = 0;
    bool stop = false;
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
      for (int e = lane; e < tiles * (tm::C - L) * 8; e += 32) {
        const int tile = e / ((tm::C - L) * 8), rest = e - tile * ((tm::C - L) * 8);
        *reinterpret_cast<uint4*>(clear + tile * 8192 + (L + rest / 8) * 128 + (rest % 8) * 16) =
            make_uint4(0u, 0u, 0u, 0u);
      }
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
    for (int64_t it = blockIdx.x; !stop; it += gridDim.x) {
      Chunk ch;
      int64_t slot;
      int hk;
      if (!locate(it, ch, slot, hk)) break;
      const int32_t t0 = (int32_t)ch.t0;
      for (int gi = 0; gi < G; ++gi) {
        const int h = hk * G + gi;
        const size_t sh = (size_t)slot * P.Hv + h;
        if (!may(B_HE, x)) {
          stop = true;
          break;
        }
        if (!group(B_H, TX_HEAD, ch.L, smem + SM_OW, 4, [&](uint64_t* fb) {
              tma_load_3d(smem + SM_OW, &map_do, fb, 0, h, t0);
              tma_load_3d(smem + SM_OW + 8192, &map_dv, fb, 0, h, t0);
              tma_load_3d(smem + SM_OW + 16384, &map_do, fb, 64, h, t0);
              tma_load_3d(smem + SM_OW + 24576, &map_dv, fb, 64, h, t0);
              bulk_load(smem + SM_U, P.ws + P.at.u + sh * 16384, 16384, fb);
              bulk_load(smem + SM_S, P.ws + P.at.s + sh * 32768, 32768, fb);
              bulk_load(smem + SM_DS, P.ws + P.at.ds + sh * 32768, 32768, fb);
              bulk_load(smem + SM_GD + (x & 1) * GD_BYTES, P.ws + P.at.gd + sh * GD_BYTES, GD_BYTES,
                        fb);
            })) {
          stop = true;
          break;
        }
        ++x;
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
    }
    // never leave the CTA with copies still landing in shared memory (each wait bounded)
    if (lane == 0) {
      if (x > 0 && !mbar_wait(&bars[B_H], (uint32_t)(x - 1) & 1)) report(P.status, GDN_ERR_TIMEOUT);
      if (y > 0 && !mbar_wait(&bars[B_KQ], (uint32_t)(y - 1) & 1)) report(P.status, GDN_ERR_TIMEOUT);
    }
  } else {
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
    for (int64_t it = blockIdx.x;; it += gridDim.x, ++y) {
      Chunk ch;
      int64_t slot;
      int hk;
      if (!locate(it, ch, slot, hk)) break;
      for (int gi = 0; gi < G; ++gi, ++x) {
        const bool have = wait_w(B_H, x & 1);
        if (have && live()) {
          tc_fence_after();
          // D2 was read before the previous step's NB_NM
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_bf16_ss(tmem + TM_D2, dadd(dOW, (ks >> 2) * 16384 + (ks & 3) * 32),
                          dadd(dU, ks * 2048), id_p, ks > 0);
            mma_commit(&bars[B_P]);
          }
        }
        __syncwarp();
        if (x > 0) named_bar(NB_D, NB_ALL);  // the previous step's D1, D3, D4, D5 are read
        if (have && live()) {
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_bf16_ss(tmem + TM_D1, dadd(dSt, ks * 2048),
                          dadd(dOW, (ks >> 2) * 16384 + (ks & 3) * 32), id_d1, ks > 0);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_bf16_ss(tmem + TM_D3, dadd(dDSt, ks * 2048), dadd(dU, ks * 2048), id_d3, ks > 0);
            mma_commit(&bars[B_HE]);
          }
        }
        __syncwarp();
        const bool kq = wait_w(B_KQ, y & 1);
        named_bar(NB_NM, NB_ALL);  // [dN; dM] written
        if (have && kq && live()) {
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
          }
        }
        __syncwarp();
      }
    }
    if (x > 0) named_bar(NB_D, NB_ALL);  // the last step's arrivals
    if (elect_one()) {
      mma_commit(&bars[B_DRAIN]);
      if (!mbar_wait(&bars[B_DRAIN], 0)) fail(GDN_ERR_TIMEOUT);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_bwd_grads(const Args& a, cudaStream_t s) {
  const int64_t n_tok = (int64_t)a.B * a.T, slots = max_slots(a.N, n_tok, tm::C);
  unsigned char* ws = reinterpret_cast<unsigned char*>(a.ws);
  GradParams p;
  p.beta = a.beta;
  p.cu = a.cu;
  p.ws = ws;
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
  if (n_tok > 0x7fffffff) return cudaErrorInvalidConfiguration;  // TMA coordinates are 32-bit
  CUtensorMap mk, mq, mo, mv;
  const int64_t hv = (int64_t)a.Hv * tm::D;
  if (!make_tok_map(&mk, a.k, a.Hk, n_tok, a.ts.k) || !make_tok_map(&mq, a.q, a.Hk, n_tok, a.ts.q) ||
      !make_tok_map(&mo, a.dout, a.Hv, n_tok, hv) || !make_tok_map(&mv, a.dv_, a.Hv, n_tok, hv))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(bwd_grads_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SM_BYTES);
  if (e != cudaSuccess) return e;
  const int64_t grid = p.items < sms ? p.items : sms;
  bwd_grads_kernel<<<(unsigned)grid, THREADS, SM_BYTES, s>>>(mk, mq, mo, mv, p);
  return cudaGetLastError();
}

size_t tc_workspace_bytes(int N, int64_t n_tok, int Hv) {
  return tc_layout(max_slots(N, n_tok, tm::C), Hv).end;
}

cudaError_t launch_tc(const Args& a, cudaStream_t s) {
  ChunkFusion f;
  const TcLayout at = tc_layout(max_slots(a.N, (int64_t)a.B * a.T, tm::C), a.Hv);
  f.bwd_gd_off = at.gd;
  f.bwd_qg_off = at.qg;
  f.scale = a.scale;
  cudaError_t e = launch_chunk_prep(a.q, a.k, a.ts, a.g, a.beta, a.cu, a.N, a.B, a.T, a.Hk, a.Hv,
                                    a.ws, a.status, s, f);
  if (e == cudaSuccess) e = launch_bwd_chain(a, s);
  if (e == cudaSuccess) e = launch_bwd_grads(a, s);
  return e;
}

}  // namespace bwd
}  // namespace gdn
