// bwd_internal.cuh -- declarations shared by the kernels of the layer core's backward passes.
#pragma once

#include "gdn_internal.cuh"

namespace gdn {
namespace bwd {

constexpr size_t HEADER = 1024;  // status word and padding at the start of the rule's workspace
constexpr size_t COUNTER = 8;    // tensor-core path: items handed out (bwd_grads.cu), in the header

// Arguments of gdn_chunk_bwd after the host checks.
struct Args {
  const void *q, *k, *v, *dout;
  TokStrides ts;
  const float *g, *beta, *S0, *dST;
  const int32_t* cu;
  gdn_dtype dt;
  float scale;
  int N, B;
  int64_t T;
  int Hk, Hv, dk, dv, C;
  void *dq, *dk_, *dv_, *dg, *dbeta;
  float* dS0;
  void* ws;
  size_t ws_bytes;
  int* status;
};

// Record of a (slot, v-head) on the tensor-core path: Gamma, d, beta (floored), gamma log2 e; 64 fp32 each
constexpr size_t GD_BYTES = 1024;

size_t simt_workspace_bytes(int N, int64_t n_tok, int Hv, int dk, int dv, int C);
cudaError_t launch_simt(const Args& a, cudaStream_t s);

// Tensor-core path (bf16, dk = dv = 128, chunk 64, at least one token); see bwd_tc.cuh.
size_t tc_workspace_bytes(int N, int64_t n_tok, int Hv);
cudaError_t launch_tc(const Args& a, cudaStream_t s);

// A "slot" is the ordinal of a chunk among all chunks of all sequences, in sequence order.
__host__ __device__ inline int64_t max_slots(int N, int64_t n_tok, int C) {
  return (n_tok + C - 1) / C + N;
}

// The smallest magnitude of beta used in T' (see bwd_simt.cu): 2^-30.
constexpr float kBetaFloor = 1.0f / (1 << 30);
__device__ __forceinline__ float floor_beta(float b) {
  return fabsf(b) < kBetaFloor ? copysignf(kBetaFloor, b) : b;
}

// The searches in cu_seqlens below are a warp's work: its lanes read 32 entries at once, since one after the other
// each costs a way to L2.  (32768 tokens as 2048 sequences: the walks 102 ms so, 9.3 ms now; as four sequences 577
// and 582 us.)  Every lane of the warp calls them and gets the answer.
constexpr uint32_t kWarp = 0xffffffffu;

// Whether [a, b) cannot be the tokens of a sequence.
__device__ __forceinline__ bool bad_range(int64_t a, int64_t b, int64_t T) { return a < 0 || b < a || b > T; }

// Sequence n's tokens and the slot of its first chunk; false for a malformed cu_seqlens met up to n
// (nothing may be read through it).
__device__ __forceinline__ bool seq_range(const int32_t* cu, int64_t T, int n, int C, int64_t& s_beg,
                                          int64_t& s_end, int64_t& slot0) {
  if (!cu) {
    s_beg = (int64_t)n * T;
    s_end = s_beg + T;
    slot0 = (int64_t)n * ((T + C - 1) / C);
    return true;
  }
  const int lane = threadIdx.x & 31;
  int64_t base = 0;
#pragma unroll 1
  for (int m0 = 0; m0 <= n; m0 += 128) {
    int32_t a[4], b[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int m = m0 + 32 * q + lane;
      a[q] = m <= n ? cu[m] : 0;
      b[q] = m <= n ? cu[m + 1] : 0;
    }
    bool bad = false;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      bad = bad || bad_range(a[q], b[q], T);
      if (m0 + 32 * q + lane < n) base += ((int64_t)b[q] - a[q] + C - 1) / C;
    }
    if (__any_sync(kWarp, bad)) return false;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) base += __shfl_xor_sync(kWarp, base, o);
  s_beg = cu[n];
  s_end = cu[n + 1];
  slot0 = base;
  return true;
}

struct Chunk {
  int n, L;
  int64_t t0;
  bool first;  // of its sequence
};

// The chunk of a slot; false past the last one or for a malformed cu_seqlens (reported).
__device__ __forceinline__ bool find_chunk(const int32_t* cu, int64_t T, int N, int C, int64_t slot,
                                           Chunk& ch, int* status) {
  if (!cu) {
    const int64_t per = (T + C - 1) / C;
    if (per == 0 || slot >= per * N) return false;
    ch.n = (int)((uint32_t)slot / (uint32_t)per);  // both below 2^31: they count blocks of a grid
    const int64_t c = slot - (int64_t)ch.n * per;
    ch.t0 = (int64_t)ch.n * T + c * C;
    ch.first = c == 0;
    ch.L = (int)(T - c * C < C ? T - c * C : C);
    return true;
  }
  const int lane = threadIdx.x & 31;
  int64_t base = 0;  // slot of the first chunk of sequence m0
#pragma unroll 1
  for (int m0 = 0; m0 < N; m0 += 32) {
    const int m = m0 + lane;
    const int64_t a = m < N ? cu[m] : 0, b = m < N ? cu[m + 1] : 0;
    const uint32_t wrong = __ballot_sync(kWarp, bad_range(a, b, T));
    const int64_t nch = (b - a + C - 1) / C;
    int64_t end = nch;  // slots up to and with this lane's sequence
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t l = __shfl_up_sync(kWarp, end, o);
      if (lane >= o) end += l;
    }
    end += base;
    // of lanes behind a malformed entry nothing is used: it comes before what they hold
    const uint32_t hit = __ballot_sync(kWarp, m < N && slot < end);
    const int take = hit ? __ffs(hit) - 1 : 31;
    if (wrong && __ffs(wrong) - 1 <= take) {
      if (threadIdx.x == 0) report(status, GDN_ERR_DEVICE_ARG);
      return false;
    }
    base = __shfl_sync(kWarp, end, take);
    if (hit) {
      const int64_t first = __shfl_sync(kWarp, end - nch, take), t = __shfl_sync(kWarp, a, take);
      ch.n = m0 + take;
      ch.t0 = t + (slot - first) * C;
      ch.first = slot == first;
      ch.L = (int)min((int64_t)C, __shfl_sync(kWarp, b, take) - ch.t0);
      return true;
    }
  }
  return false;
}

// find_chunk for slots that never decrease: the search goes on from the sequence found last, so a
// persistent block reads each entry of cu_seqlens about once.
struct ChunkCursor {
  int m = 0;
  bool bad = false;  // a malformed entry was met (and reported)
  int64_t base = 0, a = -1, b = -1;  // sequence m: slot of its first chunk, its tokens (a < 0: not read yet)
  __device__ __forceinline__ bool find(const int32_t* cu, int64_t T, int N, int C, int64_t slot,
                                       Chunk& ch, int* status) {
    if (!cu) return find_chunk(nullptr, T, N, C, slot, ch, status);
#pragma unroll 1
    for (; m < N; ++m, a = -1) {
      if (a < 0) {
        a = cu[m];
        b = cu[m + 1];
        if (a < 0 || b < a || b > T) {
          if (threadIdx.x == 0) report(status, GDN_ERR_DEVICE_ARG);
          a = -1;
          bad = true;
          return false;
        }
      }
      const int64_t nch = (b - a + C - 1) / C;
      if (slot < base + nch) {
        ch.n = m;
        ch.t0 = a + (slot - base) * C;
        ch.L = (int)(b - ch.t0 < C ? b - ch.t0 : C);
        ch.first = slot == base;
        return true;
      }
      base += nch;
    }
    return false;
  }
};

}  // namespace bwd
}  // namespace gdn
