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
  int64_t base = 0;
#pragma unroll 1
  for (int m = 0; m <= n; ++m) {
    const int64_t a = cu[m], b = cu[m + 1];
    if (a < 0 || b < a || b > T) return false;
    if (m < n) base += (b - a + C - 1) / C;
    s_beg = a;
    s_end = b;
  }
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
  int64_t base = 0;
#pragma unroll 1
  for (int m = 0; m < N; ++m) {
    const int64_t a = cu[m], b = cu[m + 1];
    if (a < 0 || b < a || b > T) {
      if (threadIdx.x == 0) report(status, GDN_ERR_DEVICE_ARG);
      return false;
    }
    const int64_t nch = (b - a + C - 1) / C;
    if (slot < base + nch) {
      ch.n = m;
      ch.t0 = a + (slot - base) * C;
      ch.first = slot == base;
      ch.L = (int)(b - ch.t0 < C ? b - ch.t0 : C);
      return true;
    }
    base += nch;
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
    if (!cu) return find_chunk(cu, T, N, C, slot, ch, status);
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
