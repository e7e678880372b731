// bwd_tc.cuh -- layout of the tensor-core backward pass of the chunked rule (bf16, dk = dv = 128,
// chunks of 64 tokens); the mathematics is in bwd_simt.cu.
//
// Three kernels, one after the other on the caller's stream:
//   chunk_prep<BWD>   (chunk_prep.cu)  per (chunk, k-head): T~, P, scale Gamma Q and the decay records
//   bwd_chain         (bwd_chain.cu)   per (sequence, v-head): a walk forward, which leaves the state S entering
//                                      each chunk and U, and a walk backward: dS leaving each chunk, and dv
//   bwd_grads         (bwd_grads.cu)   per (chunk, k-head): dq, dk, dg, dbeta
// Only the two chains are serial; they carry the fp32 state (or its gradient) in tensor memory and leave
// bf16 copies, the same roundings their own next product uses, so that everything else is parallel.
//
// T' = diag(beta) T~ (chunk_prep.cu): with X = V - diag(Gamma) K S^T,
//   U = beta o (T~ X),   dW = T~^T (beta o dU),   dbeta_r = dW_r . U_r / beta_r^2.
//
// Workspace from its 256-byte-aligned base (n = slots * Hv, a slot being a chunk's ordinal):
//   [0, 1024)        status word, item counter of bwd_grads (at 8), padding
//   TP [n][128][64]  bf16: rows 0..63 T~, rows 64..127 scale P
//   GD [n][4][64]    fp32: Gamma, d, beta (floored), gamma log2 e
//   S  [n][2][128][64]  bf16: two 64-column halves of the state (rows: value index)
//   DS [n][2][128][64]  bf16: the gradient of the state leaving the chunk
//   U  [n][128][64]  bf16: U^T (rows: value index, columns: tokens of the chunk)
//   QG [n][2][64][64]   bf16: two 64-column halves of scale Gamma Q
// S, DS, U and QG are kept as the 128-byte-swizzled images that the MMAs read (ptx::sw128), written and read by
// plain bulk copies.
#pragma once

#include "bwd_internal.cuh"
#include "chunk_tm.cuh"

namespace gdn {
namespace bwd {

struct TcLayout {
  size_t tp, gd, s, ds, u, qg, end;
};

__host__ __device__ inline TcLayout tc_layout(int64_t slots, int Hv) {
  const size_t n = (size_t)slots * Hv;
  TcLayout l;
  l.tp = HEADER;
  l.gd = l.tp + n * 16384;
  l.s = l.gd + n * GD_BYTES;
  l.ds = l.s + n * 32768;
  l.u = l.ds + n * 32768;
  l.qg = l.u + n * 16384;
  l.end = l.qg + n * 16384;
  return l;
}

// One warp: zeros into rows L .. 63 of `tiles` 64-row, 128-byte-wide tiles, one after the other.  Eight lanes a
// row; no division by L (9000 cycles against 500 for four tiles of which one row is kept).
__device__ __forceinline__ void clear_rows(unsigned char* tile, int tiles, int L, int lane) {
  for (int i = 0; i < tiles; ++i, tile += 8192)
#pragma unroll 4
    for (int r = L + (lane >> 3); r < tm::C; r += 4)
      *reinterpret_cast<uint4*>(tile + r * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
}

// Tensor maps of a call: boxes of 64 tokens x 64 channels of one head; t: 64 rows of T~, tp: 128 of [T~; P].
struct TcMaps {
  CUtensorMap q, k, v, dout, dq, dk, dv, t, tp;
};

cudaError_t launch_bwd_chain(const Args& a, const TcMaps& m, cudaStream_t s);
cudaError_t launch_bwd_grads(const Args& a, const TcMaps& m, cudaStream_t s);

}  // namespace bwd
}  // namespace gdn
