// bwd_api.cu -- the exported C ABI of the training calls (include/gdn.h): backward passes and 8-bit
// activation checkpoints.  As in gdn_api.cu every check happens on the host before anything is
// enqueued.
#include <nvtx3/nvToolsExt.h>

#include "bwd_internal.cuh"

using namespace gdn;

namespace {

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};

inline bool bad_dtype(gdn_dtype d) { return d != GDN_BF16 && d != GDN_F32; }
inline size_t elem(gdn_dtype d) { return d == GDN_BF16 ? 2 : 4; }
inline gdn_status from_cuda(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }
inline bool ptr_ok(const void* p) { return p != nullptr && aligned16(p); }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// whether every pointer (null is fine) lies on a multiple of `bytes`, a power of two
template <typename... Ptr>
inline bool aligned_to(size_t bytes, Ptr... p) {
  return (((reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0) && ...);
}

// A range of device memory that a call reads or writes; ranges without a pointer or bytes overlap
// nothing.
struct Span {
  const void* p;
  size_t n;
};
inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const char *x = (const char*)a.p, *y = (const char*)b.p;
  return x < y + b.n && y < x + a.n;
}
// whether some output overlaps an input or another output
template <size_t I, size_t O>
bool clash(const Span (&in)[I], const Span (&out)[O]) {
  for (size_t o = 0; o < O; ++o) {
    for (size_t i = 0; i < I; ++i)
      if (overlap(out[o], in[i])) return true;
    for (size_t i = 0; i < o; ++i)
      if (overlap(out[o], out[i])) return true;
  }
  return false;
}

inline size_t round256(size_t b) { return (b + 255) & ~size_t(255); }
inline bool ws_ok(const void* ws, size_t have, size_t need) {
  return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && have >= need;
}

// Partial rows of the sums over tokens that a call's workspace has room for: enough for the blocks
// of a launch on a B200, fewer for short inputs.
int64_t gates_parts(int64_t n_tok) { return n_tok < 512 ? n_tok : 512; }
int64_t norm_parts(int64_t rows, int dim) {
  const int64_t per = 2 * (256 / (dim / 8)), need = (rows + per - 1) / per;
  return need < 1184 ? need : 1184;
}
int64_t conv_parts(int64_t n_tok, int C) {
  const int64_t tiles = (C + 255) / 256, most = 4736 / tiles > 1 ? 4736 / tiles : 1;
  const int64_t need = (n_tok + 15) / 16;
  return need < 1 ? 1 : need < most ? need : most;
}
// Whether the rule's backward pass runs on tensor cores: the shape of the forward's tensor-core path, and
// at least 512 gate values (tokens x v-heads).  The tensor-core kernels round their operands to bf16.  That costs
// dg 3e-3 of its norm where many independent values make it up, and more where few do, since their sum of squares
// may happen to be small.  Share of one-head calls whose dg is over 5e-3 of its norm off, 512 to 1024 calls each,
// at 16, 64, 128, 256, 512 and 1024 tokens: 16, 8, 5, 2, 0.4 and 0.2 % where a token keeps e^-6 of the state on
// average, 12, 8, 6, 2, 1 and 0.6 % where it keeps 97 % -- but 14 to 31 % at every length where it
// keeps more than the call is long, which no count of values tells.  The CUDA-core kernels carry fp32
// throughout.  At 100 tokens and 4 v-heads they take 84 us, the tensor cores 47.
constexpr int64_t TC_MIN_VALUES = 512;
bool tensor_cores(gdn_dtype dtype, int64_t n_tok, int Hv, int dk, int dv, int chunk) {
  return dtype == GDN_BF16 && dk == 128 && dv == 128 && chunk == 64 && n_tok * Hv >= TC_MIN_VALUES;
}
// Chunk length on CUDA cores: the caller's, but no longer than is fast (it changes no result beyond rounding).
// bf16, d = 128, one v-head per k-head and 1 token: 33 us with chunks of 16, 49 with 32, 98 with 64; 250
// tokens, 2 v-heads: 129, 143, 221; 500 tokens, 1 v-head: 182, 172, 231.  fp32, d = 128, 1024 tokens, 4
// v-heads: 327, 290, 365; sixteen such sequences of 8 v-heads: 3.2 ms with 32, 3.5 with 64.
int simt_chunk(int64_t n_tok, int chunk) {
  const int most = n_tok <= 256 ? 16 : 32;
  return chunk < most ? chunk : most;
}
bool norm_dim_ok(int dim) {
  return dim == 8 || dim == 16 || dim == 32 || dim == 64 || dim == 128 || dim == 256;
}

// gdn_gates_bwd of the tokens that cu_seqlens spans, of all where it is null
gdn_status gates_bwd(const void* a, const void* b, gdn_dtype dtype, const float* A_log,
                     const float* dt_bias, const void* dg, const void* dbeta,
                     const int32_t* cu_seqlens, int N, int64_t n_tok, int Hv, void* da,
                     void* db, float* dA_log, float* ddt_bias, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (bad_dtype(dtype) || n_tok < 0 || Hv < 1 || N < 0) return GDN_ERR_INVALID_ARG;
  if (!A_log || !dt_bias || !dA_log || !ddt_bias) return GDN_ERR_INVALID_ARG;
  if (n_tok > 0 && (!a || !b || !dg || !dbeta || !da || !db)) return GDN_ERR_INVALID_ARG;
  if (!aligned_to(elem(dtype), a, b, dg, dbeta, da, db) ||
      !aligned_to(4, A_log, dt_bias, dA_log, ddt_bias, cu_seqlens))
    return GDN_ERR_INVALID_ARG;
  if (!ws_ok(workspace, workspace_bytes, gdn_gates_bwd_workspace_size(n_tok, Hv)))
    return GDN_ERR_INVALID_ARG;
  const size_t n = (size_t)n_tok * Hv * elem(dtype), hb = (size_t)Hv * sizeof(float);
  const Span in[] = {{a, n},      {b, n},        {dg, n}, {dbeta, n},
                     {A_log, hb}, {dt_bias, hb}, {cu_seqlens, (size_t)(N + 1) * 4}};
  const Span out[] = {{da, n}, {db, n}, {dA_log, hb}, {ddt_bias, hb}, {workspace, workspace_bytes}};
  if (clash(in, out)) return GDN_ERR_INVALID_ARG;
  return from_cuda(launch_gates_bwd(a, b, dtype, A_log, dt_bias, dg, dbeta, TokRange{cu_seqlens, N}, n_tok,
                                    Hv, da, db, dA_log, ddt_bias, (float*)workspace,
                                    gates_parts(n_tok), as_stream(stream)));
}

// gdn_gated_rmsnorm_bwd of the rows of the tokens that cu_seqlens spans, of all where it is null
gdn_status rmsnorm_bwd(const void* dy, const void* x, const float* x_scales, const void* z,
                       const float* z_scales, gdn_dtype dtype, const float* w, float eps,
                       const int32_t* cu_seqlens, int N, int rows_per_token, int64_t n_rows, int dim,
                       void* dx, void* dz, float* dw, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (bad_dtype(dtype) || n_rows < 0 || dim < 1 || !(eps >= 0.0f)) return GDN_ERR_INVALID_ARG;
  if (N < 0 || rows_per_token < 1 || n_rows % rows_per_token != 0) return GDN_ERR_INVALID_ARG;
  if (!norm_dim_ok(dim)) return GDN_ERR_UNSUPPORTED;
  if (!w || !dw) return GDN_ERR_INVALID_ARG;
  if (!ws_ok(workspace, workspace_bytes, gdn_gated_rmsnorm_bwd_workspace_size(n_rows, dim)))
    return GDN_ERR_INVALID_ARG;
  if ((x_scales == nullptr) != (z_scales == nullptr)) return GDN_ERR_INVALID_ARG;
  if (n_rows > 0 && (!ptr_ok(dy) || !ptr_ok(x) || !ptr_ok(z) || !ptr_ok(dx) || !ptr_ok(dz)))
    return GDN_ERR_INVALID_ARG;
  if (!aligned_to(4, x_scales, z_scales, cu_seqlens, w, dw)) return GDN_ERR_INVALID_ARG;
  const size_t n = (size_t)n_rows * dim, nb = n * elem(dtype), kept = x_scales ? n : nb;
  const size_t sb = x_scales ? (size_t)n_rows * sizeof(float) : 0, wb = dim * sizeof(float);
  const Span in[] = {{dy, nb}, {x, kept}, {z, kept}, {x_scales, sb}, {z_scales, sb}, {w, wb},
                     {cu_seqlens, (size_t)(N + 1) * 4}};
  const Span out[] = {{dx, nb}, {dz, nb}, {dw, wb}, {workspace, workspace_bytes}};
  if (clash(in, out)) return GDN_ERR_INVALID_ARG;
  return from_cuda(launch_rmsnorm_bwd(dy, x, x_scales, z, z_scales, dtype, w, eps,
                                      TokRange{cu_seqlens, N}, rows_per_token, n_rows, dim, dx, dz, dw,
                                      (float*)workspace, norm_parts(n_rows, dim), as_stream(stream)));
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------------------- gates -----

size_t gdn_gates_bwd_workspace_size(int64_t n_tok, int Hv) {
  if (n_tok < 0 || Hv < 1) return 256;
  return round256(256 + (size_t)gates_parts(n_tok) * 2 * Hv * sizeof(float));
}

gdn_status gdn_gates_bwd(const void* a, const void* b, gdn_dtype dtype, const float* A_log,
                         const float* dt_bias, const void* dg, const void* dbeta, int64_t n_tok,
                         int Hv, void* da, void* db, float* dA_log, float* ddt_bias,
                         void* workspace, size_t workspace_bytes, void* stream) {
  CallRange range_("gdn_gates_bwd");
  return gates_bwd(a, b, dtype, A_log, dt_bias, dg, dbeta, nullptr, 0, n_tok, Hv, da, db, dA_log, ddt_bias,
                   workspace, workspace_bytes, stream);
}

gdn_status gdn_gates_bwd_varlen(const void* a, const void* b, gdn_dtype dtype, const float* A_log,
                                const float* dt_bias, const void* dg, const void* dbeta,
                                const int32_t* cu_seqlens, int N, int64_t n_tok, int Hv, void* da,
                                void* db, float* dA_log, float* ddt_bias, void* workspace,
                                size_t workspace_bytes, void* stream) {
  CallRange range_("gdn_gates_bwd_varlen");
  return gates_bwd(a, b, dtype, A_log, dt_bias, dg, dbeta, cu_seqlens, N, n_tok, Hv, da, db, dA_log, ddt_bias,
                   workspace, workspace_bytes, stream);
}

// ------------------------------------------------------------------- 8-bit checkpoints -----

gdn_status gdn_act_pack8(const void* x, gdn_dtype dtype, int64_t n_rows, int dim, int group,
                         int8_t* codes, float* scales, void* stream) {
  CallRange range_("gdn_act_pack8");
  if (bad_dtype(dtype) || n_rows < 0 || dim < 1 || group < 1 || dim % group != 0)
    return GDN_ERR_INVALID_ARG;
  if (!norm_dim_ok(group)) return GDN_ERR_UNSUPPORTED;
  if (n_rows == 0) return GDN_OK;
  if (!ptr_ok(x) || !ptr_ok(codes) || !scales || !aligned4(scales)) return GDN_ERR_INVALID_ARG;
  const size_t n = (size_t)n_rows * dim;
  const Span in[] = {{x, n * elem(dtype)}};
  const Span out[] = {{codes, n}, {scales, n / group * sizeof(float)}};
  if (clash(in, out)) return GDN_ERR_INVALID_ARG;
  return from_cuda(launch_act_pack8(x, dtype, n_rows * (dim / group), group, codes, scales,
                                    as_stream(stream)));
}

gdn_status gdn_act_unpack8(const int8_t* codes, const float* scales, gdn_dtype dtype,
                           int64_t n_rows, int dim, int group, void* x, void* stream) {
  CallRange range_("gdn_act_unpack8");
  if (bad_dtype(dtype) || n_rows < 0 || dim < 1 || group < 1 || dim % group != 0)
    return GDN_ERR_INVALID_ARG;
  if (!norm_dim_ok(group)) return GDN_ERR_UNSUPPORTED;
  if (n_rows == 0) return GDN_OK;
  if (!ptr_ok(x) || !ptr_ok(codes) || !scales || !aligned4(scales)) return GDN_ERR_INVALID_ARG;
  const size_t n = (size_t)n_rows * dim;
  const Span in[] = {{codes, n}, {scales, n / group * sizeof(float)}};
  const Span out[] = {{x, n * elem(dtype)}};
  if (clash(in, out)) return GDN_ERR_INVALID_ARG;
  return from_cuda(launch_act_unpack8(codes, scales, dtype, n_rows * (dim / group), group, x,
                                      as_stream(stream)));
}

// -------------------------------------------------------------------------------- norm -----

gdn_status gdn_gated_rmsnorm_ckpt8(const void* x, const void* z, gdn_dtype dtype, const float* w,
                                   float eps, int64_t n_rows, int dim, void* y, int8_t* x_codes,
                                   float* x_scales, int8_t* z_codes, float* z_scales,
                                   void* stream) {
  CallRange range_("gdn_gated_rmsnorm_ckpt8");
  if (bad_dtype(dtype) || n_rows < 0 || dim < 1 || !(eps >= 0.0f)) return GDN_ERR_INVALID_ARG;
  if (!norm_dim_ok(dim)) return GDN_ERR_UNSUPPORTED;
  if (n_rows == 0) return GDN_OK;
  if (!ptr_ok(x) || !ptr_ok(z) || !ptr_ok(y) || !w || !ptr_ok(x_codes) || !ptr_ok(z_codes) ||
      !x_scales || !z_scales || !aligned_to(4, w, x_scales, z_scales))
    return GDN_ERR_INVALID_ARG;
  const size_t n = (size_t)n_rows * dim, sb = (size_t)n_rows * sizeof(float);
  const Span in[] = {{z, n * elem(dtype)}, {w, dim * sizeof(float)}};
  const Span out[] = {{y, n * elem(dtype)}, {x_codes, n}, {x_scales, sb}, {z_codes, n},
                      {z_scales, sb}};
  if (clash(in, out)) return GDN_ERR_INVALID_ARG;
  const Span xin[] = {{x, n * elem(dtype)}};
  const Span codes[] = {{x_codes, n}, {x_scales, sb}, {z_codes, n}, {z_scales, sb}};
  if (clash(xin, codes)) return GDN_ERR_INVALID_ARG;
  if (y != x && overlap({y, n * elem(dtype)}, xin[0])) return GDN_ERR_INVALID_ARG;  // in place only
  return from_cuda(launch_rmsnorm_ckpt8(x, z, dtype, w, eps, n_rows, dim, y, x_codes, x_scales,
                                        z_codes, z_scales, as_stream(stream)));
}

size_t gdn_gated_rmsnorm_bwd_workspace_size(int64_t n_rows, int dim) {
  if (n_rows < 0 || !norm_dim_ok(dim)) return 256;
  return round256(256 + (size_t)norm_parts(n_rows, dim) * dim * sizeof(float));
}

gdn_status gdn_gated_rmsnorm_bwd(const void* dy, const void* x, const float* x_scales,
                                 const void* z, const float* z_scales, gdn_dtype dtype,
                                 const float* w, float eps, int64_t n_rows, int dim, void* dx,
                                 void* dz, float* dw, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  CallRange range_("gdn_gated_rmsnorm_bwd");
  return rmsnorm_bwd(dy, x, x_scales, z, z_scales, dtype, w, eps, nullptr, 0, 1, n_rows, dim, dx, dz, dw,
                     workspace, workspace_bytes, stream);
}

gdn_status gdn_gated_rmsnorm_bwd_varlen(const void* dy, const void* x, const float* x_scales,
                                        const void* z, const float* z_scales, gdn_dtype dtype,
                                        const float* w, float eps, const int32_t* cu_seqlens, int N,
                                        int rows_per_token, int64_t n_rows, int dim, void* dx,
                                        void* dz, float* dw, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  CallRange range_("gdn_gated_rmsnorm_bwd_varlen");
  return rmsnorm_bwd(dy, x, x_scales, z, z_scales, dtype, w, eps, cu_seqlens, N, rows_per_token, n_rows,
                     dim, dx, dz, dw, workspace, workspace_bytes, stream);
}

// -------------------------------------------------------------------------------- conv -----

size_t gdn_causal_conv1d_silu_bwd_workspace_size(int B, int64_t T, int C, int K) {
  if (B < 0 || T < 0 || C < 1 || K < 1) return 256;
  return round256(256 + (size_t)conv_parts((int64_t)B * T, C) * C * (K + 1) * sizeof(float));
}

gdn_status gdn_causal_conv1d_silu_bwd(const void* dy, const void* x, const float* x_scales,
                                      int x_group, gdn_dtype dtype, const float* w,
                                      const float* bias, int B, int64_t T, int C, int K,
                                      const int32_t* cu_seqlens, int N, int n_l2norm_ch,
                                      int l2norm_group, float l2_eps, const float* conv_state_in,
                                      const float* dconv_state_out, void* dx, float* dw,
                                      float* dbias, float* dconv_state_in, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  CallRange range_("gdn_causal_conv1d_silu_bwd");
  if (bad_dtype(dtype) || B < 0 || T < 0 || C < 1 || K < 1 || N < 0) return GDN_ERR_INVALID_ARG;
  if (cu_seqlens ? (B != 1 && !(B == 0 && T == 0)) : (N != B)) return GDN_ERR_INVALID_ARG;
  if (n_l2norm_ch < 0 || n_l2norm_ch > C || l2norm_group < 0) return GDN_ERR_INVALID_ARG;
  if (!(l2_eps >= 0.0f)) return GDN_ERR_INVALID_ARG;
  if (K > 8 || C % 8 != 0) return GDN_ERR_UNSUPPORTED;
  if (l2norm_group != 0 && l2norm_group != 32 && l2norm_group != 64 && l2norm_group != 128 &&
      l2norm_group != 256)
    return GDN_ERR_UNSUPPORTED;
  if (l2norm_group == 0 ? n_l2norm_ch != 0 : n_l2norm_ch % l2norm_group != 0)
    return GDN_ERR_INVALID_ARG;
  if (x_scales) {
    if (x_group < 1 || C % x_group != 0) return GDN_ERR_INVALID_ARG;
    if (!norm_dim_ok(x_group)) return GDN_ERR_UNSUPPORTED;
  }
  const int64_t n_tok = (int64_t)B * T;
  if (cu_seqlens && n_tok > 0 && N < 1) return GDN_ERR_INVALID_ARG;
  if (!w || !dw || (bias != nullptr) != (dbias != nullptr)) return GDN_ERR_INVALID_ARG;
  if (n_tok > 0 && (!ptr_ok(dy) || !ptr_ok(x) || !ptr_ok(dx))) return GDN_ERR_INVALID_ARG;
  if (!aligned_to(4, x_scales, cu_seqlens, w, bias, conv_state_in, dconv_state_out, dw, dbias,
                  dconv_state_in))
    return GDN_ERR_INVALID_ARG;
  if (!ws_ok(workspace, workspace_bytes, gdn_causal_conv1d_silu_bwd_workspace_size(B, T, C, K)))
    return GDN_ERR_INVALID_ARG;
  const size_t n = (size_t)n_tok * C, nb = n * elem(dtype);
  const size_t st = (size_t)N * C * (K - 1) * sizeof(float), wb = (size_t)C * K * sizeof(float);
  const size_t cb = (size_t)C * sizeof(float);
  const Span in[] = {{dy, nb},
                     {x, x_scales ? n : nb},
                     {x_scales, x_scales ? n / x_group * sizeof(float) : 0},
                     {w, wb},
                     {bias, cb},
                     {cu_seqlens, (size_t)(N + 1) * 4},
                     {conv_state_in, st},
                     {dconv_state_out, st}};
  const Span out[] = {{dx, nb}, {dw, wb}, {dbias, cb}, {dconv_state_in, st},
                      {workspace, workspace_bytes}};
  if (clash(in, out)) return GDN_ERR_INVALID_ARG;
  ConvBwdArgs a;
  a.dy = dy;
  a.x = x;
  a.xs = x_scales;
  a.xgroup = x_group;
  a.xgroups = x_scales ? C / x_group : 0;
  a.w = w;
  a.bias = bias;
  a.n_tok = n_tok;
  a.T = T;
  a.C = C;
  a.K = K;
  a.N = N;
  a.n_l2 = n_l2norm_ch;
  a.group = l2norm_group;
  a.cu = cu_seqlens;
  a.eps = l2_eps;
  a.cs_in = K > 1 ? conv_state_in : nullptr;
  a.dcs_out = K > 1 ? dconv_state_out : nullptr;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.dcs_in = K > 1 ? dconv_state_in : nullptr;
  a.part = (float*)workspace;
  a.max_parts = conv_parts(n_tok, C);
  return from_cuda(launch_conv_bwd(a, dtype, as_stream(stream)));
}

// -------------------------------------------------------------------------------- rule -----

size_t gdn_chunk_bwd_workspace_size(gdn_dtype dtype, int N, int B, int64_t T, int Hk, int Hv,
                                    int dk, int dv, int chunk) {
  (void)Hk;
  if (N < 0 || B < 0 || T < 0 || Hv < 1 || dk < 1 || dv < 1 || chunk < 1) return 256;
  const int64_t n_tok = (int64_t)B * T;
  if (n_tok == 0) return bwd::HEADER;
  return round256(tensor_cores(dtype, n_tok, Hv, dk, dv, chunk)
                      ? bwd::tc_workspace_bytes(N, n_tok, Hv)
                      : bwd::simt_workspace_bytes(N, n_tok, Hv, dk, dv,
                                                  simt_chunk(n_tok, chunk)));
}

gdn_status gdn_chunk_bwd(const void* q, int64_t q_tok_stride, const void* k, int64_t k_tok_stride,
                         const void* v, int64_t v_tok_stride, const float* g, const float* beta,
                         const void* dout, gdn_dtype dtype, float scale,
                         const float* initial_state, const float* dfinal_state,
                         const int32_t* cu_seqlens, int N, int B, int64_t T, int Hk, int Hv, int dk,
                         int dv, int chunk, void* dq, void* dk_out, void* dv_out, void* dg,
                         void* dbeta, float* dinitial_state, void* workspace,
                         size_t workspace_bytes, void* stream) {
  CallRange range_("gdn_chunk_bwd");
  if (bad_dtype(dtype) || N < 0 || B < 0 || T < 0 || Hk < 1 || Hv < 1 || dk < 1 || dv < 1)
    return GDN_ERR_INVALID_ARG;
  if (Hv % Hk != 0) return GDN_ERR_INVALID_ARG;
  if (cu_seqlens ? (B != 1) : (N != B)) return GDN_ERR_INVALID_ARG;
  if (!(scale == scale)) return GDN_ERR_INVALID_ARG;
  if (dk % 16 != 0 || dv % 16 != 0 || dk > 128 || dv > 128) return GDN_ERR_UNSUPPORTED;
  if (chunk != 16 && chunk != 32 && chunk != 64) return GDN_ERR_UNSUPPORTED;
  if (q_tok_stride < (int64_t)Hk * dk || k_tok_stride < (int64_t)Hk * dk ||
      v_tok_stride < (int64_t)Hv * dv || q_tok_stride % 8 || k_tok_stride % 8 || v_tok_stride % 8)
    return GDN_ERR_INVALID_ARG;
  if (!ws_ok(workspace, workspace_bytes,
             gdn_chunk_bwd_workspace_size(dtype, N, B, T, Hk, Hv, dk, dv, chunk)))
    return GDN_ERR_INVALID_ARG;
  if (N == 0) return GDN_OK;
  const int64_t n_tok = (int64_t)B * T;
  if (n_tok > 0 && (!ptr_ok(q) || !ptr_ok(k) || !ptr_ok(v) || !ptr_ok(g) || !ptr_ok(beta) ||
                    !ptr_ok(dout) || !ptr_ok(dq) || !ptr_ok(dk_out) || !ptr_ok(dv_out) || !dg ||
                    !dbeta))
    return GDN_ERR_INVALID_ARG;
  if (!aligned_to(16, initial_state, dfinal_state, dinitial_state) || !aligned4(cu_seqlens) ||
      !aligned_to(elem(dtype), dg, dbeta))
    return GDN_ERR_INVALID_ARG;
  const size_t e = elem(dtype), st = (size_t)N * Hv * dv * dk * sizeof(float);
  const size_t hk = (size_t)Hk * dk, hv = (size_t)Hv * dv, nt = (size_t)n_tok;
  auto rows = [&](int64_t stride, size_t width) {
    return nt ? ((nt - 1) * (size_t)stride + width) * e : 0;
  };
  const Span in[] = {{q, rows(q_tok_stride, hk)}, {k, rows(k_tok_stride, hk)},
                     {v, rows(v_tok_stride, hv)}, {dout, nt * hv * e},
                     {g, nt * Hv * 4},            {beta, nt * Hv * 4},
                     {initial_state, st},         {dfinal_state, st},
                     {cu_seqlens, (size_t)(N + 1) * 4}};
  const Span out[] = {{dq, nt * hk * e}, {dk_out, nt * hk * e}, {dv_out, nt * hv * e},
                      {dg, nt * Hv * e}, {dbeta, nt * Hv * e},  {dinitial_state, st},
                      {workspace, workspace_bytes}};
  if (clash(in, out)) return GDN_ERR_INVALID_ARG;
  bwd::Args a;
  a.q = q; a.k = k; a.v = v; a.dout = dout;
  a.ts = TokStrides{q_tok_stride, k_tok_stride, v_tok_stride};
  a.g = g; a.beta = beta; a.S0 = initial_state; a.dST = dfinal_state;
  a.cu = cu_seqlens;
  a.dt = dtype;
  a.scale = scale;
  a.N = N; a.B = B; a.T = T; a.Hk = Hk; a.Hv = Hv; a.dk = dk; a.dv = dv; a.C = chunk;
  a.dq = dq; a.dk_ = dk_out; a.dv_ = dv_out; a.dg = dg; a.dbeta = dbeta;
  a.dS0 = dinitial_state;
  a.ws = workspace;
  a.ws_bytes = workspace_bytes;
  a.status = reinterpret_cast<int*>(workspace);
  const cudaStream_t s = as_stream(stream);
  if (tensor_cores(dtype, n_tok, Hv, dk, dv, chunk)) return from_cuda(bwd::launch_tc(a, s));
  if (cudaMemsetAsync(workspace, 0, sizeof(int), s) != cudaSuccess) return GDN_ERR_CUDA;  // status word
  a.C = simt_chunk(n_tok, chunk);
  return from_cuda(bwd::launch_simt(a, s));
}

}  // extern "C"
