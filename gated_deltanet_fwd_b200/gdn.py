"""Thin ctypes binding over libgdn.so (include/gdn.h): argument marshalling only.

Every function takes torch CUDA tensors, passes their device pointers and the current CUDA stream
to the C entry point of the same name, and raises ``GdnError`` on a non-OK status.  All arithmetic
happens in the library's kernels; there is no fallback of any kind -- if ``libgdn.so`` is missing
the first call raises.  torch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn.so")

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_TIMEOUT, \
    GDN_ERR_DEVICE_ARG = range(6)
GDN_BF16, GDN_F32 = 0, 1

# name -> (restype, argtypes); mirrors include/gdn.h
_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float
_SZ = ctypes.c_size_t
SIGNATURES = {
    "gdn_status_string": (ctypes.c_char_p, [_I]),
    "gdn_gates": (_I, [_P, _P, _I, _P, _P, _I64, _I, _P, _P, _P]),
    "gdn_causal_conv1d_silu": (_I, [_P, _I, _P, _P, _I, _I64, _I, _I, _P, _I, _I, _I, _F, _P, _P,
                                    _P, _P]),
    "gdn_chunk_fwd": (_I, [_P, _P, _P, _P, _P, _I, _F, _P, _P, _I, _I, _I64, _I, _I, _I, _I, _I,
                           _P, _P, _P, _SZ, _P]),
    "gdn_chunk_fwd_strided": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _P, _I, _F, _P, _P, _I, _I,
                                   _I64, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "gdn_chunk_fwd_gated_norm": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _F,
                                      _I, _F, _P, _P, _I, _I, _I64, _I, _I, _I, _I, _I, _P, _P,
                                      _P, _SZ, _P]),
    "gdn_chunk_fwd_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _F, _P, _P, _I, _I, _I64, _I, _I, _I,
                                   _I, _I, _P, _P, _P]),
    "gdn_chunk_fwd_workspace_size": (_SZ, [_I, _I, _I64, _I, _I, _I, _I, _I]),
    "gdn_workspace_status": (_I, [_P, _P, ctypes.POINTER(_I)]),
    "gdn_recurrent_step": (_I, [_P, _P, _P, _P, _P, _I, _F, _P, _I, _I, _I, _I, _I, _P, _P]),
    "gdn_gated_rmsnorm": (_I, [_P, _P, _I, _P, _F, _I64, _I, _P, _P]),
    "gdn_chunk_bwd_workspace_size": (_SZ, [_I, _I, _I, _I64, _I, _I, _I, _I, _I]),
    "gdn_chunk_bwd": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _I, _F, _P, _P, _P, _I, _I,
                           _I64, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "gdn_gates_bwd_workspace_size": (_SZ, [_I64, _I]),
    "gdn_gates_bwd": (_I, [_P, _P, _I, _P, _P, _P, _P, _I64, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "gdn_gates_bwd_varlen": (_I, [_P, _P, _I, _P, _P, _P, _P, _P, _I, _I64, _I, _P, _P, _P, _P, _P,
                                  _SZ, _P]),
    "gdn_gated_rmsnorm_bwd_workspace_size": (_SZ, [_I64, _I]),
    "gdn_gated_rmsnorm_bwd": (_I, [_P, _P, _P, _P, _P, _I, _P, _F, _I64, _I, _P, _P, _P, _P, _SZ,
                                   _P]),
    "gdn_gated_rmsnorm_bwd_varlen": (_I, [_P, _P, _P, _P, _P, _I, _P, _F, _P, _I, _I, _I64, _I, _P,
                                          _P, _P, _P, _SZ, _P]),
    "gdn_causal_conv1d_silu_bwd_workspace_size": (_SZ, [_I, _I64, _I, _I]),
    "gdn_causal_conv1d_silu_bwd": (_I, [_P, _P, _P, _I, _I, _P, _P, _I, _I64, _I, _I, _P, _I, _I,
                                        _I, _F, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "gdn_act_pack8": (_I, [_P, _I, _I64, _I, _I, _P, _P, _P]),
    "gdn_act_unpack8": (_I, [_P, _P, _I, _I64, _I, _I, _P, _P]),
    "gdn_gated_rmsnorm_ckpt8": (_I, [_P, _P, _I, _P, _F, _I64, _I, _P, _P, _P, _P, _P, _P]),
    "gdn_decode_layer_step": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _P, _P, _P, _P, _P, _F, _F, _F,
                                   _P, _I, _I, _I, _I, _I, _P, _P]),
}

_lib = None


class GdnError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)}")


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgdn.so (built by ``python -m gated_deltanet_fwd_b200.build``); raises if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"libgdn.so not found at {path}; build it with "
                               "`python -m gated_deltanet_fwd_b200.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().gdn_status_string(int(status)).decode()


def _check(fn, status):
    if status != GDN_OK:
        raise GdnError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _dt(t):
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"unsupported activation dtype {t.dtype}")


def _cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def _tok_stride(t):
    """Token stride of a [B, T, H, d] view whose heads are packed inside each token, else None."""
    B, T, H, d = t.shape
    if not t.is_cuda or t.stride(3) != 1 or (H > 1 and t.stride(2) != d):
        return None
    if B * T < 2:  # no distance between tokens
        return H * d
    if T == 1:
        return t.stride(0)
    if B > 1 and t.stride(0) != T * t.stride(1):
        return None
    return t.stride(1)


# ------------------------------------------------------------------------------ calls ------

def gdn_gates(a, b, A_log, dt_bias, g=None, beta=None):
    """beta = sigmoid(b), g = -exp(A_log) * softplus(a + dt_bias).  a, b: [..., Hv]."""
    _cuda(a, b, A_log, dt_bias, g, beta)
    Hv = A_log.numel()
    g = torch.empty(a.shape, dtype=torch.float32, device=a.device) if g is None else g
    beta = torch.empty(a.shape, dtype=torch.float32, device=a.device) if beta is None else beta
    _check("gdn_gates", load().gdn_gates(_ptr(a), _ptr(b), _dt(a), _ptr(A_log), _ptr(dt_bias),
                                         a.numel() // Hv, Hv, _ptr(g), _ptr(beta), _stream(a)))
    return g, beta


def gdn_causal_conv1d_silu(x, w, bias=None, cu_seqlens=None, n_l2norm_ch=0, l2norm_group=0,
                           l2_eps=1e-6, conv_state_in=None, conv_state_out=None, y=None):
    """Depthwise causal conv + SiLU (+ per-group L2 norm of the first n_l2norm_ch channels).

    x: [B, T, C]; w: [C, K] fp32; returns y [B, T, C] (x's dtype).
    """
    _cuda(x, w, bias, cu_seqlens, conv_state_in, conv_state_out, y)
    B, T, C = x.shape
    K = w.shape[1]
    N = cu_seqlens.numel() - 1 if cu_seqlens is not None else B
    y = torch.empty_like(x) if y is None else y
    _check("gdn_causal_conv1d_silu", load().gdn_causal_conv1d_silu(
        _ptr(x), _dt(x), _ptr(w), _ptr(bias), B, T, C, K, _ptr(cu_seqlens), N, n_l2norm_ch,
        l2norm_group, float(l2_eps), _ptr(conv_state_in), _ptr(conv_state_out), _ptr(y),
        _stream(x)))
    return y


def workspace_size(N, B, T, Hk, Hv, dk, dv, chunk):
    return int(load().gdn_chunk_fwd_workspace_size(N, B, T, Hk, Hv, dk, dv, chunk))


def workspace_status(workspace) -> int:
    """Blocks on the current stream, then returns the device status word of `workspace`."""
    out = ctypes.c_int(-1)
    _check("gdn_workspace_status", load().gdn_workspace_status(
        _ptr(workspace), _stream(workspace), ctypes.byref(out)))
    return out.value


def gdn_chunk_fwd(q, k, v, g, beta, scale=None, initial_state=None, cu_seqlens=None, chunk=64,
                  out=None, final_state=None, output_final_state=True, workspace=None):
    """Chunked prefill: (q, k, v, g, beta, initial_state, cu_seqlens) -> (out, final_state).

    q, k: [B, T, Hk, dk]; v: [B, T, Hv, dv]; g, beta: [B, T, Hv] fp32; states [N, Hv, dv, dk].
    q, k, v may be views whose tokens are not packed back to back (e.g. slices of the conv's
    [q | k | v] output); those go through gdn_chunk_fwd_strided.
    """
    _cuda(g, beta, initial_state, cu_seqlens, out, final_state, workspace)
    qs, ks, vs = _tok_stride(q), _tok_stride(k), _tok_stride(v)
    if qs is None or ks is None or vs is None:
        raise ValueError("q, k, v must be CUDA [B, T, H, d] tensors with each token's heads packed")
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    N = cu_seqlens.numel() - 1 if cu_seqlens is not None else B
    scale = dk ** -0.5 if scale is None else scale
    out = torch.empty(v.shape, dtype=v.dtype, device=v.device) if out is None else out
    if final_state is None and output_final_state:
        final_state = torch.empty((N, Hv, dv, dk), dtype=torch.float32, device=q.device)
    ws_bytes = workspace_size(N, B, T, Hk, Hv, dk, dv, chunk)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    ws_b = workspace.numel() * workspace.element_size()
    if (qs, ks, vs) == (Hk * dk, Hk * dk, Hv * dv):
        _check("gdn_chunk_fwd", load().gdn_chunk_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q), float(scale),
            _ptr(initial_state), _ptr(cu_seqlens), N, B, T, Hk, Hv, dk, dv, chunk, _ptr(out),
            _ptr(final_state), _ptr(workspace), ws_b, _stream(q)))
    else:
        _check("gdn_chunk_fwd_strided", load().gdn_chunk_fwd_strided(
            _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(g), _ptr(beta), _dt(q), float(scale),
            _ptr(initial_state), _ptr(cu_seqlens), N, B, T, Hk, Hv, dk, dv, chunk, _ptr(out),
            _ptr(final_state), _ptr(workspace), ws_b, _stream(q)))
    return out, final_state


def gdn_chunk_fwd_gated_norm(q, k, v, a, b, A_log, dt_bias, z, norm_w, norm_eps=1e-6, scale=None,
                             initial_state=None, cu_seqlens=None, y=None, final_state=None,
                             output_final_state=True, workspace=None):
    """Layer core after the conv in one call: gates(a, b) -> chunked delta rule -> gated RMSNorm
    with z.  q, k: [B, T, Hk, 128]; v: [B, T, Hv, 128] (may be strided views of the conv output);
    a, b: [B, T, Hv] bf16; z: [B, T, Hv, 128] bf16.  Returns (y, final_state)."""
    _cuda(a, b, A_log, dt_bias, z, norm_w, initial_state, cu_seqlens, y, final_state, workspace)
    if len({t.dtype for t in (q, k, v, a, b, z)}) != 1:
        raise TypeError("q, k, v, a, b and z must share one activation dtype")
    qs, ks, vs = _tok_stride(q), _tok_stride(k), _tok_stride(v)
    if qs is None or ks is None or vs is None:
        raise ValueError("q, k, v must be CUDA [B, T, H, d] tensors with each token's heads packed")
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    N = cu_seqlens.numel() - 1 if cu_seqlens is not None else B
    scale = dk ** -0.5 if scale is None else scale
    y = torch.empty(v.shape, dtype=v.dtype, device=v.device) if y is None else y
    if final_state is None and output_final_state:
        final_state = torch.empty((N, Hv, dv, dk), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(workspace_size(N, B, T, Hk, Hv, dk, dv, 64), dtype=torch.uint8,
                                device=q.device)
    _check("gdn_chunk_fwd_gated_norm", load().gdn_chunk_fwd_gated_norm(
        _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias),
        _ptr(z), _ptr(norm_w), float(norm_eps), _dt(q), float(scale), _ptr(initial_state),
        _ptr(cu_seqlens), N, B, T, Hk, Hv, dk, dv, 64, _ptr(y), _ptr(final_state),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(q)))
    return y, final_state


def gdn_recurrent_step(q, k, v, g, beta, state, scale=None, out=None):
    """One decode token per sequence; `state` [N, Hv, dv, dk] fp32 is updated in place.

    q, k: [N, Hk, dk]; v: [N, Hv, dv]; g, beta: [N, Hv] fp32.  Returns out [N, Hv, dv].
    """
    _cuda(q, k, v, g, beta, state, out)
    N, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    scale = dk ** -0.5 if scale is None else scale
    out = torch.empty_like(v) if out is None else out
    _check("gdn_recurrent_step", load().gdn_recurrent_step(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q), float(scale), _ptr(state), N, Hk,
        Hv, dk, dv, _ptr(out), _stream(q)))
    return out


def gdn_decode_layer_step(mix, a, b, z, conv_w, conv_state_in, conv_state_out, A_log, dt_bias,
                          norm_w, state, Hk, conv_bias=None, l2_eps=1e-6, norm_eps=1e-6,
                          scale=None, y=None):
    """One decode token of the layer core: conv (history in conv_state_in, advanced into
    conv_state_out) + SiLU + q/k L2 norm, gates, recurrent step on `state` (in place), gated
    RMSNorm with z.  mix: [N, C]; a, b: [N, Hv]; z: [N, Hv, dv]; returns y [N, Hv, dv]."""
    _cuda(mix, a, b, z, conv_w, conv_bias, conv_state_in, conv_state_out, A_log, dt_bias, norm_w,
          state, y)
    N, Hv, dv = z.shape
    dk = state.shape[3]
    K = conv_w.shape[1]
    scale = dk ** -0.5 if scale is None else scale
    y = torch.empty_like(z) if y is None else y
    _check("gdn_decode_layer_step", load().gdn_decode_layer_step(
        _ptr(mix), _ptr(a), _ptr(b), _ptr(z), _dt(mix), _ptr(conv_w), _ptr(conv_bias), K,
        _ptr(conv_state_in), _ptr(conv_state_out), _ptr(A_log), _ptr(dt_bias), _ptr(norm_w),
        float(l2_eps), float(norm_eps), float(scale), _ptr(state), N, Hk, Hv, dk, dv, _ptr(y),
        _stream(mix)))
    return y


def gdn_gated_rmsnorm(x, z, w, eps=1e-6, y=None):
    """y = x * rsqrt(mean(x^2) + eps) * (1 + w) * silu(z) over the last dim."""
    _cuda(x, z, w, y)
    dim = x.shape[-1]
    y = torch.empty_like(x) if y is None else y
    _check("gdn_gated_rmsnorm", load().gdn_gated_rmsnorm(
        _ptr(x), _ptr(z), _dt(x), _ptr(w), float(eps), x.numel() // dim, dim, _ptr(y),
        _stream(x)))
    return y


# ---------------------------------------------------------------- training: backward passes ----

def _ws(need, given, device):
    """The workspace to pass and its bytes: the caller's, or a new one of `need` bytes."""
    w = torch.empty(need, dtype=torch.uint8, device=device) if given is None else given
    return w, w.numel() * w.element_size()


def _kept(x):
    """An activation, or its 8-bit checkpoint (codes, scales): (tensor, scales or None)."""
    if isinstance(x, (tuple, list)):
        codes, scales = x
        if codes.dtype != torch.int8 or scales.dtype != torch.float32:
            raise TypeError("a checkpoint is (int8 codes, fp32 scales)")
        if not scales.numel() or codes.numel() % scales.numel():
            if codes.numel() or scales.numel():
                raise ValueError("codes and scales of a checkpoint do not match")
        return codes, scales
    return x, None


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# the same without building a Stream object (2 us of a small call), where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


def _run(name, device, *args):
    """Calls the entry point on `device` and on torch's current stream there (the last argument)."""
    i = device.index
    if i == torch.cuda.current_device():
        _check(name, getattr(_lib, name)(*args, _raw_stream(i)))
    else:
        with torch.cuda.device(device):
            _check(name, getattr(_lib, name)(*args, _raw_stream(i)))


def _adr(t):
    return None if t is None else t.data_ptr()


def _all_cuda(*ts):
    """Contiguous CUDA tensors of one device (None is skipped)."""
    load()
    dev = -1
    for t in ts:
        if t is not None:
            d = t.get_device()  # -1 on the CPU
            if d < 0 or not t.is_contiguous():
                raise ValueError("tensors must be contiguous CUDA tensors")
            if d != dev:
                if dev >= 0:
                    raise ValueError("tensors must be on one device")
                dev = d


def _same(dtype, *ts):
    for t in ts:
        if t is not None and t.dtype != dtype:
            raise TypeError(f"expected tensors of {dtype}")


def _shape(shape, *ts):
    for t in ts:
        if t is not None and t.shape != shape:
            raise ValueError(f"expected tensors of shape {tuple(shape)}")


def _width(t):
    """The last dimension of a tensor, which must not be empty."""
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError("the last dimension must have at least one element")
    return t.shape[-1]


def chunk_bwd_workspace_size(dtype, N, B, T, Hk, Hv, dk, dv, chunk=64):
    """Bytes of workspace for gdn_chunk_bwd with activations of the torch dtype."""
    dt = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}[dtype]
    return int(load().gdn_chunk_bwd_workspace_size(dt, N, B, T, Hk, Hv, dk, dv, chunk))


def gdn_chunk_bwd(q, k, v, g, beta, dout, scale=None, initial_state=None, cu_seqlens=None,
                  dfinal_state=None, chunk=64, dq=None, dk=None, dv=None, dg=None, dbeta=None,
                  dinitial_state=None, output_dinitial_state=None, workspace=None):
    """Gradients of gdn_chunk_fwd: (dq, dk, dv, dg, dbeta, dinitial_state).

    q, k, v (possibly strided views), g, beta, scale, initial_state, cu_seqlens as given to the forward;
    dout [B, T, Hv, dv]; dfinal_state [N, Hv, dv, dk] fp32 or None (zero).  dg and dbeta are of
    the activations' dtype.  dinitial_state is computed when initial_state is given, unless
    output_dinitial_state says otherwise; else None.  Tokens outside every sequence of cu_seqlens are
    not written: tensors that are given keep what they held there, dg and dbeta made here hold zeros, and
    dq, dk and dv made here anything (gdn_causal_conv1d_silu_bwd with the same cu_seqlens does not
    read those rows).
    """
    _all_cuda(g, beta, dout, initial_state, cu_seqlens, dfinal_state, dq, dk, dv, dg, dbeta,
              dinitial_state, workspace)
    if any(t.device != g.device for t in (q, k, v)):
        raise ValueError("tensors must be on one device")
    qs, ks, vs = _tok_stride(q), _tok_stride(k), _tok_stride(v)
    if qs is None or ks is None or vs is None:
        raise ValueError("q, k, v must be CUDA [B, T, H, d] tensors with each token's heads packed")
    B, T, Hk, d_k = q.shape
    Hv, d_v = v.shape[2], v.shape[3]
    N = cu_seqlens.numel() - 1 if cu_seqlens is not None else B
    _same(q.dtype, k, v, dout, dq, dk, dv, dg, dbeta)
    _same(torch.float32, g, beta, initial_state, dfinal_state, dinitial_state)
    _same(torch.int32, cu_seqlens)
    _shape((B, T, Hk, d_k), k, dq, dk)
    _shape((B, T, Hv, d_v), v, dout, dv)
    _shape((B, T, Hv), g, beta, dg, dbeta)
    _shape((N, Hv, d_v, d_k), initial_state, dfinal_state, dinitial_state)
    new = lambda t, shape: dout.new_empty(shape) if t is None else t  # noqa: E731
    dq, dk, dv = new(dq, (B, T, Hk, d_k)), new(dk, (B, T, Hk, d_k)), new(dv, (B, T, Hv, d_v))
    if cu_seqlens is not None and (dg is None or dbeta is None):  # zeros, from one allocation
        zeros = dout.new_zeros((2, B, T, Hv)).unbind()
        dg, dbeta = (z if t is None else t for t, z in zip((dg, dbeta), zeros))
    dg, dbeta = new(dg, (B, T, Hv)), new(dbeta, (B, T, Hv))
    if output_dinitial_state is None:
        output_dinitial_state = initial_state is not None
    if dinitial_state is None and output_dinitial_state:
        dinitial_state = torch.empty((N, Hv, d_v, d_k), dtype=torch.float32, device=q.device)
    lib, dt = _lib, _dt(q)
    ws, ws_b = _ws(lib.gdn_chunk_bwd_workspace_size(dt, N, B, T, Hk, Hv, d_k, d_v, chunk),
                   workspace, q.device)
    _run("gdn_chunk_bwd", q.device,
        _adr(q), qs, _adr(k), ks, _adr(v), vs, _adr(g), _adr(beta), _adr(dout), dt,
        float(d_k ** -0.5 if scale is None else scale), _adr(initial_state), _adr(dfinal_state),
        _adr(cu_seqlens), N, B, T, Hk, Hv, d_k, d_v, chunk, _adr(dq), _adr(dk), _adr(dv), _adr(dg),
        _adr(dbeta), _adr(dinitial_state), _adr(ws), ws_b)
    return dq, dk, dv, dg, dbeta, dinitial_state


def gdn_gates_bwd(a, b, A_log, dt_bias, dg, dbeta, da=None, db=None, dA_log=None, ddt_bias=None,
                  workspace=None, cu_seqlens=None):
    """Gradients of gdn_gates: (da, db, dA_log, ddt_bias).  a, b, dg, dbeta: [..., Hv] of one dtype.

    With cu_seqlens, as after gdn_chunk_bwd with the same, tokens outside every sequence take no part:
    da and db made here are zero there, tensors that are given keep what they held.
    """
    _all_cuda(a, b, A_log, dt_bias, dg, dbeta, da, db, dA_log, ddt_bias, workspace, cu_seqlens)
    Hv = A_log.numel()
    _same(a.dtype, b, dg, dbeta, da, db)
    _same(torch.float32, A_log, dt_bias, dA_log, ddt_bias)
    _shape(a.shape, b, dg, dbeta, da, db)
    _shape((Hv,), A_log, dt_bias, dA_log, ddt_bias)
    if Hv < 1 or a.shape[-1] != Hv:
        raise ValueError("the last dimension of a must be the number of heads")
    new, N = torch.empty_like, 0
    if cu_seqlens is not None:
        _same(torch.int32, cu_seqlens)
        new, N = torch.zeros_like, cu_seqlens.numel() - 1
    da = new(a) if da is None else da
    db = new(b) if db is None else db
    dA_log = torch.empty_like(A_log) if dA_log is None else dA_log
    ddt_bias = torch.empty_like(dt_bias) if ddt_bias is None else ddt_bias
    n_tok, lib = a.numel() // Hv, _lib
    ws, ws_b = _ws(lib.gdn_gates_bwd_workspace_size(n_tok, Hv), workspace, a.device)
    _run("gdn_gates_bwd_varlen", a.device,
        _adr(a), _adr(b), _dt(a), _adr(A_log), _adr(dt_bias), _adr(dg), _adr(dbeta),
        _adr(cu_seqlens), N, n_tok, Hv, _adr(da), _adr(db), _adr(dA_log), _adr(ddt_bias), _adr(ws), ws_b)
    return da, db, dA_log, ddt_bias


def gdn_gated_rmsnorm_bwd(dy, x, z, w, eps=1e-6, dx=None, dz=None, dw=None, workspace=None,
                          cu_seqlens=None):
    """Gradients of gdn_gated_rmsnorm: (dx, dz, dw).

    x and z are the forward's inputs, or their 8-bit checkpoints as (codes, scales) pairs.  With
    cu_seqlens dy is [.., tokens, heads, dim] and tokens outside every sequence take no part: their rows of
    dx and dz are not written (anything where they are made here).
    """
    (x, xs), (z, zs) = _kept(x), _kept(z)
    if (xs is None) != (zs is None):
        raise ValueError("x and z must both be activations or both be checkpoints")
    _all_cuda(dy, x, xs, z, zs, w, dx, dz, dw, workspace, cu_seqlens)
    _same(torch.int32, cu_seqlens)
    N, per = 0, 1
    if cu_seqlens is not None:
        if dy.dim() < 3:
            raise ValueError("with cu_seqlens dy must be [.., tokens, heads, dim]")
        N, per = cu_seqlens.numel() - 1, dy.shape[-2]
    dim = _width(dy)
    n_rows = dy.numel() // dim
    _shape(dy.shape, x, z, dx, dz)
    _shape((dim,), w, dw)
    _same(dy.dtype, dx, dz)
    _same(torch.int8 if xs is not None else dy.dtype, x, z)
    _same(torch.float32, w, dw)
    if xs is not None and (xs.numel() != n_rows or zs.numel() != n_rows):
        raise ValueError("the norm's checkpoints have one scale per row")
    dx = torch.empty_like(dy) if dx is None else dx
    dz = torch.empty_like(dy) if dz is None else dz
    dw = torch.empty_like(w) if dw is None else dw
    lib = _lib
    ws, ws_b = _ws(lib.gdn_gated_rmsnorm_bwd_workspace_size(n_rows, dim), workspace, dy.device)
    _run("gdn_gated_rmsnorm_bwd_varlen", dy.device,
        _adr(dy), _adr(x), _adr(xs), _adr(z), _adr(zs), _dt(dy), _adr(w), float(eps),
        _adr(cu_seqlens), N, per, n_rows, dim,
        _adr(dx), _adr(dz), _adr(dw), _adr(ws), ws_b)
    return dx, dz, dw


def gdn_causal_conv1d_silu_bwd(dy, x, w, bias=None, cu_seqlens=None, n_l2norm_ch=0, l2norm_group=0,
                               l2_eps=1e-6, conv_state_in=None, dconv_state_out=None, dx=None,
                               dw=None, dbias=None, dconv_state_in=None, workspace=None):
    """Gradients of gdn_causal_conv1d_silu: (dx, dw, dbias, dconv_state_in).

    x [B, T, C] is the forward's input, or its 8-bit checkpoint as a (codes, scales) pair.  dbias is
    None without bias; dconv_state_in [N, C, K-1] is computed when conv_state_in is given.  Rows of dx of
    tokens outside every sequence of cu_seqlens are not written (anything where dx is made here).
    """
    x, xs = _kept(x)
    _all_cuda(dy, x, xs, w, bias, cu_seqlens, conv_state_in, dconv_state_out, dx, dw, dbias,
              dconv_state_in, workspace)
    B, T, C = dy.shape
    K = w.shape[1]
    N = cu_seqlens.numel() - 1 if cu_seqlens is not None else B
    _shape((B, T, C), x, dx)
    _shape((C, K), w, dw)
    _shape((C,), bias, dbias)
    _shape((N, C, K - 1), conv_state_in, dconv_state_out, dconv_state_in)
    _same(dy.dtype, dx)
    _same(torch.int8 if xs is not None else dy.dtype, x)
    _same(torch.float32, w, bias, conv_state_in, dconv_state_out, dw, dbias, dconv_state_in)
    _same(torch.int32, cu_seqlens)
    group = 0
    if xs is not None:
        if xs.shape[:-1] != dy.shape[:-1] or C % _width(xs):
            raise ValueError("scales must be [B, T, C / group]")
        group = C // xs.shape[-1]
    dx = torch.empty_like(dy) if dx is None else dx
    dw = torch.empty_like(w) if dw is None else dw
    dbias = torch.empty_like(bias) if dbias is None and bias is not None else dbias
    if dconv_state_in is None and conv_state_in is not None:
        dconv_state_in = torch.empty_like(conv_state_in)
    lib = _lib
    ws, ws_b = _ws(lib.gdn_causal_conv1d_silu_bwd_workspace_size(B, T, C, K), workspace, dy.device)
    _run("gdn_causal_conv1d_silu_bwd", dy.device,
        _adr(dy), _adr(x), _adr(xs), group, _dt(dy), _adr(w), _adr(bias), B, T, C, K,
        _adr(cu_seqlens), N, n_l2norm_ch, l2norm_group, float(l2_eps), _adr(conv_state_in),
        _adr(dconv_state_out), _adr(dx), _adr(dw), _adr(dbias), _adr(dconv_state_in), _adr(ws),
        ws_b)
    return dx, dw, dbias, dconv_state_in


# ------------------------------------------------------- training: 8-bit activation checkpoints ----

def gdn_act_pack8(x, group=128, codes=None, scales=None):
    """x [..., dim] -> (codes int8 of x's shape, scales fp32 [..., dim / group])."""
    _all_cuda(x, codes, scales)
    dim = _width(x)
    if group < 1 or dim % group:
        raise ValueError("group must divide the last dimension")
    codes = torch.empty(x.shape, dtype=torch.int8, device=x.device) if codes is None else codes
    if scales is None:
        scales = torch.empty((*x.shape[:-1], dim // group), dtype=torch.float32, device=x.device)
    _shape(x.shape, codes)
    _shape((*x.shape[:-1], dim // group), scales)
    _same(torch.int8, codes)
    _same(torch.float32, scales)
    _run("gdn_act_pack8", x.device, _adr(x), _dt(x), x.numel() // dim, dim, group, _adr(codes),
         _adr(scales))
    return codes, scales


def gdn_act_unpack8(codes, scales, dtype=torch.bfloat16, x=None):
    """The values that (codes, scales) of gdn_act_pack8 stand for, as a tensor of `dtype`."""
    _all_cuda(codes, scales, x)
    _same(torch.int8, codes)
    _same(torch.float32, scales)
    dim = _width(codes)
    if codes.shape[:-1] != scales.shape[:-1] or dim % _width(scales):
        raise ValueError("scales must be [..., dim / group]")
    x = torch.empty(codes.shape, dtype=dtype, device=codes.device) if x is None else x
    _shape(codes.shape, x)
    _run("gdn_act_unpack8", codes.device,
        _adr(codes), _adr(scales), _dt(x), codes.numel() // dim, dim, dim // scales.shape[-1],
        _adr(x))
    return x


def gdn_gated_rmsnorm_ckpt8(x, z, w, eps=1e-6, y=None):
    """gdn_gated_rmsnorm that keeps 8-bit checkpoints: (y, (x codes, scales), (z codes, scales)).

    The pairs go to gdn_gated_rmsnorm_bwd; y may be x (in place).
    """
    _all_cuda(x, z, w, y)
    dim = _width(x)
    y = torch.empty_like(x) if y is None else y
    _shape(x.shape, z, y)
    _shape((dim,), w)
    _same(x.dtype, z, y)
    _same(torch.float32, w)
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device=x.device)  # noqa: E731
    xc, zc = new(x.shape, torch.int8), new(x.shape, torch.int8)
    xs, zs = new((*x.shape[:-1], 1), torch.float32), new((*x.shape[:-1], 1), torch.float32)
    _run("gdn_gated_rmsnorm_ckpt8", x.device,
        _adr(x), _adr(z), _dt(x), _adr(w), float(eps), x.numel() // dim, dim, _adr(y), _adr(xc),
        _adr(xs), _adr(zc), _adr(zs))
    return y, (xc, xs), (zc, zs)
