"""Calls before and after the device's context is replaced, in a child process that uses the C ABI and the driver
API alone: what a kernel needs to be told (its shared memory) belongs to the context, so nothing of it may be
remembered from the first call.  The same would show on a second device."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import ctypes
import sys
import numpy as np

cuda, lib = ctypes.CDLL("libcuda.so.1"), ctypes.CDLL(sys.argv[1])
for n in ("gdn_chunk_fwd_workspace_size", "gdn_chunk_bwd_workspace_size"):
    getattr(lib, n).restype = ctypes.c_size_t
V, I64, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float


def ok(r):
    assert r == 0, r


def run():
    """Every call with dynamic shared memory once; the outputs."""
    ctx = V()
    ok(cuda.cuDevicePrimaryCtxRetain(ctypes.byref(ctx), dev))
    ok(cuda.cuCtxSetCurrent(ctx))
    rng, at = np.random.default_rng(1), {}

    def put(name, a):
        p = ctypes.c_uint64()
        ok(cuda.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(a.nbytes)))
        ok(cuda.cuMemcpyHtoD_v2(p, a.ctypes.data_as(V), ctypes.c_size_t(a.nbytes)))
        at[name] = p.value
        return V(p.value)

    def bf(*s):  # about normal / 11: unit rows of 128
        return ((rng.standard_normal(s).astype(np.float32) * 0.088).view(np.uint32) >> 16).astype(np.uint16)

    T, H, d = 4096, 1, 128
    q, k, v, do = (put(n, bf(T, H, d)) for n in ("q", "k", "v", "do"))
    g = put("g", -rng.random((T, H), np.float32))
    b = put("b", rng.random((T, H), np.float32))
    out = {n: np.zeros(s, t) for n, s, t in (("o", (T, H, d), np.uint16), ("o2", (256, H, d), np.uint16),
           ("S", (H, d, d), np.float32), ("dq", (T, H, d), np.uint16), ("dk", (T, H, d), np.uint16),
           ("dv", (T, H, d), np.uint16), ("dg", (T, H), np.uint16), ("db", (T, H), np.uint16),
           ("y", (T, H * d), np.uint16), ("dq3", (T, H, d), np.uint16))}
    for n, a in out.items():
        put(n, a)
    p = lambda n: V(at[n])
    nf = lib.gdn_chunk_fwd_workspace_size(1, 1, I64(T), H, H, d, d, 64)
    nb = max(lib.gdn_chunk_bwd_workspace_size(0, 1, 1, I64(T), H, H, d, d, c) for c in (64, 32))
    ws = put("ws", np.zeros(max(nf, nb), np.uint8))
    ok(lib.gdn_chunk_fwd(q, k, v, g, b, 0, F(0.1), None, None, 1, 1, I64(T), H, H, d, d, 64, p("o"), p("S"), ws,
                         ctypes.c_size_t(nf), None))
    ok(lib.gdn_chunk_fwd_noalloc(q, k, v, g, b, 0, F(0.1), None, None, 1, 1, I64(256), H, H, d, d, 64, p("o2"),
                                 None, None))
    for chunk, dq in ((64, "dq"), (32, "dq3")):
        ok(lib.gdn_chunk_bwd(q, I64(H * d), k, I64(H * d), v, I64(H * d), g, b, do, 0, F(0.1), None, None, None, 1,
                             1, I64(T), H, H, d, d, chunk, p(dq), p("dk"), p("dv"), p("dg"), p("db"), None, ws,
                             ctypes.c_size_t(nb), None))
    ok(lib.gdn_causal_conv1d_silu(q, 0, put("w", rng.random((H * d, 4), np.float32)), None, 1, I64(T), H * d, 4,
                                  None, 1, 0, 0, F(1e-6), None, None, p("y"), None))
    ok(cuda.cuCtxSynchronize())
    for n, a in out.items():
        ok(cuda.cuMemcpyDtoH_v2(a.ctypes.data_as(V), p(n), ctypes.c_size_t(a.nbytes)))
        assert a.any(), n
    return out


ok(cuda.cuInit(0))
dev = ctypes.c_int()
ok(cuda.cuDeviceGet(ctypes.byref(dev), 0))
first = run()
ok(cuda.cuDevicePrimaryCtxReset_v2(dev))  # ends this process's context, no more
second = run()
for n in first:
    assert np.array_equal(first[n], second[n]), n
print("same")
'''


@pytest.mark.gpu
def test_calls_after_the_context_was_replaced():
    lib = os.path.join(ROOT, "gated_deltanet_fwd_b200", "libgdn.so")
    r = subprocess.run([sys.executable, "-c", CHILD, lib], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr
