"""Backward passes of the gates, the gated RMSNorm and the conv, and the 8-bit activation checkpoints,
against 64-bit references; and one training step of the whole layer core.

Tolerances.  Outputs in bf16 are one rounding of a value computed in fp32: 2^-8 of the value, and an
absolute part for values that cancel, ABS = 2e-6 times the sizes of the terms (here about 1 to 10, so
2e-5).  fp32 outputs: a few dozen fp32 operations and fast exponentials of relative error 2e-6, and
sums whose terms' errors add in squares: 1e-5 norm-wise, and 2e-5 relative to the largest of a row or
of the terms elementwise.  Codes and scales are exact."""
import numpy as np
import pytest
import torch

import bwd_reference as ref
from gdn_testutil import rel_l2
from gated_deltanet_fwd_b200 import gdn

gpu = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SUM_TOL = 1e-5


def near(y, want, what):
    """y within its type's rounding of want."""
    y, w = ref.d64(y).reshape(want.shape), want
    if not w.numel():
        return
    half = 2.0 ** -8
    rel = half if what.startswith("bf16") else 0.0
    size = max(1.0, w.abs().max().item())
    err = (y - w).abs()
    assert (err <= rel * w.abs() + 2e-5 * size).all(), (what, (err - rel * w.abs()).max().item(), size)


def sums(y, want, what):
    n = want.norm().item()
    assert (ref.d64(y) - want).norm().item() <= SUM_TOL * max(n, 1e-30) or n == 0 and not y.any(), \
        (what, rel_l2(y, want))


def rn(gen, *s, std=1.0):
    return torch.randn(*s, generator=gen) * std


# ------------------------------------------------------------------------------- gates -----

@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,Hv", [(1, 1), (3, 32), (1000, 6), (777, 64), (33, 300), (5, 2056), (4096, 32)])
def test_gates(n, Hv, dtype):
    gen = torch.Generator().manual_seed(n)
    a, b, dg, dbeta = (rn(gen, n, Hv, std=s).to(DT[dtype]) for s in (2.0, 2.0, 1.0, 1.0))
    A, bias = torch.log(torch.rand(Hv, generator=gen) * 15 + 1), rn(gen, Hv, std=0.1)
    want = ref.gates_grads(a, b, A, bias, dg, dbeta)
    got = gdn.gdn_gates_bwd(*(t.cuda() for t in (a, b, A, bias, dg, dbeta)))
    near(got[0], want[0], dtype + " da")
    near(got[1], want[1], dtype + " db")
    sums(got[2], want[2], "dA_log")
    sums(got[3], want[3], "ddt_bias")


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_extremes_and_views(dtype):
    """Pre-activations far out on both sides; rows that start off a 16-byte boundary."""
    vals = torch.tensor([0.0, 80.0, -80.0, 300.0, -300.0, 20.0, -20.0, 1.0])
    a = vals[None].repeat(3, 1).to(DT[dtype])
    one = torch.ones(3, 8, dtype=DT[dtype])
    A, bias = torch.zeros(8), torch.zeros(8)
    want = ref.gates_grads(a, a, A, bias, one, one)
    buf = [torch.empty(25, dtype=DT[dtype], device="cuda") for _ in range(4)]
    odd = [t[1:].view(3, 8) for t in buf]
    for t, v in zip(odd, (a, a, one, one)):
        t.copy_(v)
    for args in ([t.cuda() for t in (a, a, one, one)], odd):
        got = gdn.gdn_gates_bwd(args[0], args[1], A.cuda(), bias.cuda(), args[2], args[3])
        near(got[0], want[0], dtype + " da")
        near(got[1], want[1], dtype + " db")
        assert all(torch.isfinite(t).all() for t in got)


@gpu
def test_gates_no_tokens():
    e = torch.empty(0, 4, device="cuda")
    A = torch.ones(4, device="cuda")
    got = gdn.gdn_gates_bwd(e, e, A, A, e, e)
    assert (got[2] == 0).all() and (got[3] == 0).all()


# -------------------------------------------------------------------------------- norm -----

@gpu
@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dim", [(1, 8), (5, 16), (33, 32), (257, 64), (1, 128), (1003, 128), (130, 256),
                                      (40000, 128)])
def test_norm(rows, dim, dtype, ckpt):
    gen = torch.Generator().manual_seed(rows + dim)
    x, z, dy = (rn(gen, rows, dim, std=s).to(DT[dtype]) for s in (1.0, 1.0, 1.0))
    w = rn(gen, dim, std=0.1)
    if ckpt:
        (xc, xs, xv), (zc, zs, zv) = ref.act8(x, dim), ref.act8(z, dim)
        want = ref.norm_grads(dy, xv, zv, w, 1e-6)
        xin, zin = (xc.cuda(), xs.cuda()), (zc.cuda(), zs.cuda())
    else:
        want = ref.norm_grads(dy, x, z, w, 1e-6)
        xin, zin = x.cuda(), z.cuda()
    got = gdn.gdn_gated_rmsnorm_bwd(dy.cuda(), xin, zin, w.cuda())
    near(got[0], want[0], dtype + " dx")
    near(got[1], want[1], dtype + " dz")
    sums(got[2], want[2], "dw")
    again = gdn.gdn_gated_rmsnorm_bwd(dy.cuda(), xin, zin, w.cuda())
    assert all(torch.equal(p, q) for p, q in zip(got, again))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_rows_of_zeros_and_far_gates(dtype):
    x = torch.zeros(4, 64)
    x[1:] = torch.linspace(-1, 1, 64)
    z = torch.zeros(4, 64)
    z[2], z[3] = -200.0, 200.0
    dy, w = torch.ones(4, 64), torch.zeros(64)
    x, z, dy = (t.to(DT[dtype]) for t in (x, z, dy))
    want = ref.norm_grads(dy, x, z, w, 1e-6)
    got = gdn.gdn_gated_rmsnorm_bwd(dy.cuda(), x.cuda(), z.cuda(), w.cuda())
    assert all(torch.isfinite(t).all() for t in got)
    near(got[0], want[0], dtype + " dx")
    near(got[1], want[1], dtype + " dz")


@gpu
def test_norm_no_rows():
    e = torch.empty(0, 64, device="cuda")
    assert (gdn.gdn_gated_rmsnorm_bwd(e, e, e, torch.ones(64, device="cuda"))[2] == 0).all()


# ------------------------------------------------------------------ 8-bit checkpoints -----

@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dim,group", [(1, 8, 8), (7, 48, 16), (100, 96, 32), (33, 640, 64), (1000, 384, 128),
                                            (3, 512, 256)])
def test_pack_unpack(rows, dim, group, dtype):
    gen = torch.Generator().manual_seed(rows)
    x = rn(gen, rows, dim).to(DT[dtype])
    x[0, :group] = 0.0
    if rows > 2:
        x[1] *= 1e-20
        x[2] *= 1e20
        x[2, 3] = 5e22  # one value far above its group
    codes, scales, vals = ref.act8(x, group)
    c, s = gdn.gdn_act_pack8(x.cuda(), group=group)
    assert torch.equal(c.cpu(), codes) and torch.equal(s.cpu(), scales)
    assert int(c.abs().max()) == (127 if vals.any() else 0)
    y = gdn.gdn_act_unpack8(c, s, dtype=DT[dtype]).cpu()
    assert torch.equal(y, vals.float().to(DT[dtype]))
    m = x.double().unflatten(-1, (-1, group)).abs().amax(-1, keepdim=True)
    off = (vals.unflatten(-1, (-1, group)) - x.double().unflatten(-1, (-1, group))).abs()
    # |x inv - code| <= 1/2, inv = 127/m (1 + d), scale = m/127 (1 + e), |d|, |e| <= 2^-24:
    # |code scale - x| <= scale / 2 + |x| |inv scale - 1| <= m/254 (1 + 2^-24) + m (2^-23 + 2^-48)
    assert (off <= m / 254 + m * 2.0 ** -22.9).all()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pack_non_finite_and_tiny_groups(dtype):
    x = torch.ones(4, 64)
    x[0, 5], x[1, 40], x[2, :32] = float("inf"), float("nan"), 1e-38
    c, s = gdn.gdn_act_pack8(x.to(DT[dtype]).cuda(), group=32)
    y = gdn.gdn_act_unpack8(c, s, dtype=torch.float32).cpu()
    assert torch.isnan(y[0, :32]).all() and torch.isnan(y[1, 32:]).all()
    assert (y[2, :32] == 0).all()
    assert torch.allclose(y[0, 32:], torch.ones(32)) and torch.allclose(y[3], torch.ones(64))


@gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,dim", [(1, 8), (77, 32), (999, 128), (40, 256)])
def test_norm_that_keeps_its_checkpoint(rows, dim, dtype, in_place):
    gen = torch.Generator().manual_seed(rows)
    x, z = rn(gen, rows, dim).to(DT[dtype]), rn(gen, rows, dim).to(DT[dtype])
    w = rn(gen, dim, std=0.1)
    xg = x.cuda()
    plain = gdn.gdn_gated_rmsnorm(xg, z.cuda(), w.cuda())
    y, x8, z8 = gdn.gdn_gated_rmsnorm_ckpt8(xg, z.cuda(), w.cuda(), y=xg if in_place else None)
    assert torch.equal(y, plain) and (y.data_ptr() == xg.data_ptr()) == in_place
    for (c, s), src in ((x8, x), (z8, z)):
        codes, scales, _ = ref.act8(src, dim)
        assert torch.equal(c.cpu(), codes) and torch.equal(s.cpu(), scales)


# -------------------------------------------------------------------------------- conv -----

CONV = [
    # lens, packed, C, K, n_l2, group, bias, states
    ([1], False, 8, 1, 0, 0, False, False),
    ([5, 5], False, 64, 4, 32, 32, True, True),
    ([17, 1, 0, 33, 2], True, 256, 4, 128, 64, True, True),
    ([0, 3, 0], True, 136, 8, 0, 0, False, True),
    ([40, 7], True, 384, 3, 256, 128, False, True),
    ([50, 1, 30], True, 768, 2, 512, 256, True, True),
    ([300], False, 520, 5, 512, 256, False, False),
    ([700, 2, 701], True, 128, 4, 128, 128, False, True),
    ([64], False, 1024, 7, 256, 32, True, False),
]


def conv_case(lens, packed, C, K, n_l2, group, bias, states, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed + sum(lens))
    T, N = sum(lens), len(lens)
    s = dict(x=rn(gen, T, C).to(DT[dtype]), dy=rn(gen, T, C).to(DT[dtype]),
             w=(torch.rand(C, K, generator=gen) * 2 - 1) / K ** 0.5,
             bias=rn(gen, C, std=0.1) if bias else None,
             hist=rn(gen, N, C, K - 1) if states else None, dleft=rn(gen, N, C, K - 1) if states else None,
             cu=torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32) if packed else None)
    s["shape"] = (1, T, C) if packed else (N, lens[0], C)
    return s


def conv_call(s, n_l2, group, x=None, **kw):
    up = lambda t: None if t is None else t.cuda()
    x = s["x"].reshape(s["shape"]).cuda() if x is None else x
    return gdn.gdn_causal_conv1d_silu_bwd(
        s["dy"].reshape(s["shape"]).cuda(), x, s["w"].cuda(), up(s["bias"]), cu_seqlens=up(s["cu"]),
        n_l2norm_ch=n_l2, l2norm_group=group, conv_state_in=up(s["hist"]), dconv_state_out=up(s["dleft"]), **kw)


@gpu
@pytest.mark.parametrize("ckpt", [0, 8, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,packed,C,K,n_l2,group,bias,states", CONV)
def test_conv(lens, packed, C, K, n_l2, group, bias, states, dtype, ckpt):
    s = conv_case(lens, packed, C, K, n_l2, group, bias, states, dtype)
    if ckpt and C % ckpt:
        ckpt = 8
    x, xin = s["x"], None
    if ckpt:
        codes, scales, x = ref.act8(s["x"], ckpt)
        xin = (codes.reshape(s["shape"]).cuda(), scales.reshape(*s["shape"][:-1], -1).cuda())
    want = ref.conv_grads(s["dy"], x, s["w"], s["bias"], s["hist"], s["dleft"], lens, n_l2, group, 1e-6)
    got = conv_call(s, n_l2, group, xin)
    near(got[0], want[0], dtype + " dx")
    sums(got[1], want[1], "dw")
    if bias:
        sums(got[2], want[2], "dbias")
    else:
        assert got[2] is None
    if states:
        near(got[3], want[3], "f32 dhist")
    else:
        assert got[3] is None
    assert all(torch.equal(p, q) for p, q in zip(got, conv_call(s, n_l2, group, xin)) if p is not None)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_conv_no_tokens_and_tokens_behind(dtype):
    s = conv_case([0, 0], True, 16, 4, 0, 0, True, True, dtype)
    dx, dw, dbias, dh = conv_call(s, 0, 0)
    assert (dw == 0).all() and (dbias == 0).all() and torch.equal(dh.cpu(), s["dleft"])
    lens = [9, 20]
    s = conv_case(lens, True, 64, 4, 64, 32, False, True, dtype)
    want = conv_call(s, 64, 32)
    grow = lambda t: torch.cat([t, torch.full((21, 64), float("nan"), dtype=t.dtype)])
    t = dict(s, x=grow(s["x"]), dy=grow(s["dy"]), shape=(1, 50, 64))
    dx = torch.full((1, 50, 64), 7.0, dtype=DT[dtype], device="cuda")
    got = conv_call(t, 64, 32, dx=dx)
    assert torch.equal(got[0][:, :29], want[0]) and (dx[:, 29:] == 7.0).all()
    sums(got[1], ref.d64(want[1]), "dw")
    assert torch.equal(got[3], want[3])


# ------------------------------------------------------- conduct shared by these calls -----

@gpu
def test_graph_replay_and_second_stream():
    """Norm, gates and conv backward captured in one graph, replayed on new inputs, and run on a stream
    of their own: the eager results."""
    def inputs(seed):
        gen = torch.Generator().manual_seed(seed)
        b = torch.bfloat16
        return dict(dy=rn(gen, 300, 128).to(b), x=rn(gen, 300, 128).to(b), z=rn(gen, 300, 128).to(b), w=rn(gen, 128),
                    a=rn(gen, 90, 8).to(b), b=rn(gen, 90, 8).to(b), A=rn(gen, 8), dt=rn(gen, 8),
                    dg=rn(gen, 90, 8).to(b), db=rn(gen, 90, 8).to(b), cx=rn(gen, 2, 40, 64).to(b),
                    cy=rn(gen, 2, 40, 64).to(b), cw=rn(gen, 64, 4))

    def step(t):
        y, x8, z8 = gdn.gdn_gated_rmsnorm_ckpt8(t["x"], t["z"], t["w"])
        return [y, *gdn.gdn_gated_rmsnorm_bwd(t["dy"], x8, z8, t["w"]),
                *gdn.gdn_gates_bwd(t["a"], t["b"], t["A"], t["dt"], t["dg"], t["db"]),
                *gdn.gdn_causal_conv1d_silu_bwd(t["cy"], gdn.gdn_act_pack8(t["cx"], group=32), t["cw"],
                                                n_l2norm_ch=32, l2norm_group=32)[:2]]

    one, two = ({n: v.cuda() for n, v in inputs(s).items()} for s in (1, 2))
    want1, want2 = step(one), step(two)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        side = step(two)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(side, want2))
    live = {n: v.clone() for n, v in one.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(live)
    for src, want in ((two, want2), (one, want1)):
        for n in live:
            live[n].copy_(src[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))


@gpu
@pytest.mark.parametrize("ckpt", [False, True])
def test_training_step_of_the_layer_core(ckpt):
    """conv -> gates -> rule -> norm and back through all of them, fp32, against automatic differentiation of
    the 64-bit composition.  With checkpoints the backward reads the conv's input, the rule's output and
    z from 8 bits: its gradients are those of the kept values, compared with the same composition around
    them; the rule itself recomputes from the conv's exact output."""
    lens, Hk, Hv, d, K, eps = [37, 20], 1, 2, 32, 4, 1e-6
    C, T = 2 * Hk * d + Hv * d, sum(lens)
    gen = torch.Generator().manual_seed(4)
    p = dict(mix=rn(gen, T, C), w=(torch.rand(C, K, generator=gen) * 2 - 1) / 2, a=rn(gen, T, Hv), b=rn(gen, T, Hv),
             A=torch.log(torch.rand(Hv, generator=gen) * 3 + 1), dt=rn(gen, Hv, std=0.1), z=rn(gen, T, Hv, d),
             nw=rn(gen, d, std=0.1))
    dy = rn(gen, T, Hv, d)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32).cuda()
    g = {n: v.cuda() for n, v in p.items()}
    # forward
    y = gdn.gdn_causal_conv1d_silu(g["mix"][None], g["w"], cu_seqlens=cu, n_l2norm_ch=2 * Hk * d, l2norm_group=d)
    q, k, v = (t.unflatten(-1, (-1, d)) for t in y.split([Hk * d, Hk * d, Hv * d], -1))
    gate, beta = gdn.gdn_gates(g["a"][None], g["b"][None], g["A"], g["dt"])
    q, k, v = (t.contiguous() for t in (q, k, v))
    o, _ = gdn.gdn_chunk_fwd(q, k, v, gate, beta, cu_seqlens=cu, chunk=32)
    z = g["z"][None]
    if ckpt:
        mix8 = gdn.gdn_act_pack8(g["mix"][None], group=32)
        _, o_in, z_in = gdn.gdn_gated_rmsnorm_ckpt8(o, z, g["nw"])
    else:
        mix8, o_in, z_in = g["mix"][None], o, z
    # backward
    do, dz, dnw = gdn.gdn_gated_rmsnorm_bwd(dy[None].cuda(), o_in, z_in, g["nw"])
    dq, dk, dv, dg, dbeta, _ = gdn.gdn_chunk_bwd(q, k, v, gate, beta, do, cu_seqlens=cu, chunk=32)
    da, db, dA, ddt = gdn.gdn_gates_bwd(g["a"][None], g["b"][None], g["A"], g["dt"], dg, dbeta)
    dconv = torch.cat([dq.flatten(2), dk.flatten(2), dv.flatten(2)], -1)
    dmix, dw, _, _ = gdn.gdn_causal_conv1d_silu_bwd(dconv, mix8, g["w"], cu_seqlens=cu, n_l2norm_ch=2 * Hk * d,
                                                    l2norm_group=d)
    got = dict(mix=dmix, w=dw, a=da, b=db, A=dA, dt=ddt, z=dz, nw=dnw)
    # reference
    zero = torch.zeros(len(lens), C, K - 1, dtype=ref.D)
    r = {n: ref.d64(t).requires_grad_() for n, t in p.items()}

    def conv_of(mix):
        return ref.conv(mix, r["w"], torch.zeros(C, dtype=ref.D), zero, lens, 2 * Hk * d, d, eps)[0]

    def core(yc):
        qr, kr, vr = (t.unflatten(-1, (-1, d)) for t in yc.split([Hk * d, Hk * d, Hv * d], -1))
        gr = -torch.exp(r["A"]) * torch.logaddexp(r["a"] + r["dt"], torch.zeros((), dtype=ref.D))
        return ref.rule(qr, kr, vr, gr, torch.sigmoid(r["b"]), d ** -0.5, None, lens)[0]

    if not ckpt:
        loss = (ref.norm(core(conv_of(r["mix"])), r["z"], r["nw"], eps) * ref.d64(dy)).sum()
        want = dict(zip(r, torch.autograd.grad(loss, list(r.values()))))
    else:
        ok, zk = (ref.act8(t[0], d)[2].requires_grad_() for t in (o, z))
        dok, dzk, dnwk = torch.autograd.grad((ref.norm(ok, zk, r["nw"], eps) * ref.d64(dy)).sum(), (ok, zk, r["nw"]))
        yc = ref.d64(y[0]).requires_grad_()
        dyc, *rest = torch.autograd.grad((core(yc) * dok).sum(), (yc, r["a"], r["b"], r["A"], r["dt"]))
        mk = ref.act8(p["mix"], 32)[2].requires_grad_()
        dmk, dwk = torch.autograd.grad((conv_of(mk) * dyc).sum(), (mk, r["w"]))
        want = dict(mix=dmk, w=dwk, z=dzk, nw=dnwk, **dict(zip(("a", "b", "A", "dt"), rest)))
    for n in got:
        # four operators of at most 1e-5 and 2e-5 each in a row
        err = rel_l2(got[n].reshape(want[n].shape), want[n].detach())
        assert err <= 5e-5, (n, err)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hv", [3, 16])
@pytest.mark.parametrize("cu", [[0, 40, 75], [4, 4, 30], [0, 0], [100], [-9, 50, 300], [60, 20]])
def test_gates_outside_every_sequence(cu, Hv, dtype):
    """Only the tokens that cu_seqlens spans are read and written, whatever the others hold; entries outside the
    tensor are clamped to it."""
    gen = torch.Generator().manual_seed(6)
    n, dt = 100, DT[dtype]
    lo = min(max(cu[0], 0), n)
    hi = min(max(cu[-1], lo), n)
    x = [rn(gen, n, Hv).to(dt) for _ in range(4)]
    A, bias = rn(gen, Hv), rn(gen, Hv, std=0.1)
    want = ref.gates_grads(x[0][lo:hi], x[1][lo:hi], A, bias, x[2][lo:hi], x[3][lo:hi])
    for t in x:
        t[:lo] = t[hi:] = float("nan")
    a, b, dg, db_ = (t.cuda() for t in x)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    held = [torch.full((n, Hv), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    got = gdn.gdn_gates_bwd(a, b, A.cuda(), bias.cuda(), dg, db_, da=held[0], db=held[1], cu_seqlens=c)
    new = gdn.gdn_gates_bwd(a, b, A.cuda(), bias.cuda(), dg, db_, cu_seqlens=c)
    for i in range(2):
        near(got[i][lo:hi], want[i], dtype)
        assert torch.equal(got[i][lo:hi], new[i][lo:hi])
        for rows in (slice(0, lo), slice(hi, n)):
            assert (held[i][rows] == 7.0).all() and (new[i][rows] == 0.0).all()
    for y, z, w in zip(got[2:], new[2:], want[2:]):
        sums(y, w, dtype)
        assert torch.equal(y, z)


@gpu
@pytest.mark.parametrize("dtype,d", [("f32", 32), ("bf16", 128)])
@pytest.mark.parametrize("given", [True, False])
def test_gates_after_the_rule_on_a_padded_batch(given, dtype, d):
    """The sums over tokens start from dg and dbeta of the rule, whose padding tokens are never written."""
    from test_bwd_rule import make
    lens, T, Hv, dt = [250, 0, 40], 320, 2, DT[dtype]
    x = make(lens, 1, Hv, d, d, dtype, False, seed=89)
    gen = torch.Generator().manual_seed(7)
    x["a"], x["b"] = rn(gen, 290, Hv).to(dt), rn(gen, 290, Hv).to(dt)
    A, bias, cu = rn(gen, Hv).cuda(), rn(gen, Hv, std=0.1).cuda(), x["cu"].cuda()
    nan = lambda *s: torch.full(s, float("nan"), dtype=dt, device="cuda")
    pad = lambda t: torch.cat([t, torch.full((T - 290, *t.shape[1:]), float("nan"), dtype=t.dtype)])[None].cuda()
    t = {n: pad(x[n]) for n in ("q", "k", "v", "g", "beta", "dout", "a", "b")}
    own = dict(dg=nan(1, T, Hv), dbeta=nan(1, T, Hv)) if given else {}
    _, _, _, dg, dbeta, _ = gdn.gdn_chunk_bwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["dout"], cu_seqlens=cu,
                                              **own)
    if not given:
        assert (dg[:, 290:] == 0).all() and (dbeta[:, 290:] == 0).all()
        for n in ("dg", "dbeta"):  # one given, one made
            two = gdn.gdn_chunk_bwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["dout"], cu_seqlens=cu,
                                    **{n: nan(1, T, Hv)})[3:5]
            made, kept = two[n == "dg"], two[n != "dg"]
            assert (made[:, 290:] == 0).all() and kept[:, 290:].isnan().all()
    da, db, dA, ddt = gdn.gdn_gates_bwd(t["a"], t["b"], A, bias, dg, dbeta, cu_seqlens=cu)
    want = gdn.gdn_gates_bwd(*(v[:, :290].contiguous() for v in (t["a"], t["b"])), A, bias,
                             *(v[:, :290].contiguous() for v in (dg, dbeta)))
    assert torch.equal(da[:, :290], want[0]) and torch.equal(db[:, :290], want[1])
    assert (da[:, 290:] == 0).all() and (db[:, 290:] == 0).all()
    # the same fp32 terms in another order: a thread's sum over its few tokens
    for y, w in zip((dA, ddt), want[2:]):
        sums(y, ref.d64(w), dtype)


@gpu
@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("dtype,H,dim", [("bf16", 3, 128), ("f32", 2, 64), ("bf16", 1, 8)])
@pytest.mark.parametrize("cu", [[0, 40, 75], [4, 4, 30], [0, 0], [100], [-9, 50, 300], [60, 20]])
def test_norm_outside_every_sequence(cu, dtype, H, dim, ckpt):
    """As for the gates: rows of other tokens are neither read nor written."""
    gen = torch.Generator().manual_seed(8)
    n, dt, eps = 100, DT[dtype], 1e-6
    lo = min(max(cu[0], 0), n)
    hi = min(max(cu[-1], lo), n)
    dy, x, z = (rn(gen, n, H, dim).to(dt) for _ in range(3))
    w = rn(gen, dim, std=0.1)
    for t in (dy, x, z):
        t[:lo] = t[hi:] = float("nan")
    dy, x, z = (t.cuda() for t in (dy, x, z))
    kept = [gdn.gdn_act_pack8(t, dim) for t in (x, z)] if ckpt else [x, z]
    vals = [ref.d64(k[0][lo:hi]) * ref.d64(k[1][lo:hi]) if ckpt else ref.d64(k[lo:hi]) for k in kept]
    want = ref.norm_grads(dy[lo:hi], *vals, w, eps)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    held = [torch.full((n, H, dim), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    got = gdn.gdn_gated_rmsnorm_bwd(dy, *kept, w.cuda(), dx=held[0], dz=held[1], cu_seqlens=c)
    for y, v in zip(got[:2], want):
        near(y[lo:hi], v, dtype)
        assert (y[:lo] == 7.0).all() and (y[hi:] == 7.0).all()
    sums(got[2], want[2], dtype)


@gpu
@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("dtype,d", [("f32", 32), ("bf16", 128)])
def test_training_step_on_a_padded_batch(dtype, d, ckpt):
    """Sequences packed into a longer row: NaN in every padding row of the inputs and in every buffer that a
    call leaves partly unwritten.  Each gradient has the bits, and each sum over tokens the value, of the
    step on the packed tokens alone."""
    lens, pad_, Hk, Hv, K, dt = [250, 0, 40], 30, 1, 2, 4, DT[dtype]
    C, n = 2 * Hk * d + Hv * d, sum(lens)
    gen = torch.Generator().manual_seed(9)
    p = dict(mix=rn(gen, n, C), a=rn(gen, n, Hv), b=rn(gen, n, Hv), z=rn(gen, n, Hv, d), dy=rn(gen, n, Hv, d))
    w = dict(w=(torch.rand(C, K, generator=gen) * 2 - 1) / 2, A=torch.log(torch.rand(Hv, generator=gen) * 3 + 1),
             dt=rn(gen, Hv, std=0.1), nw=rn(gen, d, std=0.1))
    w = {m: v.cuda() for m, v in w.items()}
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32).cuda()

    def step(T):
        nan = lambda *s, t=dt: torch.full((1, T, *s), float("nan"), dtype=t, device="cuda")
        t = {m: nan(*v.shape[1:]) for m, v in p.items()}
        for m, v in p.items():
            t[m][0, :n] = v.to(dt)
        y = gdn.gdn_causal_conv1d_silu(t["mix"], w["w"], cu_seqlens=cu, n_l2norm_ch=2 * Hk * d, l2norm_group=d,
                                       y=nan(C))
        q, k, v = (s.unflatten(-1, (-1, d)) for s in y.split([Hk * d, Hk * d, Hv * d], -1))
        g, beta = gdn.gdn_gates(t["a"], t["b"], w["A"], w["dt"])
        # the rule's output, as any: what a forward leaves behind the last sequence is not defined
        o = nan(Hv, d)
        o[0, :n] = (v[0, :n].float() * beta[0, :n, :, None]).to(dt)
        o8, z8 = (o, t["z"]) if not ckpt else gdn.gdn_gated_rmsnorm_ckpt8(o, t["z"], w["nw"])[1:]
        mix8 = gdn.gdn_act_pack8(t["mix"], group=32) if ckpt else t["mix"]
        do, dz, dnw = gdn.gdn_gated_rmsnorm_bwd(t["dy"], o8, z8, w["nw"], dx=nan(Hv, d), cu_seqlens=cu)
        dq, dk, dv, dg, db, _ = gdn.gdn_chunk_bwd(q, k, v, g, beta, do, cu_seqlens=cu, dq=nan(Hk, d), dk=nan(Hk, d),
                                                  dv=nan(Hv, d), dg=nan(Hv), dbeta=nan(Hv))
        da, dbb, dA, ddt = gdn.gdn_gates_bwd(t["a"], t["b"], w["A"], w["dt"], dg, db, cu_seqlens=cu)
        dmix, dw, _, _ = gdn.gdn_causal_conv1d_silu_bwd(torch.cat([s.flatten(2) for s in (dq, dk, dv)], -1), mix8,
                                                        w["w"], cu_seqlens=cu, n_l2norm_ch=2 * Hk * d, l2norm_group=d)
        return dict(dmix=dmix, dz=dz, da=da, db=dbb), dict(dw=dw, dnw=dnw, dA=dA, ddt=ddt)

    rows, total = step(n)
    padded, total2 = step(n + pad_)
    for m in rows:
        assert torch.equal(padded[m][:, :n], rows[m]), m
    for m in total:  # the same terms, split into other ranges
        sums(total2[m], ref.d64(total[m]), m)


# ------------------------------------------------------------------------ refusals (CPU) ----

P = 0x7f0000000000
at = lambda i: P + (i << 32)
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: only without a GPU")
E, U = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED
BIG = 1 << 31


@no_gpu
def test_gates_refusals():
    f = gdn.load().gdn_gates_bwd

    def c(a=at(1), b=at(2), dt=0, A=at(3), bi=at(4), dg=at(5), de=at(6), n=64, Hv=8, da=at(7), db=at(8),
          dA=at(9), dbi=at(10), ws=at(11), wsb=BIG):
        return f(a, b, dt, A, bi, dg, de, n, Hv, da, db, dA, dbi, ws, wsb, None)

    assert c(dt=3) == E and c(n=-1) == E and c(Hv=0) == E
    for n in ("a", "b", "A", "bi", "dg", "de", "da", "db", "dA", "dbi", "ws"):
        assert c(**{n: None}) == E, n
    assert c(ws=at(11) + 8) == E and c(wsb=16) == E
    assert c(da=at(1)) == E and c(db=at(7) + 16) == E


@no_gpu
def test_gates_varlen_refusals():
    f = gdn.load().gdn_gates_bwd_varlen

    def c(a=at(1), cu=at(12), N=2, n=64, da=at(7), ws=at(11), wsb=BIG):
        return f(a, at(2), 0, at(3), at(4), at(5), at(6), cu, N, n, 8, da, at(8), at(9), at(10), ws, wsb, None)

    assert c(N=-1) == E and c(cu=at(12) + 2) == E and c(a=None) == E and c(n=-1) == E and c(wsb=16) == E
    assert c(cu=at(7)) == E               # da over cu_seqlens
    assert c(cu=at(11) + 8) == E          # the workspace over it


@no_gpu
def test_norm_refusals():
    f = gdn.load().gdn_gated_rmsnorm_bwd

    def c(dy=at(1), x=at(2), xs=None, z=at(3), zs=None, dt=0, w=at(4), eps=1e-6, n=64, dim=128, dx=at(5),
          dz=at(6), dw=at(7), ws=at(8), wsb=BIG):
        return f(dy, x, xs, z, zs, dt, w, eps, n, dim, dx, dz, dw, ws, wsb, None)

    assert c(dt=3) == E and c(n=-1) == E and c(eps=-1.0) == E and c(eps=float("nan")) == E
    assert c(dim=96) == U and c(dim=512) == U
    for n in ("dy", "x", "z", "w", "dx", "dz", "dw", "ws"):
        assert c(**{n: None}) == E, n
    assert c(xs=at(9)) == E and c(zs=at(9)) == E       # one checkpoint, one activation
    assert c(x=at(2) + 8) == E and c(dx=at(5) + 2) == E
    assert c(wsb=64) == E and c(dx=at(1)) == E and c(dz=at(3)) == E
    g = gdn.load().gdn_gated_rmsnorm_ckpt8
    k = lambda x=at(1), z=at(2), y=at(3), xc=at(4), xs=at(5), zc=at(6), zs=at(7), dim=128: \
        g(x, z, 0, at(8), 1e-6, 64, dim, y, xc, xs, zc, zs, None)
    assert k(dim=48) == U
    for n in ("x", "z", "y", "xc", "xs", "zc", "zs"):
        assert k(**{n: None}) == E, n
    assert k(y=at(2)) == E and k(y=at(1) + 16) == E and k(zc=at(4)) == E and k(xc=at(1)) == E


@no_gpu
def test_norm_varlen_refusals():
    f = gdn.load().gdn_gated_rmsnorm_bwd_varlen

    def c(dy=at(1), cu=at(12), N=2, per=4, n=64, dx=at(5), ws=at(8), wsb=BIG):
        return f(dy, at(2), None, at(3), None, 0, at(4), 1e-6, cu, N, per, n, 128, dx, at(6), at(7), ws, wsb, None)

    assert c(N=-1) == E and c(per=0) == E and c(per=7) == E and c(cu=at(12) + 2) == E
    assert c(dy=None) == E and c(wsb=64) == E and c(cu=at(5)) == E and c(cu=at(8) + 8) == E


@no_gpu
def test_pack_refusals():
    lib = gdn.load()
    for f, first in ((lib.gdn_act_pack8, True), (lib.gdn_act_unpack8, False)):
        def c(x=at(1), c8=at(2), sc=at(3), dt=0, n=4, dim=256, group=64):
            return f(x, dt, n, dim, group, c8, sc, None) if first else f(c8, sc, dt, n, dim, group, x, None)
        assert c(dt=4) == E and c(n=-1) == E and c(dim=0) == E and c(group=0) == E
        assert c(group=96) == E and c(group=512, dim=512) == U and c(group=4) == U
        for n in ("x", "c8", "sc"):
            assert c(**{n: None}) == E, n
        assert c(x=at(1) + 8) == E and c(c8=at(1)) == E
        assert c(n=0, x=None, c8=None, sc=None) == gdn.GDN_OK


@no_gpu
def test_conv_refusals():
    f = gdn.load().gdn_causal_conv1d_silu_bwd

    def c(dy=at(1), x=at(2), xs=None, xg=0, dt=0, w=at(3), bias=None, B=1, T=64, C=256, K=4, cu=None, N=1, l2=0,
          group=0, eps=1e-6, h=None, dl=None, dx=at(4), dw=at(5), db=None, dh=None, ws=at(6), wsb=BIG):
        return f(dy, x, xs, xg, dt, w, bias, B, T, C, K, cu, N, l2, group, eps, h, dl, dx, dw, db, dh, ws, wsb, None)

    assert c(dt=3) == E and c(T=-1) == E and c(N=2) == E and c(cu=at(9), B=2, N=2) == E
    assert c(C=260) == U and c(K=9) == U and c(group=48, l2=48) == U
    assert c(l2=100, group=32) == E and c(l2=512, group=32) == E and c(l2=32) == E
    assert c(eps=-1.0) == E
    for n in ("dy", "x", "w", "dx", "dw", "ws"):
        assert c(**{n: None}) == E, n
    assert c(bias=at(7)) == E and c(db=at(7)) == E     # dbias exactly with bias
    assert c(xs=at(8), xg=0) == E and c(xs=at(8), xg=96) == E and c(xs=at(8), xg=4) == U
    assert c(dx=at(1)) == E and c(dx=at(2)) == E and c(wsb=100) == E
    assert c(dh=at(10), dl=at(10)) == E


def test_binding_refuses_before_the_library():
    """Shapes, types and pairs that do not fit are refused on the host (CPU tensors are refused first)."""
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        gdn.gdn_act_pack8(x)
    with pytest.raises(ValueError):
        gdn.gdn_gated_rmsnorm_bwd(x, x, (x.to(torch.int8), x[:, :1].contiguous()), x[0])
    with pytest.raises(TypeError):
        gdn.gdn_gated_rmsnorm_bwd(x, (x, x), (x, x), x[0])


@gpu
def test_binding_refusals():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")
    f32 = torch.float32
    with pytest.raises(TypeError):  # gradients of another type than the activations
        gdn.gdn_gates_bwd(z(4, 8), z(4, 8), z(8, dt=f32), z(8, dt=f32), z(4, 8, dt=f32), z(4, 8))
    with pytest.raises(ValueError):
        gdn.gdn_gates_bwd(z(4, 8), z(4, 8), z(4, dt=f32), z(4, dt=f32), z(4, 8), z(4, 8))
    with pytest.raises(ValueError):  # one scale for two rows
        gdn.gdn_gated_rmsnorm_bwd(z(4, 64), (z(4, 64, dt=torch.int8), z(2, 1, dt=f32)),
                                  (z(4, 64, dt=torch.int8), z(2, 1, dt=f32)), z(64, dt=f32))
    with pytest.raises(ValueError):
        gdn.gdn_causal_conv1d_silu_bwd(z(1, 8, 64), z(1, 9, 64), z(64, 4, dt=f32))
    with pytest.raises(ValueError):  # scales of another number of tokens
        gdn.gdn_causal_conv1d_silu_bwd(z(1, 8, 64), (z(1, 8, 64, dt=torch.int8), z(1, 7, 1, dt=f32)),
                                       z(64, 4, dt=f32))
    with pytest.raises(ValueError):
        gdn.gdn_chunk_bwd(z(1, 8, 1, 64), z(1, 8, 1, 64), z(1, 8, 2, 64), z(1, 8, 2, dt=f32), z(1, 8, 2, dt=f32),
                          z(1, 8, 1, 64))
    with pytest.raises(gdn.GdnError):  # the library's own refusal: a workspace that is too small
        gdn.gdn_gates_bwd(z(4, 8), z(4, 8), z(8, dt=f32), z(8, dt=f32), z(4, 8), z(4, 8),
                          workspace=z(64, dt=torch.uint8))


@gpu
def test_binding_refuses_empty_last_dimensions():
    """ValueError, as for every other shape that does not fit; no rows at all are not refused."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")
    i8, f32 = torch.int8, torch.float32
    ck = lambda *s: (z(*s, 64, dt=i8), z(*s, 0, dt=f32))
    for call in (lambda: gdn.gdn_act_unpack8(*ck(2)),
                 lambda: gdn.gdn_act_unpack8(*ck(0)),
                 lambda: gdn.gdn_act_unpack8(z(2, 0, dt=i8), z(2, 1, dt=f32)),
                 lambda: gdn.gdn_act_pack8(z(2, 0), group=64),
                 lambda: gdn.gdn_act_pack8(z(()), group=64),
                 lambda: gdn.gdn_gated_rmsnorm_bwd(z(2, 0), z(2, 0), z(2, 0), z(0, dt=f32)),
                 lambda: gdn.gdn_gated_rmsnorm_ckpt8(z(2, 0), z(2, 0), z(0, dt=f32)),
                 lambda: gdn.gdn_gates_bwd(z(2, 0), z(2, 0), z(0, dt=f32), z(0, dt=f32), z(2, 0), z(2, 0)),
                 lambda: gdn.gdn_causal_conv1d_silu_bwd(z(1, 0, 64), ck(1, 0), z(64, 4, dt=f32))):
        with pytest.raises(ValueError):
            call()
    assert gdn.gdn_act_unpack8(z(0, 64, dt=i8), z(0, 1, dt=f32)).shape == (0, 64)
    assert gdn.gdn_act_pack8(z(0, 64), group=64)[1].shape == (0, 1)
    assert gdn.gdn_gated_rmsnorm_ckpt8(z(0, 64), z(0, 64), z(64, dt=f32))[0].shape == (0, 64)


@no_gpu
def test_addresses_between_elements_are_refused():
    """Vectors that are read one element at a time have to lie on a multiple of that element."""
    lib = gdn.load()
    gates = lambda **o: lib.gdn_gates_bwd(*[o.get(n, d) for n, d in dict(
        a=at(1), b=at(2), dt=o.get("dt", 0), A=at(3), bi=at(4), dg=at(5), de=at(6), n=64, Hv=8, da=at(7), db=at(8),
        dA=at(9), dbi=at(10), ws=at(11), wsb=BIG, st=None).items()])
    for n, i in dict(a=1, b=2, dg=5, de=6, da=7, db=8).items():
        assert gates(**{n: at(i) + 1}) == E and gates(**{n: at(i) + 2}, dt=1) == E, n
    for n, i in dict(A=3, bi=4, dA=9, dbi=10).items():
        assert gates(**{n: at(i) + 2}) == E, n
    norm = lambda **o: lib.gdn_gated_rmsnorm_bwd(*[o.get(n, d) for n, d in dict(
        dy=at(1), x=at(2), xs=None, z=at(3), zs=None, dt=0, w=at(4), eps=1e-6, n=64, dim=128, dx=at(5), dz=at(6),
        dw=at(7), ws=at(8), wsb=BIG, st=None).items()])
    assert norm(w=at(4) + 2) == E and norm(dw=at(7) + 1) == E
    assert norm(xs=at(9) + 2, zs=at(10)) == E
    assert lib.gdn_gated_rmsnorm_ckpt8(at(1), at(2), 0, at(8) + 2, 1e-6, 64, 128, at(3), at(4), at(5), at(6), at(7),
                                       None) == E
    conv = lambda **o: lib.gdn_causal_conv1d_silu_bwd(*[o.get(n, d) for n, d in dict(
        dy=at(1), x=at(2), xs=None, xg=0, dt=0, w=at(3), bias=at(7), B=1, T=64, C=256, K=4, cu=None, N=1, l2=0,
        group=0, eps=1e-6, h=at(8), dl=at(9), dx=at(4), dw=at(5), db=at(10), dh=at(12), ws=at(6), wsb=BIG,
        st=None).items()])
    for n, i in dict(w=3, bias=7, h=8, dl=9, dw=5, db=10, dh=12).items():
        assert conv(**{n: at(i) + 2}) == E, n
    rule = lambda dt, dg, db: lib.gdn_chunk_bwd(
        at(1), 256, at(2), 256, at(3), 512, at(4), at(5), at(6), dt, 0.1, None, None, None, 1, 1, 64, 2, 4, 128, 128,
        64, at(7), at(8), at(9), dg, db, None, at(64), 1 << 40, None)
    assert rule(0, at(10) + 1, at(11)) == E and rule(0, at(10), at(11) + 1) == E and rule(1, at(10) + 2, at(11)) == E
