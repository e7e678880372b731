"""gdn_chunk_bwd against a 64-bit token-by-token reference, against differences of the oracle's forward,
and its conduct: bits, graphs, streams, strides, bad cu_seqlens, tokens behind the last sequence.

Tolerances.
fp32: an output is the end of about ten sums of up to 192 terms, each with a rounding error of about
  sqrt(192) 2^-24 = 8e-7 of its norm, so 8e-6 if all add; F32_TOL = 2e-5.
bf16 in the CUDA-core kernels: fp32 inside, then one rounding, at most 2^-8 of the value: norm-wise
  2^-8 + F32_TOL.
bf16 on tensor cores: every operand is rounded to bf16, an rms error of 2^-8 / sqrt(6) = 1.6e-3 of its
  norm; up to eight rounded operands in a row (state, X', T', U, its scaled copy, dU, dW, dN) and the
  output add in squares to 1.6e-3 * 3 = 4.8e-3: 5e-3, the forward's own tolerance."""
import numpy as np
import pytest
import torch

import bwd_reference as ref
import oracle
from gdn_testutil import rel_l2
from gated_deltanet_fwd_b200 import gdn

gpu = pytest.mark.gpu
F32_TOL = 2e-5
TC_TOL = 5e-3


def make(lens, Hk, Hv, dk, dv, dtype, states, packed=True, a_mean=-2.0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s, std=1.0: torch.randn(*s, generator=gen) * std
    T, N = sum(lens), len(lens)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    x = dict(q=unit(rn(T, Hk, dk)).to(dt), k=unit(rn(T, Hk, dk)).to(dt), v=rn(T, Hv, dv).to(dt),
             dout=rn(T, Hv, dv).to(dt))
    A = torch.rand(Hv, generator=gen) * 15 + 1
    x["g"] = -A * torch.nn.functional.softplus(rn(T, Hv) + a_mean)
    x["beta"] = torch.sigmoid(rn(T, Hv))
    x["S0"] = rn(N, Hv, dv, dk, std=0.1) if states else None
    x["dST"] = rn(N, Hv, dv, dk, std=0.1) if states else None
    x["cu"] = torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32) if packed else None
    x["B"], x["T"] = (1, T) if packed else (N, lens[0])
    return x


def call(x, chunk=64, scale=None, dev="cuda", **kw):
    to = lambda n: x[n].reshape(x["B"], x["T"], *x[n].shape[1:]).to(dev)
    opt = lambda t: None if t is None else t.to(dev)
    return gdn.gdn_chunk_bwd(to("q"), to("k"), to("v"), to("g"), to("beta"), to("dout"), scale=scale,
                             initial_state=opt(x["S0"]), cu_seqlens=opt(x["cu"]),
                             dfinal_state=opt(x["dST"]), chunk=chunk, **kw)


def check(x, lens, got, tol, scale):
    want = ref.rule_grads(x, lens, scale)
    names = ["dq", "dk", "dv", "dg", "dbeta"] + (["dS0"] if x["S0"] is not None else [])
    for n, y in zip(names, got):
        w = want[n].numpy()
        if np.linalg.norm(w) == 0:
            assert not y.numel() or y.abs().max().item() == 0, n
            continue
        r = rel_l2(y.reshape(w.shape), w)
        print(f"MARGIN {n} {r:.2e} of {tol:.1e}")
        assert r <= tol, (n, r)
    return want


CASES = [
    # lens, packed, Hk, Hv, dk, dv, chunk, states
    ([1], False, 1, 1, 16, 16, 16, False),
    ([2, 2], False, 1, 2, 32, 16, 16, True),
    ([17, 1, 0, 33], True, 2, 4, 48, 80, 16, True),
    ([64, 31, 0], True, 1, 3, 128, 128, 32, True),
    ([0, 65, 1, 130], True, 2, 2, 64, 96, 64, True),
    ([100, 100], False, 2, 6, 112, 32, 64, False),
    ([129], False, 1, 1, 128, 128, 64, False),
]


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,packed,Hk,Hv,dk,dv,chunk,states", CASES)
def test_gradients(lens, packed, Hk, Hv, dk, dv, chunk, states, dtype):
    x = make(lens, Hk, Hv, dk, dv, dtype, states, packed)
    tensor_cores = dtype == "bf16" and dk == dv == 128 and chunk == 64
    tol = F32_TOL if dtype == "f32" else TC_TOL if tensor_cores else 2.0 ** -8 + F32_TOL
    check(x, lens, call(x, chunk), tol, dk ** -0.5)


TC_CASES = [
    # lens, packed, Hk, Hv, states, a_mean
    ([1], False, 1, 1, False, 0.0),
    ([1, 0, 2], True, 1, 2, True, -2.0),
    ([63, 64, 65, 0, 1], True, 1, 2, True, -2.0),
    ([200], False, 2, 2, False, 0.0),
    ([130, 130], False, 1, 4, True, -6.0),
    ([257, 3, 500], True, 2, 4, True, -4.0),
    ([96], False, 1, 3, False, -2.0),
]


@gpu
@pytest.mark.parametrize("lens,packed,Hk,Hv,states,a_mean", TC_CASES)
def test_gradients_tensor_core_shape(lens, packed, Hk, Hv, states, a_mean):
    x = make(lens, Hk, Hv, 128, 128, "bf16", states, packed, a_mean, seed=3)
    check(x, lens, call(x), TC_TOL, 128 ** -0.5)


@gpu
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_long_sequence_slow_decay(dtype, d):
    """1500 tokens that hardly decay: gradients that cross many chunks."""
    x = make([1500], 1, 2, d, d, dtype, True, a_mean=-8.0, seed=5)
    check(x, [1500], call(x), F32_TOL if dtype == "f32" else TC_TOL, d ** -0.5)


@gpu
@pytest.mark.parametrize("dtype,d", [("f32", 48), ("bf16", 128)])
def test_gate_extremes(dtype, d):
    """beta of exactly zero, tiny and one; no decay, and decay that wipes the state out."""
    x = make([150], 1, 2, d, d, dtype, True, seed=7)
    x["beta"][::5] = 0.0
    x["beta"][1::5] = 1e-12
    x["beta"][2::5] = 1.0
    x["g"][::3] = 0.0
    x["g"][40:42] = -200.0
    got = call(x)
    check(x, [150], got, F32_TOL if dtype == "f32" else TC_TOL, d ** -0.5)
    dv = got[2].reshape(150, 2, d)
    assert (dv[::5] == 0).all()
    assert all(torch.isfinite(t).all() for t in got)


@gpu
@pytest.mark.parametrize("dtype,d", [("f32", 32), ("bf16", 128)])
def test_against_differences(dtype, d):
    """The change of the loss along a random direction, by central differences of the oracle's forward."""
    lens, Hk, Hv = [70, 1, 40], 1, 2
    x = make(lens, Hk, Hv, d, d, dtype, True, seed=11)
    got = dict(zip(("q", "k", "v", "g", "beta", "S0"), call(x)))
    gen = torch.Generator().manual_seed(1)
    cu = x["cu"].numpy()

    def loss(step):
        y = {n: ref.d64(x[n]) + step * way[n] for n in got}
        o, S = oracle.gated_delta_rule(*(y[n][None].numpy() for n in ("q", "k", "v", "g", "beta")),
                                       d ** -0.5, initial_state=y["S0"].numpy(), cu_seqlens=cu)
        return ((torch.from_numpy(o)[0] * ref.d64(x["dout"])).sum()
                + (torch.from_numpy(S) * ref.d64(x["dST"])).sum()).item()

    for only in list(got):
        # along the gradient itself, where the change is the gradient's norm: no cancellation
        way = {n: torch.zeros_like(ref.d64(x[n])) for n in got}
        w = ref.d64(got[only]).reshape(way[only].shape)
        way[only] = w / w.norm() + 0.1 * torch.randn(w.shape, generator=gen, dtype=ref.D) / w.numel() ** 0.5
        want = (loss(1e-4) - loss(-1e-4)) / 2e-4
        have = (w * way[only]).sum().item()
        # differences: third derivatives times 1e-8 and 1e-16 / 1e-4; the gradient's own error enters once
        assert abs(have - want) <= (1e-4 if dtype == "f32" else 1e-2) * abs(want), (only, have, want)


@gpu
@pytest.mark.parametrize("dtype,dk,dv,chunk", [("f32", 64, 96, 32), ("f32", 128, 128, 64), ("bf16", 48, 32, 16),
                                               ("bf16", 128, 128, 32), ("bf16", 128, 128, 64)])
@pytest.mark.parametrize("packed", [True, False])
def test_first_token_without_a_state_has_no_decay_gradient(dtype, dk, dv, chunk, packed):
    """Exactly zero, also on the CUDA-core path (the last bf16 case has fewer than 512 gate values); not so for
    the first token of a later chunk, nor with a state."""
    lens, Hv = ([100, 1, 0, 64, 35] if packed else [70, 70]), 2
    x = make(lens, 1, Hv, dk, dv, dtype, False, packed, seed=83)
    first = [sum(lens[:n]) for n in range(len(lens)) if lens[n]]
    dg = call(x, chunk)[3].reshape(-1, Hv)
    assert (dg[first] == 0).all()
    assert (dg[1:chunk + 1] != 0).any(1).all()
    x = make(lens, 1, Hv, dk, dv, dtype, True, packed, seed=83)
    assert (call(x, chunk)[3].reshape(-1, Hv)[first] != 0).all()


@gpu
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_strided_inputs_match_dense(dtype, d):
    lens, Hk, Hv = [77, 60], 1, 2
    x = make(lens, Hk, Hv, d, d, dtype, False, seed=13)
    dense = call(x)
    mix = torch.cat([x["q"].flatten(1), x["k"].flatten(1), x["v"].flatten(1),
                     torch.full((137, 8), float("nan"), dtype=x["q"].dtype)], 1)[None].cuda()
    q = mix[..., :Hk * d].unflatten(-1, (Hk, d))
    k = mix[..., Hk * d:2 * Hk * d].unflatten(-1, (Hk, d))
    v = mix[..., 2 * Hk * d:2 * Hk * d + Hv * d].unflatten(-1, (Hv, d))
    got = gdn.gdn_chunk_bwd(q, k, v, x["g"][None].cuda(), x["beta"][None].cuda(),
                            x["dout"][None].cuda(), cu_seqlens=x["cu"].cuda())
    for a, b in zip(dense[:5], got[:5]):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("B,T,Hk", [(3, 1, 2), (1, 1, 1), (300, 1, 1), (2, 5, 1)])
@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128)])
def test_strided_single_tokens(dtype, d, B, T, Hk):
    """Slices of [q | k | v] with one token a sequence: the tokens' distance is the sequences'."""
    Hv = 2 * Hk
    x = make([T] * B, Hk, Hv, d, d, dtype, True, packed=False, seed=15)
    mix = torch.cat([x["q"].flatten(1), x["k"].flatten(1), x["v"].flatten(1)], 1).view(B, T, -1).cuda()
    q, k, v = (t.unflatten(-1, (-1, d)) for t in mix.split([Hk * d, Hk * d, Hv * d], -1))
    g, beta, do = (x[n].view(B, T, *x[n].shape[1:]).cuda() for n in ("g", "beta", "dout"))
    S0, dST = x["S0"].cuda(), x["dST"].cuda()
    got = gdn.gdn_chunk_bwd(q, k, v, g, beta, do, initial_state=S0, dfinal_state=dST)
    assert all(torch.equal(a, b) for a, b in zip(call(x), got))
    one = gdn.gdn_chunk_fwd(q, k, v, g, beta, initial_state=S0)
    two = gdn.gdn_chunk_fwd(q.contiguous(), k.contiguous(), v.contiguous(), g, beta, initial_state=S0)
    assert all(torch.equal(a, b) for a, b in zip(one, two))


@gpu
@pytest.mark.parametrize("dtype,d,chunk", [("f32", 64, 32), ("bf16", 128, 64)])
def test_bits_graph_and_streams(dtype, d, chunk):
    """Twice the same bits; two calls at once on two streams; captured, and replayed on new inputs."""
    lens = [150, 20]
    x, y = (make(lens, 2, 4, d, d, dtype, True, seed=s) for s in (17, 18))
    first, other = call(x, chunk), call(y, chunk)
    for a, b in zip(first, call(x, chunk)):
        assert torch.equal(a, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        a1 = call(x, chunk)
    with torch.cuda.stream(s2):
        a2 = call(y, chunk)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, a1))
    assert all(torch.equal(a, b) for a, b in zip(other, a2))
    names = ("q", "k", "v", "g", "beta", "dout", "S0", "dST")
    st = {n: (x[n][None] if n not in ("S0", "dST") else x[n]).cuda() for n in names}
    cu = x["cu"].cuda()

    def step():
        return gdn.gdn_chunk_bwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["dout"],
                                 initial_state=st["S0"], cu_seqlens=cu, dfinal_state=st["dST"],
                                 chunk=chunk)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for src, want in ((y, other), (x, first)):
        for n in names:
            st[n].copy_(src[n][None] if n not in ("S0", "dST") else src[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))


@gpu
@pytest.mark.parametrize("dtype,d", [("f32", 32), ("bf16", 128)])
def test_tokens_behind_the_last_sequence_stay(dtype, d):
    lens, T = [70, 5], 100
    x = make(lens, 1, 2, d, d, dtype, False, seed=19)
    want = call(x)
    big = {n: torch.full((1, T, *x[n].shape[1:]), float("nan"), dtype=x[n].dtype, device="cuda")
           for n in ("q", "k", "v", "g", "beta", "dout")}
    for n in big:
        big[n][0, :75] = x[n].cuda()
    dt = x["q"].dtype
    out = {n: torch.full(s, 7.0, dtype=dt, device="cuda") for n, s in
           dict(dq=(1, T, 1, d), dk=(1, T, 1, d), dv=(1, T, 2, d), dg=(1, T, 2), dbeta=(1, T, 2)).items()}
    gdn.gdn_chunk_bwd(big["q"], big["k"], big["v"], big["g"], big["beta"], big["dout"],
                      cu_seqlens=x["cu"].cuda(), **out)
    for (n, t), w in zip(out.items(), want):
        assert torch.equal(t[:, :75], w), n
        assert (t[:, 75:] == 7.0).all(), n


@gpu
@pytest.mark.parametrize("dtype,d", [("f32", 32), ("bf16", 128)])
@pytest.mark.parametrize("bad", [[0, 30, 20, 75], [0, 30, 60, 80], [-1, 30, 60, 75]])
def test_malformed_cu_seqlens_is_reported(dtype, d, bad):
    x = make([30, 30, 15], 1, 2, d, d, dtype, False, seed=23)
    good = call(x)
    ws = torch.empty(gdn.chunk_bwd_workspace_size(x["q"].dtype, 3, 1, 75, 1, 2, d, d),
                     dtype=torch.uint8, device="cuda")
    call(dict(x, cu=torch.tensor(bad, dtype=torch.int32)), workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_ERR_DEVICE_ARG
    again = call(x, workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_OK
    assert all(torch.equal(a, b) for a, b in zip(good[:5], again[:5]))


@gpu
@pytest.mark.parametrize("dtype,d,chunk", [("f32", 32, 16), ("bf16", 128, 64)])
def test_many_sequences(dtype, d, chunk):
    """Several rounds of the warps' searches in cu_seqlens (32 and 128 entries each): each sequence's gradients have
    the bits of a call of its neighbours alone, and an entry that is malformed stops what lies behind it."""
    gen = torch.Generator().manual_seed(107)
    lens = [int(n) for n in torch.randint(0, 4, (700,), generator=gen)]
    lens[130], lens[300], lens[699] = 70, 0, 33
    x = make(lens, 1, 2, d, d, dtype, True, seed=109)
    got = call(x, chunk)
    check(x, lens, got, F32_TOL if dtype == "f32" else TC_TOL, d ** -0.5)
    at = np.cumsum([0] + lens)
    for lo, hi in ((0, 500), (100, 420), (290, 700)):  # bf16: enough gate values for the same path
        part = {n: x[n][at[lo]:at[hi]] for n in ("q", "k", "v", "g", "beta", "dout")}
        part.update(S0=x["S0"][lo:hi], dST=x["dST"][lo:hi], B=1, T=int(at[hi] - at[lo]),
                    cu=torch.tensor(at[lo:hi + 1] - at[lo], dtype=torch.int32))
        for a, b in zip(call(part, chunk)[:5], got[:5]):
            assert torch.equal(a, b[:, at[lo]:at[hi]])
    dt = x["q"].dtype
    ws = torch.empty(gdn.chunk_bwd_workspace_size(dt, 700, 1, x["T"], 1, 2, d, d, chunk), dtype=torch.uint8,
                     device="cuda")
    for bad in (1, 31, 32, 33, 128, 129, 411, 700):
        cu = x["cu"].clone()
        cu[bad] = -1
        part = call(dict(x, cu=cu), chunk, workspace=ws)
        assert gdn.workspace_status(ws) == gdn.GDN_ERR_DEVICE_ARG
        assert all(torch.equal(a[:, :at[bad - 1]], b[:, :at[bad - 1]]) for a, b in zip(part[:5], got[:5])), bad


@gpu
@pytest.mark.parametrize("dtype,d", [("f32", 32), ("bf16", 128)])
def test_no_tokens_passes_the_state_gradient(dtype, d):
    x = make([0, 0], 1, 2, d, d, dtype, True)
    got = call(x)
    assert torch.equal(got[5].cpu(), x["dST"])
    z = dict(x, dST=None)
    assert (call(z)[5] == 0).all()


# ---------------------------------------------------------------------------- refusals (CPU) ----

P = 0x7f0000000000


def _lib():
    return gdn.load()


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: only without a GPU")


@no_gpu
def test_refusals():
    f = _lib().gdn_chunk_bwd
    big = 1 << 40
    E, U = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED
    at = lambda i: P + (i << 32)

    def c(q=at(1), qs=256, k=at(2), ks=256, v=at(3), vs=512, g=at(4), b=at(5), do=at(6), dt=0, scale=0.1,
          s0=None, ds=None, cu=None, N=1, B=1, T=64, Hk=2, Hv=4, dk=128, dv=128, chunk=64, dq=at(7),
          dkk=at(8), dvv=at(9), dg=at(10), db=at(11), d0=None, ws=at(64), wsb=big):
        return f(q, qs, k, ks, v, vs, g, b, do, dt, scale, s0, ds, cu, N, B, T, Hk, Hv, dk, dv, chunk,
                 dq, dkk, dvv, dg, db, d0, ws, wsb, None)

    assert c(dt=9) == E
    assert c(Hv=3) == E
    assert c(N=2) == E
    assert c(cu=at(12), B=2, N=2) == E
    assert c(scale=float("nan")) == E
    assert c(dk=24, qs=512, ks=512) == U
    assert c(dv=144, vs=1024) == U
    assert c(chunk=48) == U
    assert c(qs=128) == E and c(ks=260) == E and c(vs=511) == E
    assert c(ws=None) == E and c(ws=at(64) + 16) == E and c(wsb=4096) == E
    for n in ("q", "k", "v", "g", "b", "do", "dq", "dkk", "dvv", "dg", "db"):
        assert c(**{n: None}) == E, n
    for n, i in dict(q=1, k=2, v=3, g=4, b=5, do=6, dq=7, dkk=8, dvv=9).items():
        assert c(**{n: at(i) + 4}) == E, n
    assert c(s0=at(13) + 4) == E and c(ds=at(13) + 4) == E and c(d0=at(13) + 4) == E
    assert c(cu=at(13) + 2) == E
    assert c(dvv=at(6)) == E              # dv over dout
    assert c(dkk=at(7)) == E              # dk over dq
    assert c(d0=at(13), ds=at(13)) == E   # state gradients over one another
    assert c(N=0, B=0) == gdn.GDN_OK


def test_workspace_size_grows_and_is_aligned():
    f = lambda T, **k: gdn.chunk_bwd_workspace_size(k.get("dt", torch.bfloat16), 1, 1, T, 2, 4, k.get("d", 128),
                                                    128, 64)
    assert f(64) % 256 == 0 and f(64) < f(640) < f(6400)
    assert f(0) >= 256
    assert f(1 << 20) > 1 << 32  # past 32 bits


def test_reference_matches_differences_of_the_oracle():
    """The reference's gradients against the oracle's forward, which shares no code with it."""
    lens = [5, 0, 3]
    x = make(lens, 1, 2, 16, 16, "f32", True, seed=2)
    grads = ref.rule_grads(x, lens, 0.25)
    gen = torch.Generator().manual_seed(0)
    for n in ("q", "k", "v", "g", "beta", "S0"):
        way = torch.randn(x[n].shape, generator=gen, dtype=ref.D)

        def loss(step):
            y = {m: ref.d64(x[m]) for m in ("q", "k", "v", "g", "beta", "S0")}
            y[n] = y[n] + step * way
            o, S = oracle.gated_delta_rule(*(y[m][None].numpy() for m in ("q", "k", "v", "g", "beta")), 0.25,
                                           initial_state=y["S0"].numpy(), cu_seqlens=x["cu"].numpy())
            return (torch.from_numpy(o)[0] * ref.d64(x["dout"])).sum().item() + \
                (torch.from_numpy(S) * ref.d64(x["dST"])).sum().item()

        want = (loss(1e-5) - loss(-1e-5)) / 2e-5
        assert abs((grads["d" + n] * way).sum().item() - want) <= 1e-7 * max(1.0, abs(want)), n
