"""gdn_chunk_bwd on the tensor-core path: bf16, heads of 128, chunk 64, at least 512 gate values (tokens times
v-heads).  The tolerances are those of test_bwd_rule.py.  Every call's status word is read: a wait in a kernel
that ran out would leave the results in place and only be told there."""
import pytest
import torch

from test_bwd_rule import TC_TOL, call, check, make
from gated_deltanet_fwd_b200 import gdn

gpu = pytest.mark.gpu
D = 128


def workspace(x, lens):
    Hk, Hv = x["q"].shape[1], x["v"].shape[1]
    return torch.empty(gdn.chunk_bwd_workspace_size(torch.bfloat16, len(lens), x["B"], x["T"], Hk, Hv, D, D),
                       dtype=torch.uint8, device="cuda")


def run(x, lens, status=gdn.GDN_OK, **kw):
    assert x["B"] * x["T"] * x["v"].shape[1] >= 512
    ws = workspace(x, lens)
    got = call(x, workspace=ws, **kw)
    assert gdn.workspace_status(ws) == status
    return got


CASES = [
    # lens, packed, Hk, Hv, states, a_mean
    ([512], False, 1, 1, False, 0.0),                                 # the fewest values
    ([1, 0, 2, 63, 64, 65, 0, 1, 128, 129, 0], True, 1, 2, True, -2.0),
    ([300], False, 2, 2, False, -2.0),
    ([171], False, 1, 3, True, -2.0),
    ([130, 130], False, 1, 4, True, -6.0),
    ([257, 3, 500], True, 2, 4, True, -4.0),
    ([2] * 150 + [0] * 120 + [1] * 30, True, 1, 2, False, 0.0),       # more sequences than are ordered by length
    ([65, 1, 200, 94], True, 40, 40, True, -2.0),                     # more (chunk, k-head) items than SMs,
    ([65, 1, 200, 94], True, 40, 80, False, -2.0),                    # one to three v-heads each
    ([65, 1, 130], True, 34, 102, True, -2.0),
    ([64, 64], True, 160, 160, False, -2.0),
]


@gpu
@pytest.mark.parametrize("lens,packed,Hk,Hv,states,a_mean", CASES)
def test_gradients(lens, packed, Hk, Hv, states, a_mean):
    x = make(lens, Hk, Hv, D, D, "bf16", states, packed, a_mean, seed=29)
    check(x, lens, run(x, lens), TC_TOL, D ** -0.5)


@gpu
@pytest.mark.parametrize("T", [511, 512])
def test_both_sides_of_the_smallest_tensor_core_call(T):
    x = make([T], 1, 1, D, D, "bf16", True, seed=31)
    check(x, [T], call(x, scale=0.5), TC_TOL, 0.5)


@gpu
def test_gate_extremes():
    """beta of exactly zero, tiny and one; no decay, and decay that wipes the state out."""
    x = make([300], 1, 2, D, D, "bf16", True, seed=37)
    x["beta"][::5] = 0.0
    x["beta"][1::5] = 1e-12
    x["beta"][2::5] = 1.0
    x["g"][::3] = 0.0
    x["g"][40:42] = -200.0
    x["g"][64] = -200.0
    got = run(x, [300])
    check(x, [300], got, TC_TOL, D ** -0.5)
    assert (got[2].reshape(300, 2, D)[::5] == 0).all()
    assert all(torch.isfinite(t).all() for t in got)


@gpu
def test_first_token_without_a_state_has_no_decay_gradient():
    lens = [200, 1, 64, 35]
    x = make(lens, 1, 2, D, D, "bf16", False, seed=41)
    dg = run(x, lens)[3].reshape(300, 2)
    assert (dg[[0, 200, 201, 265]] == 0).all()
    assert (dg[1:64] != 0).any()


@gpu
def test_strided_inputs_match_dense():
    lens, Hk, Hv = [177, 90], 1, 2
    x = make(lens, Hk, Hv, D, D, "bf16", False, seed=43)
    dense = run(x, lens)
    mix = torch.cat([x["q"].flatten(1), x["k"].flatten(1), x["v"].flatten(1),
                     torch.full((267, 8), float("nan"), dtype=torch.bfloat16)], 1)[None].cuda()
    q = mix[..., :D].unflatten(-1, (Hk, D))
    k = mix[..., D:2 * D].unflatten(-1, (Hk, D))
    v = mix[..., 2 * D:4 * D].unflatten(-1, (Hv, D))
    got = gdn.gdn_chunk_bwd(q, k, v, x["g"][None].cuda(), x["beta"][None].cuda(),
                            x["dout"][None].cuda(), cu_seqlens=x["cu"].cuda())
    for a, b in zip(dense[:5], got[:5]):
        assert torch.equal(a, b)


@gpu
@pytest.mark.parametrize("tail", [1, 60, 200])
def test_tokens_behind_the_last_sequence_stay(tail):
    lens, n = [230, 40], 270
    x = make(lens, 1, 2, D, D, "bf16", False, seed=47)
    want = run(x, lens)
    T = n + tail
    big = {m: torch.full((1, T, *x[m].shape[1:]), float("nan"), dtype=x[m].dtype, device="cuda")
           for m in ("q", "k", "v", "g", "beta", "dout")}
    for m in big:
        big[m][0, :n] = x[m].cuda()
    out = {m: torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda") for m, s in
           dict(dq=(1, T, 1, D), dk=(1, T, 1, D), dv=(1, T, 2, D), dg=(1, T, 2), dbeta=(1, T, 2)).items()}
    gdn.gdn_chunk_bwd(big["q"], big["k"], big["v"], big["g"], big["beta"], big["dout"],
                      cu_seqlens=x["cu"].cuda(), **out)
    for (m, t), w in zip(out.items(), want):
        assert torch.equal(t[:, :n], w), m
        assert (t[:, n:] == 7.0).all(), m


@gpu
@pytest.mark.parametrize("bad", [[0, 130, 20, 300], [0, 130, 260, 301], [-1, 130, 260, 300], [0, 0, 0, -5],
                                 [5, 2, 260, 300]])
def test_malformed_cu_seqlens_is_reported(bad):
    lens = [130, 130, 40]
    x = make(lens, 4, 4, D, D, "bf16", True, seed=53)
    good = run(x, lens)
    ws = workspace(x, lens)
    call(dict(x, cu=torch.tensor(bad, dtype=torch.int32)), workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_ERR_DEVICE_ARG
    again = call(x, workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_OK
    assert all(torch.equal(a, b) for a, b in zip(good, again))


@gpu
def test_bits_graphs_and_streams():
    """The same bits whichever CTA takes which item: again, on two streams at once, in two graphs that share
    a workspace and are replayed one after the other, and on a workspace full of NaN."""
    lens = [150, 20, 64, 1]
    x, y = (make(lens, 40, 80, D, D, "bf16", True, seed=s) for s in (59, 61))
    first, other = run(x, lens), run(y, lens)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, run(x, lens)))
    ws = workspace(x, lens)
    ws.fill_(255)
    assert all(torch.equal(a, b) for a, b in zip(first, call(x, workspace=ws)))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        a1 = call(x)
    with torch.cuda.stream(s2):
        a2 = call(y)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, a1))
    assert all(torch.equal(a, b) for a, b in zip(other, a2))
    cu = x["cu"].cuda()
    graphs, outs = [], []
    for z in (x, y):
        st = {n: (z[n][None] if n not in ("S0", "dST") else z[n]).cuda()
              for n in ("q", "k", "v", "g", "beta", "dout", "S0", "dST")}
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            outs.append(gdn.gdn_chunk_bwd(st["q"], st["k"], st["v"], st["g"], st["beta"], st["dout"],
                                          initial_state=st["S0"], cu_seqlens=cu, dfinal_state=st["dST"],
                                          workspace=ws))
        graphs.append((graph, st))
    for i in (0, 1, 1, 0):
        for t in outs[i]:
            t.zero_()
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert gdn.workspace_status(ws) == gdn.GDN_OK
        assert all(torch.equal(a, b) for a, b in zip((first, other)[i], outs[i]))


@gpu
@pytest.mark.parametrize("dtype,lens", [("f32", [0, 1]), ("f32", [1, 3, 2]), ("f32", [70]), ("bf16", [1] * 300),
                                        ("bf16", [3] * 40 + [70, 66])])
def test_decay_gradients_far_below_the_terms_they_leave(dtype, lens):
    """A decay of e^-15 a token, states on both ends: dg is of that size, millions of times below the products
    k.(U dS) of single tokens, which may therefore not enter its sums and cancel there."""
    x = make(lens, 1, 2, D, D, dtype, True, seed=67)
    x["g"][:] = -15.0 + 0.1 * x["g"].clamp(-10, 0)
    tol = 2e-5 if dtype == "f32" else TC_TOL
    check(x, lens, run(x, lens) if dtype == "bf16" else call(x, 32), tol, D ** -0.5)


@gpu
def test_malformed_entry_met_by_running_blocks():
    """More items than SMs in front of the bad entry: blocks meet it as a later item, and end."""
    lens = [200, 200, 200]
    x = make(lens, 64, 64, D, D, "bf16", False, seed=71)
    good = run(x, lens)
    ws = workspace(x, lens)
    got = call(dict(x, cu=torch.tensor([0, 200, 400, 390], dtype=torch.int32)), workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_ERR_DEVICE_ARG
    assert all(torch.equal(a[:, :400], b[:, :400]) for a, b in zip(good[:5], got[:5]))  # well described
    assert all(torch.equal(a, b) for a, b in zip(good[:5], call(x, workspace=ws)[:5]))
    assert gdn.workspace_status(ws) == gdn.GDN_OK


def many_heads(T, H, a_mean, kind, states, seed):
    """A call of H heads, each with its own q and k: for the kernels the same as H calls of one head."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    unit = lambda t: (t / t.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    x = dict(q=unit(rn(1, T, H, D)), k=unit(rn(1, T, H, D) + (rn(1, 1, H, D) if kind == "alike" else 0.0)),
             v=rn(1, T, H, D).to(torch.bfloat16), dout=rn(1, T, H, D).to(torch.bfloat16))
    A = torch.rand(H, generator=gen, device="cuda") * 15 + 1
    x["g"] = -A * torch.nn.functional.softplus(rn(1, T, H) + a_mean)
    x["beta"] = torch.sigmoid(rn(1, T, H) + (2.0 if kind == "strong" else 0.0))
    x["S0"], x["dST"] = (rn(1, H, D, D) * 0.1 if states else None for _ in range(2))
    return x


def exact_heads(x):
    """All gradients token by token in 64 bits, and the root sum of squares of the products that dg sums."""
    f = torch.float64
    q, k, v, do, beta, decay = (x[n][0].to(f) for n in ("q", "k", "v", "dout", "beta", "g"))
    decay, scale = decay.exp(), D ** -0.5
    T, H = beta.shape
    S = x["S0"][0].to(f) if x["S0"] is not None else torch.zeros(H, D, D, device="cuda", dtype=f)
    dS = x["dST"][0].to(f) if x["dST"] is not None else torch.zeros_like(S)

    def step(S, t):
        E = S * decay[t][:, None, None]
        e = v[t] - (E @ k[t][..., None])[..., 0]
        return E, e, E + (beta[t][:, None] * e)[..., None] * k[t][:, None, :]

    at = []
    for t in range(T):
        at.append(S)
        S = step(S, t)[2]
    out = {n: torch.zeros_like(y) for n, y in dict(dq=q, dk=k, dv=v, dg=beta, dbeta=beta, size=beta).items()}
    for t in reversed(range(T)):
        E, e, S = step(at.pop(), t)
        dS = dS + (scale * do[t])[..., None] * q[t][:, None, :]
        du = (dS @ k[t][..., None])[..., 0]
        u, b = beta[t][:, None] * e, beta[t][:, None] * du
        out["dq"][t] = scale * (do[t][:, None, :] @ S)[:, 0]
        out["dbeta"][t], out["dv"][t] = (du * e).sum(-1), b
        out["dk"][t] = (u[:, None, :] @ dS)[:, 0] - (b[:, None, :] @ E)[:, 0]
        dE = dS - b[..., None] * k[t][:, None, :]
        products = E * dE
        out["dg"][t], out["size"][t] = products.sum((-1, -2)), products.square().sum((-1, -2)).sqrt()
        dS = dE * decay[t][:, None, None]
    return out


def errors_by_head(x, chunk=64):
    """For each output the heads' errors, and their norms; dg's is taken with that of its products."""
    ws = torch.empty(gdn.chunk_bwd_workspace_size(torch.bfloat16, 1, *x["v"].shape[:2], *[x["v"].shape[2]] * 2, D, D,
                                                  chunk), dtype=torch.uint8, device="cuda")
    got = gdn.gdn_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["dout"], initial_state=x["S0"],
                            dfinal_state=x["dST"], chunk=chunk, workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_OK
    want = exact_heads(x)
    heads = lambda y: y.transpose(0, 1).flatten(1).norm(dim=1)
    found = {}
    for n, y in zip(("dq", "dk", "dv", "dg", "dbeta"), got):
        found[n] = heads(y[0].double() - want[n]), heads(want[n]), heads(want["size"]) if n == "dg" else 0.0
    return found


@gpu
@pytest.mark.parametrize("kind", ["random", "strong", "alike"])
@pytest.mark.parametrize("T,H,a_mean,states", [(512, 96, 0.0, False), (520, 64, -6.0, True), (1024, 64, -8.0, False),
                                               (1000, 64, -10.0, False), (1024, 64, -20.0, True),
                                               (2048, 32, -10.0, False)])
def test_errors_of_many_calls(T, H, a_mean, states, kind):
    """What the header says of the tensor-core path, for each of many one-head calls: keys at random, with strong
    writes, and with a direction in common; decays from e^-6 a token to none.

    Rounding to bf16 costs 2^-8 / sqrt(6) = 1.6e-3 of an operand's norm.  There are fifteen such operands (T~, P,
    scale Gamma Q; in either walk the state's copy, X, the update's operand; U, dV, the copies of S and dS, dN, dM:
    two walks share T~) and the output: if an output depends on all of them in full, sqrt(16) * 1.6e-3 = 6.4e-3.
    dg[t] = sum of (state x state gradient): the states are made of the updates' operands and their copies are
    rounded, which is four roundings in full, sqrt(4) * 1.6e-3 = 3.2e-3 of the products' root sum of squares;
    the others take part through half of a state or less (T~, P, U, the copies and X in the walks: eight at 0.8e-3),
    together 3.9e-3.  That is one standard deviation, and with one head that forgets nothing all tokens share
    nearly the same error.  Divided by both norms together, which are alike in the mean, it is 2.8e-3; 1e-2 leaves
    three and a half of those."""
    for n, (err, norm, size) in errors_by_head(many_heads(T, H, a_mean, kind, states, seed=97 + T)).items():
        if n == "dg":
            r = err / (norm * norm + size * size).sqrt()
            print(f"MARGIN {n} {r.max():.2e} of 1.0e-02, of its own norm {(err / norm).max():.2e}")
            assert (r <= 1e-2).all(), (n, r.max().item())
        else:
            r = err / norm
            print(f"MARGIN {n} {r.max():.2e} of 6.5e-03")
            assert (r <= 6.5e-3).all(), (n, r.max().item())


@gpu
@pytest.mark.parametrize("chunk", [16, 32])
def test_shorter_chunks_keep_fp32_inside(chunk):
    """The way out that the header names: each head's outputs lose their own rounding alone."""
    for n, (err, norm, _) in errors_by_head(many_heads(600, 16, -10.0, "random", True, seed=101), chunk).items():
        assert (err <= (2.0 ** -8 + 2e-5) * norm).all(), (n, (err / norm).max().item())
