"""Cases that measure the training operators of the gated delta rule layer core.

Five operators, each reached through the calls of ``gated_deltanet_fwd_b200.gdn``:

  * ``rule``   gdn_chunk_bwd: gradients of the chunked gated delta rule
  * ``gates``  gdn_gates_bwd: gradients of the two gates, with the sums over tokens for A_log, dt_bias
  * ``norm``   gdn_gated_rmsnorm_bwd: gradients of the gated RMSNorm
  * ``conv``   gdn_causal_conv1d_silu_bwd: gradients of conv + SiLU + q/k L2 norm
  * ``ckpt``   8-bit activation checkpoints: gdn_act_pack8 / gdn_act_unpack8, the norm that writes its
               checkpoint as it runs (gdn_gated_rmsnorm_ckpt8), and the backward passes that read them

Where ``own`` is false ``run`` computes the same in plain torch operations, in 32 bits (64 for the
triangular inverse and for sums over all tokens), rounded once at the end.

An 8-bit checkpoint holds, per group of consecutive channels with largest magnitude m, the codes
rint(x * fl(127 / m)) (half to even, of the exact product) and the scale fl(m / 127); a code stands
for code * scale.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
L2_EPS = 1e-6
NORM_EPS = 1e-6
C = 64  # chunk length of the plain form of the rule


def _dt(name):
    return {BF16: torch.bfloat16, F32: torch.float32}[name]


# ------------------------------------------------------------------------------- cases ------

def listed():
    return [
        # one short odd sequence on two k-heads: the call's latency
        dict(name="rule_short", op="rule", dtype=BF16, lens="257", packed=False, Hk=2, Hv=4, dk=128,
             dv=128, chunk=64, states=False, a_mean=0.0),
        # one training sequence at the layer's 16 / 32 heads
        dict(name="rule_4k", op="rule", dtype=BF16, lens="4096", packed=False, Hk=16, Hv=32, dk=128,
             dv=128, chunk=64, states=False, a_mean=0.0),
        # four documents packed into one row of 32768 tokens
        dict(name="rule_varlen_32k", op="rule", dtype=BF16, lens="16384,8192,6144,2048", packed=True,
             Hk=16, Hv=32, dk=128, dv=128, chunk=64, states=False, a_mean=0.0),
        # all-fp32 mode with other head sizes, ragged lengths, state and state gradient carried in
        dict(name="rule_f32", op="rule", dtype=F32, lens="700,1,0,333", packed=True, Hk=2, Hv=4,
             dk=64, dv=96, chunk=32, states=True, a_mean=-4.0),
        # the gates of 32768 tokens at 32 heads
        dict(name="gates_32k", op="gates", dtype=BF16, tokens=32768, Hv=32),
        # a few tokens, odd head count, fp32
        dict(name="gates_f32", op="gates", dtype=F32, tokens=1001, Hv=6),
        # the output norm of 32768 tokens at 32 heads
        dict(name="norm_32k", op="norm", dtype=BF16, rows=32768 * 32, dim=128),
        # a small fp32 norm over heads of 64
        dict(name="norm_f32", op="norm", dtype=F32, rows=4999, dim=64),
        # the layer core's conv on two sequences of 16384, q and k heads normalised
        dict(name="conv_2x16k", op="conv", dtype=BF16, lens="16384,16384", packed=False, C=8192,
             K=4, n_l2=4096, group=128, bias=False, states=False, ckpt=False),
        # packed documents, history carried in, the input kept as an 8-bit checkpoint
        dict(name="conv_varlen_ckpt8", op="conv", dtype=BF16, lens="2047,1,0,1500,548", packed=True,
             C=2048, K=4, n_l2=1024, group=128, bias=True, states=True, ckpt=True),
        # the conv's input of 16384 tokens written to and read back from 8 bits
        dict(name="ckpt_mix_16k", op="ckpt", form="pack", dtype=BF16, rows=16384, dim=8192,
             group=128),
        # norm that writes its checkpoint, then its backward from the checkpoint
        dict(name="ckpt_norm_4k", op="ckpt", form="norm", dtype=BF16, rows=4096 * 32, dim=128,
             group=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cut(rng, total, n):
    """n lengths (zeros and ones among them) that add up to `total`."""
    at = sorted(rng.randrange(total + 1) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + at, at + [total])]


def draw(rng):
    op = rng.choice(["rule", "rule", "gates", "norm", "conv", "ckpt"])
    if op == "rule":
        if rng.random() < 0.65:  # the layer's shape
            Hk = rng.choice([1, 2, 4, 8, 16])
            # training sequences start from a zero state; carried states are drawn in fp32 below
            c = dict(op=op, dtype=BF16, Hk=Hk, Hv=Hk * rng.choice([1, 2, 2, 4] if Hk < 16 else [1, 2]),
                     dk=128, dv=128, chunk=64, states=False)
            total = _log_int(rng, 1, 16384)
        else:  # every other supported shape
            Hk = rng.choice([1, 2, 3])
            dtype = rng.choice([F32, F32, BF16])
            c = dict(op=op, dtype=dtype, Hk=Hk, Hv=Hk * rng.choice([1, 2, 3]),
                     dk=16 * rng.randint(1, 8), dv=16 * rng.randint(1, 8), chunk=rng.choice([16, 32, 64]),
                     states=dtype == F32 and rng.random() < 0.7)
            total = _log_int(rng, 1, 2048)
        c["packed"] = rng.random() < 0.6
        n = rng.randint(1, 6)
        lens = _cut(rng, total, n) if c["packed"] else [max(1, total // n)] * n
        c["lens"] = ",".join(map(str, lens))
        c["a_mean"] = rng.choice([0.0, -2.0, -4.0, -6.0])
        return c
    if op == "gates":
        return dict(op=op, dtype=rng.choice([BF16, F32]), tokens=_log_int(rng, 1, 32768), Hv=rng.randint(1, 64))
    if op == "norm":
        return dict(op=op, dtype=rng.choice([BF16, F32]), rows=_log_int(rng, 1, 500000),
                    dim=rng.choice([8, 16, 32, 64, 128, 256]))
    if op == "conv":
        group = rng.choice([0, 32, 64, 128, 256])
        Cn = 256 * rng.randint(1, 16) if group else 8 * rng.randint(1, 512)
        total = _log_int(rng, 1, 8192)
        packed = rng.random() < 0.6
        n = rng.randint(1, 5)
        lens = _cut(rng, total, n) if packed else [max(1, total // n)] * n
        ckpt = group > 0 and rng.random() < 0.4
        return dict(op=op, dtype=rng.choice([BF16, F32]), lens=",".join(map(str, lens)), packed=packed, C=Cn,
                    K=rng.randint(1, 8), n_l2=group * rng.randint(0, Cn // group) if group else 0,
                    group=group, bias=rng.random() < 0.5, states=rng.random() < 0.5, ckpt=ckpt)
    if rng.random() < 0.5:
        group = rng.choice([32, 64, 128, 256])
        return dict(op=op, form="pack", dtype=rng.choice([BF16, F32]), rows=_log_int(rng, 1, 16384),
                    dim=group * rng.randint(1, 2048 // group), group=group)
    dim = rng.choice([32, 64, 128, 256])
    return dict(op=op, form="norm", dtype=rng.choice([BF16, F32]), rows=_log_int(rng, 1, 131072), dim=dim,
                group=dim)


def _lens(case):
    return [int(x) for x in case["lens"].split(",")]


# ------------------------------------------------------------------------------ inputs ------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def randn(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=gen, device=dev) * std + mean

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    s = dict(case=case)
    dt = _dt(case["dtype"])
    if case["op"] == "rule":
        lens, Hk, Hv, dk, dv = _lens(case), case["Hk"], case["Hv"], case["dk"], case["dv"]
        N = len(lens)
        B, T = (1, sum(lens)) if case["packed"] else (N, lens[0])
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
        s["q"] = unit(randn(B, T, Hk, dk)).to(dt)
        s["k"] = unit(randn(B, T, Hk, dk)).to(dt)
        s["v"] = randn(B, T, Hv, dv).to(dt)
        s["dout"] = randn(B, T, Hv, dv).to(dt)
        A = rand(Hv) * 15.0 + 1.0
        s["g"] = -A * torch.nn.functional.softplus(randn(B, T, Hv, mean=case["a_mean"]) + randn(Hv, std=0.1))
        s["beta"] = torch.sigmoid(randn(B, T, Hv))
        s["cu"] = None
        if case["packed"]:
            s["cu"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32, device=dev)
        s["S0"] = randn(N, Hv, dv, dk, std=0.02) if case["states"] else None
        s["dST"] = randn(N, Hv, dv, dk, std=0.02) if case["states"] else None
    elif case["op"] == "gates":
        n, Hv = case["tokens"], case["Hv"]
        s["a"], s["b"] = randn(n, Hv).to(dt), randn(n, Hv).to(dt)
        s["A_log"], s["dt_bias"] = torch.log(rand(Hv) * 15.0 + 1.0), randn(Hv, std=0.1)
        s["dg"], s["dbeta"] = randn(n, Hv).to(dt), randn(n, Hv).to(dt)
    elif case["op"] == "norm" or case.get("form") == "norm":
        r, d = case["rows"], case["dim"]
        # the rule's outputs are small; the norm rescales each row
        s["x"], s["z"], s["dy"] = randn(r, d, std=0.05).to(dt), randn(r, d).to(dt), randn(r, d).to(dt)
        s["w"] = randn(d, std=0.02)
    elif case["op"] == "conv":
        lens, Cn, K = _lens(case), case["C"], case["K"]
        N = len(lens)
        B, T = (1, sum(lens)) if case["packed"] else (N, lens[0])
        s["x"], s["dy"] = randn(B, T, Cn).to(dt), randn(B, T, Cn).to(dt)
        s["w"] = (rand(Cn, K) * 2.0 - 1.0) / math.sqrt(K)
        s["bias"] = randn(Cn, std=0.1) if case["bias"] else None
        s["cu"] = None
        if case["packed"]:
            s["cu"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32, device=dev)
        states = case["states"] and K > 1
        s["cs_in"] = randn(N, Cn, K - 1) if states else None
        s["dcs_out"] = randn(N, Cn, K - 1) if states else None
        if case["ckpt"]:
            s["x"] = _pack8(s["x"], case["group"])
    else:
        s["x"] = randn(case["rows"], case["dim"]).to(dt)
    return s


# --------------------------------------------------------------------------------- run ------

def run(s):
    case = s["case"]
    if own:
        from gated_deltanet_fwd_b200 import gdn
        if case["op"] == "rule":
            dq, dk, dv, dg, dbeta, dS0 = gdn.gdn_chunk_bwd(
                s["q"], s["k"], s["v"], s["g"], s["beta"], s["dout"], initial_state=s["S0"],
                cu_seqlens=s["cu"], dfinal_state=s["dST"], chunk=case["chunk"])
            out = dict(dq=dq, dk=dk, dv=dv, dg=dg, dbeta=dbeta)
            return dict(out, dS0=dS0) if case["states"] else out
        if case["op"] == "gates":
            da, db, dA, ddt = gdn.gdn_gates_bwd(s["a"], s["b"], s["A_log"], s["dt_bias"], s["dg"], s["dbeta"])
            return dict(da=da, db=db, dA_log=dA, ddt_bias=ddt)
        if case["op"] == "norm":
            dx, dz, dw = gdn.gdn_gated_rmsnorm_bwd(s["dy"], s["x"], s["z"], s["w"], eps=NORM_EPS)
            return dict(dx=dx, dz=dz, dw=dw)
        if case["op"] == "conv":
            dx, dw, dbias, dcs = gdn.gdn_causal_conv1d_silu_bwd(
                s["dy"], s["x"], s["w"], s["bias"], cu_seqlens=s["cu"], n_l2norm_ch=case["n_l2"],
                l2norm_group=case["group"], l2_eps=L2_EPS, conv_state_in=s["cs_in"],
                dconv_state_out=s["dcs_out"])
            return {k: v for k, v in dict(dx=dx, dw=dw, dbias=dbias, dcs=dcs).items() if v is not None}
        if case["form"] == "pack":
            codes, scales = gdn.gdn_act_pack8(s["x"], group=case["group"])
            return dict(x=gdn.gdn_act_unpack8(codes, scales, dtype=s["x"].dtype), scales=scales)
        y, x8, z8 = gdn.gdn_gated_rmsnorm_ckpt8(s["x"], s["z"], s["w"], eps=NORM_EPS)
        dx, dz, dw = gdn.gdn_gated_rmsnorm_bwd(s["dy"], x8, z8, s["w"], eps=NORM_EPS)
        return dict(y=y, dx=dx, dz=dz, dw=dw)
    if case["op"] == "rule":
        return _rule_plain(s)
    if case["op"] == "gates":
        return _gates_plain(s)
    if case["op"] == "norm":
        return _norm_bwd_plain(s["dy"], s["x"].float(), s["z"].float(), s["w"])
    if case["op"] == "conv":
        x = _unpack8(*s["x"]) if case["ckpt"] else s["x"].float()
        return _conv_plain(s, x)
    if case["form"] == "pack":
        codes, scales = _pack8(s["x"], case["group"])
        return dict(x=_unpack8(codes, scales).to(s["x"].dtype), scales=scales)
    x, z, w = s["x"].float(), s["z"].float(), s["w"]
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * (1.0 + w) * (z * torch.sigmoid(z))
    x8, z8 = _pack8(s["x"], case["dim"]), _pack8(s["z"], case["dim"])
    return dict(_norm_bwd_plain(s["dy"], _unpack8(*x8), _unpack8(*z8), w), y=y.to(s["x"].dtype))


def _pack8(x, group):
    """Codes (int8, x's shape) and scales (fp32, one per group of channels)."""
    xg = x.float().unflatten(-1, (-1, group))
    m = xg.abs().amax(-1, keepdim=True)
    top = torch.full_like(m, 127.0)
    inv = torch.where(m > 0, top / m, 0.0)
    codes = torch.round(xg.double() * inv.double()).to(torch.int8)  # the exact product, half to even
    return codes.flatten(-2), (m / top).squeeze(-1)


def _unpack8(codes, scales):
    group = codes.shape[-1] // scales.shape[-1]
    return (codes.float().unflatten(-1, (-1, group)) * scales.unsqueeze(-1)).flatten(-2)


def _gates_plain(s):
    a, b, dg, dbeta = (s[n].float() for n in ("a", "b", "dg", "dbeta"))
    u = a + s["dt_bias"]
    A = torch.exp(s["A_log"])
    sp = torch.clamp_min(u, 0.0) + torch.log1p(torch.exp(-torch.abs(u)))
    da = -dg * A * torch.sigmoid(u)
    beta = torch.sigmoid(b)
    db = dbeta * beta * (1.0 - beta)
    dt = s["a"].dtype
    dA = -(dg.double() * sp).sum(0) * A
    return dict(da=da.to(dt), db=db.to(dt), dA_log=dA.float(), ddt_bias=da.sum(0, dtype=torch.float64).float())


def _norm_bwd_plain(dy, x, z, w):
    dt, dy = dy.dtype, dy.float()
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS)
    xn, sg = x * inv, torch.sigmoid(z)
    silu = z * sg
    t = dy * (1.0 + w) * silu
    dx = inv * (t - xn * (t * xn).mean(-1, keepdim=True))
    dz = dy * xn * (1.0 + w) * sg * (1.0 + z * (1.0 - sg))
    dw = (dy * xn * silu).sum(0, dtype=torch.float64)
    return dict(dx=dx.to(dt), dz=dz.to(dt), dw=dw.float())


def _places(lens, dev):
    """For each token of the packed order: its sequence, its place in it, and that sequence's length."""
    n = torch.tensor(lens, device=dev)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), n)
    first = torch.cumsum(n, 0) - n
    return seq, torch.arange(sum(lens), device=dev) - first[seq], n[seq], first, n


def _conv_plain(s, x):
    case = s["case"]
    K, Cn, dt = case["K"], case["C"], s["dy"].dtype
    dev = s["dy"].device
    x, dy, w = x.reshape(-1, Cn), s["dy"].float().reshape(-1, Cn), s["w"]
    T = x.shape[0]
    seq, place, length, first, n = _places(_lens(case), dev)
    tap = torch.arange(K, device=dev)
    # inputs of every tap: in the sequence, from its history, or zero
    at = place[:, None] - (K - 1) + tap  # [T, K]
    tok = torch.arange(T, device=dev)[:, None] - (K - 1) + tap
    xw = x[tok.clamp(0, T - 1)] * (at >= 0)[..., None]  # [T, K, C]
    if s["cs_in"] is not None:
        hist = s["cs_in"].permute(0, 2, 1)  # [N, K-1, C]
        old = (at + (K - 1)).clamp(0, K - 2)
        xw = torch.where((at >= 0)[..., None], xw, hist[seq[:, None], old])
    pre = (xw * w.t()).sum(1)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    sg = torch.sigmoid(pre)
    act = pre * sg
    ds = dy
    if case["n_l2"]:
        m = case["n_l2"]
        a, d = (v[:, :m].unflatten(-1, (-1, case["group"])) for v in (act, dy))
        rn = torch.rsqrt((a * a).sum(-1, keepdim=True) + L2_EPS)
        ds = torch.cat([(rn * d - a * rn ** 3 * (a * d).sum(-1, keepdim=True)).flatten(-2), dy[:, m:]], -1)
    dpre = ds * sg * (1.0 + pre * (1.0 - sg))
    ahead = (K - 1) - tap  # token t reaches the output `ahead` later through each tap
    inside = place[:, None] + ahead < length[:, None]
    dx = ((dpre[(torch.arange(T, device=dev)[:, None] + ahead).clamp(0, T - 1)] * inside[..., None]) * w.t()).sum(1)
    out = dict(dw=(dpre[:, None] * xw).sum(0, dtype=torch.float64).t().float().contiguous())
    if s["bias"] is not None:
        out["dbias"] = dpre.sum(0, dtype=torch.float64).float()
    if s["cs_in"] is not None:
        # history place j feeds output p through tap j - p; the history left behind is the last K-1
        # of (history in, inputs)
        j = torch.arange(K - 1, device=dev)
        p = torch.arange(K - 1, device=dev)
        ok = (p[None, :] <= j[:, None])[None] & (p[None, None, :] < n[:, None, None])  # [N, j, p]
        src = (first[:, None, None] + p).clamp(0, max(T - 1, 0)).expand(-1, K - 1, -1)
        wt = w.t()[(j[:, None] - p[None, :]).clamp(0, K - 1)]  # [j, p, C]
        dcs = (dpre[src] * ok[..., None] * wt).sum(2) if T else torch.zeros(len(n), K - 1, Cn, device=dev)
        dout = s["dcs_out"].permute(0, 2, 1)  # [N, K-1, C]
        back = j[None] - n[:, None]  # place j of the old history is place j - n of the new one
        dcs = dcs + dout[torch.arange(len(n), device=dev)[:, None], back.clamp(0)] * (back >= 0)[..., None]
        new = place - length + (K - 1)  # place of a token in the history left behind
        dx = dx + torch.where((new >= 0)[:, None], dout[seq, new.clamp(0)], 0.0)
        out["dcs"] = dcs.permute(0, 2, 1).contiguous()
    return dict(out, dx=dx.to(dt).reshape(s["dy"].shape))


def _rule_plain(s):
    """Chunks of 64 over sequences padded to the longest; a pass forward over the chunks for the states, one
    back for their gradients, everything else for all chunks at once."""
    case = s["case"]
    lens, Hk, Hv, dk, dv = _lens(case), case["Hk"], case["Hv"], case["dk"], case["dv"]
    N, G, dev, dt = len(lens), Hv // Hk, s["q"].device, s["q"].dtype
    n_ch = max(1, -(-max(lens) // C))
    seq, place, _, _, _ = _places(lens, dev)
    scale = dk ** -0.5

    def pad(x, H):  # [.., H, d] packed -> [N * H, n_ch, C, d]
        x = x.reshape(-1, H, x.numel() // max(1, x.shape[0] * x.shape[1] * H) if x.dim() == 4 else 1).float()
        y = torch.zeros(N, n_ch * C, H, x.shape[-1], device=dev)
        y[seq, place] = x
        return y.permute(0, 2, 1, 3).reshape(N * H, n_ch, C, -1)

    def unpad(y, H):
        y = y.reshape(N, H, n_ch * C, -1).permute(0, 2, 1, 3)[seq, place]
        return y.to(dt)

    share = lambda x: x.reshape(N, Hk, 1, n_ch, C, -1).expand(-1, -1, G, -1, -1, -1).reshape(N * Hv, n_ch, C, -1)  # noqa: E731
    q, k = share(pad(s["q"], Hk)), share(pad(s["k"], Hk))
    v, do = pad(s["v"], Hv), pad(s["dout"], Hv) * scale
    g, beta = pad(s["g"], Hv), pad(s["beta"], Hv)
    gam = torch.cumsum(g.double(), 2)  # [NH, n_ch, C, 1]
    low = torch.ones(C, C, device=dev, dtype=torch.bool).tril()
    E = torch.where(low, (gam - gam.mT).clamp(max=0.0).exp(), 0.0).float()
    Gam, d = gam.exp().float(), (gam[:, :, -1:] - gam).exp().float()
    last = Gam[:, :, -1:]  # [NH, n_ch, 1, 1]
    Es = E.tril(-1)
    A = (beta * Es * (k @ k.mT)).double()
    Tm = torch.eye(C, device=dev, dtype=torch.float64) - A  # (I + A)^-1 = (I - A)(I + A^2)(I + A^4) ...
    for _ in range(5):
        A = A @ A
        Tm = Tm + Tm @ A
    Tm = (Tm * beta.double().mT).float()
    P = E * (q @ k.mT)
    S = s["S0"].reshape(N * Hv, dv, dk) if s["S0"] is not None else torch.zeros(N * Hv, dv, dk, device=dev)
    dS = s["dST"].reshape(N * Hv, dv, dk) if s["dST"] is not None else torch.zeros(N * Hv, dv, dk, device=dev)
    Ss, Us, dSs, dWs = [], [], [], []
    for c in range(n_ch):
        Ss.append(S)
        U = Tm[:, c] @ (v[:, c] - Gam[:, c] * (k[:, c] @ S.mT))
        Us.append(U)
        S = last[:, c] * S + (d[:, c] * U).mT @ k[:, c]
    for c in reversed(range(n_ch)):
        dSs.append(dS)
        dW = Tm[:, c].mT @ (P[:, c].mT @ do[:, c] + d[:, c] * (k[:, c] @ dS.mT))
        dWs.append(dW)
        dS = last[:, c] * dS + (Gam[:, c] * do[:, c]).mT @ q[:, c] - (Gam[:, c] * dW).mT @ k[:, c]
    S, U = torch.stack(Ss, 1), torch.stack(Us, 1)
    del Ss, Us, A, Tm
    dSc, dW = torch.stack(dSs[::-1], 1), torch.stack(dWs[::-1], 1)
    del dSs, dWs
    kk = Es * (k @ k.mT)
    err = v - Gam * (k @ S.mT) - kk @ U  # v_t - S_t-1 k_t e^g_t
    dR = P.mT @ do + d * (k @ dSc.mT) - kk.mT @ dW
    dbeta = (dR * err).sum(-1, keepdim=True)
    # pairs of tokens r > s carry a decay; a token's own pair has none and stays out of dg
    dN, dM = Es * (do @ U.mT), -Es * (dW @ U.mT)
    dq = Gam * (do @ S) + dN @ k
    dk_w = d * (U @ dSc)  # as the key written with, from later chunks
    left = last * (S * dSc).sum((-1, -2), keepdim=True) + (k * dk_w).sum((-1, -2), keepdim=True)
    dk_w = dk_w + dN.mT @ q + dM.mT @ k
    dk_e = dM @ k - Gam * (dW @ S)  # as the key erased with
    dgam = ((q * dq).sum(-1, keepdim=True) + (k * (dk_e - dk_w)).sum(-1, keepdim=True)).double()
    dg = torch.flip(torch.cumsum(torch.flip(dgam, (2,)), 2), (2,)) + left.double()
    own_pair = (do * U).sum(-1, keepdim=True)
    dq, dk_w = dq + own_pair * k, dk_w + own_pair * q
    heads = lambda x: unpad(x.reshape(N, Hk, G, n_ch, C, dk).sum(2), Hk).reshape(s["q"].shape)  # noqa: E731
    out = dict(dq=heads(dq), dk=heads(dk_e + dk_w), dv=unpad(dW, Hv).reshape(s["v"].shape),
               dg=unpad(dg, Hv).reshape(s["g"].shape), dbeta=unpad(dbeta, Hv).reshape(s["g"].shape))
    return dict(out, dS0=dS.reshape(N, Hv, dv, dk)) if case["states"] else out


# -------------------------------------------------------------------------------- work ------

def work(case):
    e = 2 if case["dtype"] == BF16 else 4
    if case["op"] == "rule":
        n, N = sum(_lens(case)), len(_lens(case))
        Hk, Hv, dk, dv = case["Hk"], case["Hv"], case["dk"], case["dv"]
        # q, k, v, dout, g, beta in; dq, dk, dv, dg, dbeta out; states
        b = n * (e * (4 * Hk * dk + 3 * Hv * dv + 2 * Hv) + 8 * Hv)
        if case["states"]:
            b += 3 * 4 * N * Hv * dk * dv
        # token by token: S k, the update, and their and the output's gradients: eleven products of
        # dk x dv per token and head
        return dict(bytes=b, flops=2 * 11 * n * Hv * dk * dv)
    if case["op"] == "gates":
        n = case["tokens"] * case["Hv"]
        return dict(bytes=6 * e * n, flops=20 * n)
    if case["op"] == "norm":
        n = case["rows"] * case["dim"]
        return dict(bytes=5 * e * n, flops=25 * n)
    if case["op"] == "conv":
        n = sum(_lens(case)) * case["C"]
        x = 1 + 4 / case["group"] if case["ckpt"] else e
        st = 3 * 4 * len(_lens(case)) * case["C"] * (case["K"] - 1) if case["states"] else 0
        return dict(bytes=n * (x + 2 * e) + st, flops=n * (6 * case["K"] + 20))
    n = case["rows"] * case["dim"]
    q8 = 1 + 4 / case["group"]
    if case["form"] == "pack":
        return dict(bytes=n * (2 * e + 2 * q8), flops=6 * n)
    return dict(bytes=n * (3 * e + 2 * q8) + n * (2 * q8 + 3 * e), flops=45 * n)


# ------------------------------------------------------------------------------- exact ------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rule":
        return _rule_exact(s)
    if case["op"] == "gates":
        a, b, dg, dbeta, Al, bias = (s[n].double().requires_grad_() for n in ("a", "b", "dg", "dbeta", "A_log", "dt_bias"))
        g = -torch.exp(Al) * torch.logaddexp(a + bias, torch.zeros_like(a))
        beta = 1.0 / (1.0 + torch.exp(-b))
        da, db, dA, dbi = torch.autograd.grad((g * dg.detach()).sum() + (beta * dbeta.detach()).sum(), (a, b, Al, bias))
        return dict(da=da, db=db, dA_log=dA, ddt_bias=dbi)
    if case["op"] == "norm":
        return _norm_exact(s["dy"], s["x"].double(), s["z"].double(), s["w"])
    if case["op"] == "conv":
        return _conv_exact(s)
    if case["form"] == "pack":
        x, sc = _codes_exact(s["x"], case["group"])
        return dict(x=x, scales=sc)
    x, z, w = s["x"].double(), s["z"].double(), s["w"].double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * (1.0 + w) * z / (1.0 + torch.exp(-z))
    return dict(_norm_exact(s["dy"], _codes_exact(s["x"], case["dim"])[0], _codes_exact(s["z"], case["dim"])[0], s["w"]), y=y)


def _codes_exact(x, group):
    """The values that the codes stand for, and the scales, which are defined with their rounding to fp32."""
    x = x.double().unflatten(-1, (-1, group))
    m = x.abs().amax(-1, keepdim=True)
    inv = torch.where(m > 0, 127.0 / m, 0.0).float().double()
    sc = (m / 127.0).float().double()
    return ((x * inv).round() * sc).flatten(-2), sc.squeeze(-1)


def _norm_exact(dy, x, z, w):
    x, z, w = (v.detach().double().requires_grad_() for v in (x, z, w))
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * (1.0 + w) * z / (1.0 + torch.exp(-z))
    dx, dz, dw = torch.autograd.grad((y * dy.double()).sum(), (x, z, w))
    return dict(dx=dx, dz=dz, dw=dw)


def _conv_exact(s):
    """Sequence by sequence, by automatic differentiation of the definition."""
    case = s["case"]
    K, Cn = case["K"], case["C"]
    x = s["x"]
    if case["ckpt"]:
        x = x[0].double().unflatten(-1, (-1, case["group"])) * x[1].double().unsqueeze(-1)
    x = x.double().reshape(-1, Cn)
    dy = s["dy"].double().reshape(-1, Cn)
    w = s["w"].double().requires_grad_()
    bias = s["bias"].double().requires_grad_() if s["bias"] is not None else None
    dw, dbias, dx, dcs = torch.zeros_like(w), None if bias is None else torch.zeros_like(bias), [], []
    at = 0
    for n, L in enumerate(_lens(case)):
        xs = x[at:at + L].detach().requires_grad_()
        hist = torch.zeros(K - 1, Cn, device=x.device, dtype=torch.float64)
        if s["cs_in"] is not None:
            hist = s["cs_in"][n].double().t().contiguous()
        hist.requires_grad_()
        full = torch.cat([hist, xs])
        pre = sum(full[i:i + L] * w[:, i] for i in range(K))
        if bias is not None:
            pre = pre + bias
        y = pre / (1.0 + torch.exp(-pre))
        if case["n_l2"]:
            m = case["n_l2"]
            a = y[:, :m].unflatten(-1, (-1, case["group"]))
            y = torch.cat([(a / torch.sqrt((a * a).sum(-1, keepdim=True) + L2_EPS)).flatten(-2), y[:, m:]], -1)
        loss = (y * dy[at:at + L]).sum()
        if s["dcs_out"] is not None:
            loss = loss + (full[L:L + K - 1] * s["dcs_out"][n].double().t()).sum()
        leaves = [xs, w, hist] + ([bias] if bias is not None else [])
        got = torch.autograd.grad(loss, leaves, allow_unused=True, materialize_grads=True)
        dx.append(got[0])
        dw = dw + got[1]
        dcs.append(got[2].t())
        if bias is not None:
            dbias = dbias + got[3]
        at += L
    out = dict(dx=torch.cat(dx).reshape(s["dy"].shape), dw=dw, dbias=dbias,
               dcs=torch.stack(dcs) if s["cs_in"] is not None else None)
    return {k: v for k, v in out.items() if v is not None}


def _rule_exact(s):
    """Token by token over all sequences at once, states kept every 64 tokens and recomputed between."""
    case = s["case"]
    lens, Hk, Hv, dk, dv = _lens(case), case["Hk"], case["Hv"], case["dk"], case["dv"]
    N, G, dev = len(lens), Hv // Hk, s["q"].device
    scale, top = float(dk) ** -0.5, max(lens)

    def rows(x):  # [top, N, H, ...], zeros behind a sequence's end
        x = x.reshape((-1,) + tuple(x.shape[2:]))
        y = torch.zeros((top, N) + tuple(x.shape[1:]), device=dev, dtype=torch.float64)
        at = 0
        for n, L in enumerate(lens):
            y[:L, n] = x[at:at + L].double()
            at += L
        return y

    def packed(y, like):
        return torch.cat([y[:L, n] for n, L in enumerate(lens)]).reshape(like.shape)

    q, k, v, do, beta = (rows(s[n]) for n in ("q", "k", "v", "dout", "beta"))
    decay = torch.exp(rows(s["g"]))
    q, k = (x.repeat_interleave(G, 2) for x in (q, k))
    zero = torch.zeros(N, Hv, dv, dk, device=dev, dtype=torch.float64)
    S = s["S0"].double() if s["S0"] is not None else zero
    dS = s["dST"].double() if s["dST"] is not None else zero

    def step(S, t):
        D = S * decay[t][..., None, None]
        e = v[t] - (D @ k[t][..., None])[..., 0]
        return D, e, D + (beta[t][..., None] * e)[..., None] * k[t][..., None, :]

    kept = []
    for t in range(top):
        if t % 64 == 0:
            kept.append(S)
        S = step(S, t)[2]
    dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, dbeta = torch.zeros_like(beta), torch.zeros_like(beta)
    for c in reversed(range(len(kept))):
        S, saved = kept.pop(), []
        for t in range(64 * c, min(top, 64 * c + 64)):
            D, e, S = step(S, t)
            saved.append((t, D, e, S))
        for t, D, e, S in reversed(saved):
            dS = dS + (scale * do[t])[..., None] * q[t][..., None, :]
            dq[t] = scale * (do[t][..., None, :] @ S)[..., 0, :]
            du = (dS @ k[t][..., None])[..., 0]
            u, b = beta[t][..., None] * e, beta[t][..., None] * du
            dbeta[t] = (du * e).sum(-1)
            dv_[t] = b
            dk_[t] = (u[..., None, :] @ dS)[..., 0, :] - (b[..., None, :] @ D)[..., 0, :]
            dD = dS - b[..., None] * k[t][..., None, :]
            dg[t] = (dD * D).sum((-1, -2))
            dS = dD * decay[t][..., None, None]
    one = lambda x: x.unflatten(2, (Hk, G)).sum(3)  # noqa: E731
    out = dict(dq=packed(one(dq), s["q"]), dk=packed(one(dk_), s["k"]), dv=packed(dv_, s["v"]),
               dg=packed(dg, s["g"]), dbeta=packed(dbeta, s["beta"]))
    return dict(out, dS0=dS) if case["states"] else out
