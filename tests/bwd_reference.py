"""Plain 64-bit references for the training calls: the forward definitions written with torch
operations on the CPU, differentiated by torch.autograd.  Shared by the backward tests."""
import torch

D = torch.float64


def d64(x):
    return None if x is None else x.detach().to("cpu", D)


def rule(q, k, v, g, beta, scale, S0, lens):
    """Token by token over packed tokens [T, H, d]; returns (out [T, Hv, dv], states [N, Hv, dv, dk])."""
    Hk, Hv, dk, dv = q.shape[1], v.shape[1], q.shape[2], v.shape[2]
    q, k = (x.repeat_interleave(Hv // Hk, 1) for x in (q, k))
    outs, states, t = [], [], 0
    for n, L in enumerate(lens):
        S = S0[n] if S0 is not None else torch.zeros(Hv, dv, dk, dtype=D)
        for _ in range(L):
            S = S * torch.exp(g[t])[:, None, None]
            u = beta[t][:, None] * (v[t] - torch.einsum("hvk,hk->hv", S, k[t]))
            S = S + u[:, :, None] * k[t][:, None, :]
            outs.append(scale * torch.einsum("hvk,hk->hv", S, q[t]))
            t += 1
        states.append(S)
    out = torch.stack(outs) if outs else torch.zeros(0, Hv, dv, dtype=D)
    return out, torch.stack(states)


def rule_grads(x, lens, scale):
    """x: dict of q, k, v, g, beta, dout [T, H, ..] and S0, dST or None -> dict of gradients."""
    names = [n for n in ("q", "k", "v", "g", "beta", "S0") if x[n] is not None]
    leaf = {n: d64(x[n]).requires_grad_() for n in names}
    out, S = rule(*(leaf[n] for n in ("q", "k", "v", "g", "beta")), scale, leaf.get("S0"), lens)
    loss = (out * d64(x["dout"])).sum()
    if x["dST"] is not None:
        loss = loss + (S * d64(x["dST"])).sum()
    got = torch.autograd.grad(loss, [leaf[n] for n in names], allow_unused=True,
                              materialize_grads=True)
    return {"d" + n: y for n, y in zip(names, got)}


def gates_grads(a, b, A_log, dt_bias, dg, dbeta):
    leaf = [d64(t).requires_grad_() for t in (a, b, A_log, dt_bias)]
    g = -torch.exp(leaf[2]) * torch.logaddexp(leaf[0] + leaf[3], torch.zeros((), dtype=D))
    beta = torch.sigmoid(leaf[1])
    return torch.autograd.grad((g * d64(dg)).sum() + (beta * d64(dbeta)).sum(), leaf)


def norm(x, z, w, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * (1 + w) * z * torch.sigmoid(z)


def norm_grads(dy, x, z, w, eps):
    leaf = [d64(t).requires_grad_() for t in (x, z, w)]
    return torch.autograd.grad((norm(*leaf, eps) * d64(dy)).sum(), leaf)


def conv(x, w, bias, hist, lens, n_l2, group, eps):
    """x [T, C], hist [N, C, K-1]; returns (y [T, C], the last K-1 inputs of each sequence)."""
    K, ys, left, t = w.shape[1], [], [], 0
    for n, L in enumerate(lens):
        full = torch.cat([hist[n].t(), x[t:t + L]])
        pre = sum((full[i:i + L] * w[:, i] for i in range(K)), torch.zeros(L, w.shape[0], dtype=D))
        y = pre + bias
        y = y * torch.sigmoid(y)
        if n_l2:
            m = y[:, :n_l2].unflatten(-1, (-1, group))
            m = m / torch.sqrt((m * m).sum(-1, keepdim=True) + eps)
            y = torch.cat([m.flatten(-2), y[:, n_l2:]], -1)
        ys.append(y)
        left.append(full[L:L + K - 1].t())
        t += L
    return torch.cat(ys), torch.stack(left)


def conv_grads(dy, x, w, bias, hist, dleft, lens, n_l2, group, eps):
    """(dx, dw, dbias, dhist); bias, hist, dleft may be None (zero)."""
    C, K, N = w.shape[0], w.shape[1], len(lens)
    b = d64(bias) if bias is not None else torch.zeros(C, dtype=D)
    h = d64(hist) if hist is not None else torch.zeros(N, C, K - 1, dtype=D)
    leaf = [t.clone().requires_grad_() for t in (d64(x), d64(w), b, h)]
    y, left = conv(*leaf, lens, n_l2, group, eps)
    loss = (y * d64(dy)).sum()
    if dleft is not None:
        loss = loss + (left * d64(dleft)).sum()
    return torch.autograd.grad(loss, leaf, allow_unused=True, materialize_grads=True)


def act8(x, group):
    """(codes, scales, the values they stand for) of finite x with every |group maximum| >= 2^-100 or 0."""
    x = x.detach().cpu().to(D).unflatten(-1, (-1, group))
    m = x.abs().amax(-1, keepdim=True)
    inv = torch.where(m > 0, 127.0 / m, 0.0).float().to(D)
    sc = (m / 127.0).float()
    codes = (x * inv).round()
    return codes.to(torch.int8).flatten(-2), sc.squeeze(-1), (codes * sc.to(D)).flatten(-2)
