"""Quadratic form of the decayed linear attention and of its gradients for one head of one document, in fp64 on
torch tensors: the whole matrix of weights lam^(t - s), so that long documents can be compared on the GPU. No
library code."""
import torch


def weights(n, g, device):
    """lam^(t - s) for s <= t, and the decay of the start state and of what is left at the end."""
    t = torch.arange(n, dtype=torch.float64, device=device)
    gap = t[:, None] - t[None]
    m = torch.where(gap >= 0, torch.exp(g * gap.clamp(min=0)), torch.zeros_like(gap))
    return m, torch.exp(g * (t + 1))[:, None], torch.exp(g * (n - 1 - t))[:, None]


def forward(q, k, v, g, start, scale):
    """q, k, v [n, 128] of the head in fp64, g a float: (out, final state)."""
    m, since, left = weights(len(q), g, q.device)
    out = ((q @ k.T) * m) @ v + since * (q @ start)
    return scale * out, (k * left).T @ v + torch.exp(torch.tensor(g * len(q), dtype=torch.float64)) * start


def backward(q, k, v, g, start, scale, do, dfin):
    """Gradients of sum(do * out) + sum(dfin * final): dq, dk, dv, dstart."""
    m, since, left = weights(len(q), g, q.device)
    p, r = (q @ k.T) * m, (do @ v.T) * m
    dq = scale * (r @ k + since * (do @ start.T))
    dk = scale * (r.T @ q) + left * (v @ dfin.T)
    dv = scale * (p.T @ do) + left * (k @ dfin)
    return dq, dk, dv, torch.exp(torch.tensor(g * len(q), dtype=torch.float64)) * dfin + scale * (q * since).T @ do


def packed(d, lens, idx=None, scale=1.0):
    """Every head of a packed batch, from its device tensors (q, k, v, do, g, pool, dfin): dict of out, fin, dqh, dkh
    (by value head), dv, dpool, in fp64."""
    q, k, v, do = (d[x].double() for x in ("q", "k", "v", "do"))
    Hk, Hv, g = q.shape[1], v.shape[1], [max(float(x), -1e4) for x in d["g"]]
    zero = torch.zeros(128, 128, dtype=torch.float64, device=q.device)
    r = dict(out=torch.zeros_like(v), dv=torch.zeros_like(v), dqh=torch.zeros_like(v), dkh=torch.zeros_like(v),
             fin=torch.zeros(len(lens), Hv, 128, 128, dtype=torch.float64, device=q.device),
             dpool=None if d["pool"] is None else torch.zeros_like(d["pool"], dtype=torch.float64))
    t0 = 0
    for i, n in enumerate(lens):
        s, x = slice(t0, t0 + n), -1 if idx is None else idx[i]
        t0 += n
        for h in range(Hv):
            hk = h // (Hv // Hk)
            start = d["pool"][x, h].double() if x >= 0 else zero
            dfin = zero if d["dfin"] is None else d["dfin"][i, h].double()
            a = (q[s, hk], k[s, hk], v[s, h], g[h], start, scale)
            r["out"][s, h], r["fin"][i, h] = forward(*a)
            r["dqh"][s, h], r["dkh"][s, h], r["dv"][s, h], dstart = backward(*a, do[s, h], dfin)
            if x >= 0:
                r["dpool"][x, h] += dstart
    return r
