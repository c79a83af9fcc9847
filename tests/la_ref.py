"""Plain fp64 definitions of the decayed linear attention (token by token, its reverse mode written out
by hand) and of the root-mean-square norm, in numpy, with the test inputs. No library code."""
from __future__ import annotations

import numpy as np

D = 128


def la_fwd(q, k, v, g, lens, idx=None, pool=None, scale=1.0):
    """q, k [T, Hk, D], v [T, Hv, D], g [Hv]; idx as init_idx (-1 zero, a pool entry, n_pool + j a fork of document
    j). Returns out, final states and every document's start state."""
    T, Hk, dk = q.shape
    Hv, dv = v.shape[1:]
    head = np.arange(Hv) // (Hv // Hk)
    n_pool = 0 if pool is None else len(pool)
    lam = np.exp(np.maximum(g, -1e4))[:, None, None]
    out, fin, starts, t = np.zeros((T, Hv, dv)), [], [], 0
    for i, n in enumerate(lens):
        x = -1 if idx is None else idx[i]
        S = np.zeros((Hv, dk, dv)) if x < 0 else (pool[x] if x < n_pool else fin[x - n_pool]).copy()
        starts.append(S)
        for t in range(sum(lens[:i]), sum(lens[:i]) + n):
            S = lam * S + k[t][head][:, :, None] * v[t][:, None, :]
            out[t] = scale * np.einsum("hk,hkv->hv", q[t][head], S)
        fin.append(S)
    return out, np.array(fin), starts


def la_bwd(q, k, v, g, lens, do, dfin=None, idx=None, pool=None, scale=1.0):
    """Gradients of sum(do * out) + sum(dfin * final): dq, dk, dv, dpool (None without a pool)."""
    T, Hk, dk_ = q.shape
    Hv, dv_ = v.shape[1:]
    G = Hv // Hk
    head = np.arange(Hv) // G
    n_pool = 0 if pool is None else len(pool)
    lam = np.exp(np.maximum(g, -1e4))[:, None, None]
    _, _, starts = la_fwd(q, k, v, g, lens, idx, pool, scale)
    dq, dk, dv = np.zeros((T, Hv, dk_)), np.zeros((T, Hv, dk_)), np.zeros((T, Hv, dv_))
    dS = [np.zeros((Hv, dk_, dv_)) if dfin is None else dfin[i].copy() for i in range(len(lens))]
    dpool = None if pool is None else np.zeros_like(pool)
    for i in range(len(lens) - 1, -1, -1):
        t0, S, states = sum(lens[:i]), starts[i], []
        for t in range(t0, t0 + lens[i]):
            S = lam * S + k[t][head][:, :, None] * v[t][:, None, :]
            states.append(S)
        X = dS[i]
        for t in range(t0 + lens[i] - 1, t0 - 1, -1):
            dq[t] = scale * np.einsum("hkv,hv->hk", states[t - t0], do[t])
            X = X + scale * q[t][head][:, :, None] * do[t][:, None, :]
            dv[t] = np.einsum("hkv,hk->hv", X, k[t][head])
            dk[t] = np.einsum("hkv,hv->hk", X, v[t])
            X = lam * X
        x = -1 if idx is None else idx[i]
        if x >= n_pool:
            dS[x - n_pool] += X
        elif x >= 0:
            dpool[x] += X
    group = lambda a: a.reshape(T, Hk, G, dk_).sum(2)  # noqa: E731
    return group(dq), group(dk), dv, dpool


def rms_fwd(x, w, r=None, eps=1e-6):
    h = x if r is None else x + r
    return h * w / np.sqrt((h * h).mean(1, keepdims=True) + eps), h


def rms_bwd(h, w, dy, dh=None, eps=1e-6):
    rs = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    dx = rs * w * dy - h * rs ** 3 * (w * dy * h).mean(1, keepdims=True)
    return dx if dh is None else dx + dh, (dy * h * rs).sum(0)


def bf16(x):
    """Rounded to bf16 (to nearest, ties to even), in fp64."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def problem(seed, lens, Hk, Hv, g, n_pool=0, dfin=False):
    """Inputs in fp64 that bf16 (q, k, v, do) and fp32 (g, states) hold exactly."""
    rng = np.random.default_rng(seed)
    T = sum(lens)
    silu = lambda x: x / (1 + np.exp(-x))  # noqa: E731
    f32 = lambda x: x.astype(np.float32).astype(np.float64)  # noqa: E731
    p = dict(q=bf16(silu(rng.standard_normal((T, Hk, D)))), k=bf16(silu(rng.standard_normal((T, Hk, D)))),
             v=bf16(rng.standard_normal((T, Hv, D))), do=bf16(rng.standard_normal((T, Hv, D))),
             g=f32(np.broadcast_to(np.asarray(g, dtype=np.float64), (Hv,))), lens=list(lens))
    p["pool"] = f32(rng.standard_normal((n_pool, Hv, D, D))) if n_pool else None
    p["dfin"] = f32(0.3 * rng.standard_normal((len(lens), Hv, D, D))) if dfin else None
    return p
