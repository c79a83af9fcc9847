"""fp64 definitions of the state-space block's operators, token by token, and the hand-written reverse of each: the
selective scan, the width-4 convolution with its activation, the norm with its gate. numpy only.

Each `*_bwd` formula is a sum of products of the quantities it is given, so the same functions called with the absolute
values of those quantities (`magnitudes`) give the sum of the terms' absolute values, which the tests' tolerances are
multiples of."""
import numpy as np


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def problem(seed, lens, C, S, G=1, gate=True, skip=True, bias=True, n_pool=0, softplus=True, dfin=False):
    """Inputs of a scan as fp64 arrays (to be rounded by the caller)."""
    rng = np.random.default_rng(seed)
    T = sum(lens)
    p = dict(lens=list(lens), softplus=softplus)
    p["x"], p["dt"] = rng.standard_normal((T, C)), rng.standard_normal((T, C)) * 0.5
    p["b"], p["c"] = rng.standard_normal((T, G, S)), rng.standard_normal((T, G, S))
    p["a"] = -np.arange(1, S + 1)[None] * np.exp(0.1 * rng.standard_normal((C, S)))
    p["z"] = rng.standard_normal((T, C)) if gate else None
    p["skip"] = 1 + 0.1 * rng.standard_normal(C) if skip else None
    p["dt_bias"] = np.log(np.expm1(np.exp(rng.uniform(np.log(1e-3), np.log(0.1), C)))) if bias else None
    if not softplus:
        p["dt"] = np.abs(p["dt"]) * 0.1
        p["dt_bias"] = None if not bias else np.full(C, 0.01)
    p["pool"] = 0.5 * rng.standard_normal((n_pool, C, S)) if n_pool else None
    p["dout"] = rng.standard_normal((T, C))
    p["dfin"] = 0.1 * rng.standard_normal((len(lens), C, S)) if dfin else None
    return p


def terms(p):
    """What the recurrence is made of: steps, decays, gates and their slopes."""
    C, G = p["x"].shape[1], p["b"].shape[1]
    g = np.arange(C) // (C // G)
    raw = p["dt"] + (0 if p["dt_bias"] is None else p["dt_bias"])
    q = dict(lens=p["lens"], x=p["x"], a=p["a"], G=G, group=g)
    q["delta"] = np.logaddexp(0, raw) if p["softplus"] else raw
    q["ddelta"] = sigmoid(raw) if p["softplus"] else np.ones_like(raw)
    q["e"] = np.exp(q["delta"][..., None] * p["a"])
    q["b"], q["c"] = p["b"][:, g], p["c"][:, g]
    q["skip"] = np.zeros(C) if p["skip"] is None else p["skip"]
    q["pool"] = p["pool"]
    if p["z"] is None:
        q["gate"], q["slope"] = np.ones_like(raw), np.zeros_like(raw)
    else:
        z, s = p["z"], sigmoid(p["z"])
        q["gate"], q["slope"] = z * s, s * (1 + z * (1 - s))
        q["slope_terms"] = s * (1 + np.abs(z) * (1 - s))
    return q


def magnitudes(q):
    m = {k: np.abs(v) if isinstance(v, np.ndarray) and v.dtype == np.float64 else v for k, v in q.items()}
    m["slope"] = q.get("slope_terms", m["slope"])
    return m


def scan_fwd(q, idx=None):
    """(out, y, states after each token, states before each token, final states)."""
    T, C = q["x"].shape
    S, N = q["a"].shape[1], len(q["lens"])
    n_pool = 0 if q["pool"] is None else len(q["pool"])
    after, before = np.zeros((T, C, S)), np.zeros((T, C, S))
    final = np.zeros((N, C, S))
    t = 0
    for d, n in enumerate(q["lens"]):
        i = -1 if idx is None else idx[d]
        h = np.zeros((C, S)) if i < 0 else q["pool"][i] if i < n_pool else final[i - n_pool]
        for t in range(t, t + n):
            before[t] = h
            h = q["e"][t] * h + (q["delta"][t] * q["x"][t])[:, None] * q["b"][t]
            after[t] = h
        t += n > 0
        final[d] = h
    y = (after * q["c"]).sum(2) + q["skip"] * q["x"]
    return y * q["gate"], y, after, before, final


def scan_bwd(q, dout, dfin=None, idx=None):
    T, C = q["x"].shape
    S, N, G = q["a"].shape[1], len(q["lens"]), q["G"]
    n_pool = 0 if q["pool"] is None else len(q["pool"])
    _, y, after, before, _ = scan_fwd(q, idx)
    dy = dout * q["gate"]
    k_at = np.zeros((T, C, S))  # the gradient of the state after each token
    dstate = np.zeros((N, C, S)) if dfin is None else dfin.copy()
    dinit = np.zeros((n_pool, C, S))
    ends = np.cumsum(q["lens"])
    for d in range(N - 1, -1, -1):
        k = dstate[d]
        for t in range(ends[d] - 1, ends[d] - q["lens"][d] - 1, -1):
            k = k + dy[t][:, None] * q["c"][t]
            k_at[t] = k
            k = k * q["e"][t]
        i = -1 if idx is None else idx[d]
        if i >= n_pool:
            dstate[i - n_pool] += k
        elif i >= 0:
            dinit[i] += k
    v = k_at * q["e"] * before
    du = (k_at * q["b"]).sum(2)
    per = lambda m: m.reshape(T, G, C // G, S).sum(2)  # noqa: E731
    ddt = (q["x"] * du + (v * q["a"]).sum(2)) * q["ddelta"]
    return dict(dx=q["delta"] * du + q["skip"] * dy, ddt=ddt, dz=dout * y * q["slope"],
                da=(v * q["delta"][..., None]).sum(0), db=per(k_at * (q["delta"] * q["x"])[..., None]),
                dc=per(dy[..., None] * after), dskip=(dy * q["x"]).sum(0), ddt_bias=ddt.sum(0), dinit=dinit)


# ------------------------------------------------------------------------------ convolution with SiLU


def _extended(x, lens, pool, idx):
    """Per document (first token, its three inputs in front and its own)."""
    tails, out, t = [], [], 0
    n_pool = 0 if pool is None else len(pool)
    for d, n in enumerate(lens):
        i = -1 if idx is None else idx[d]
        start = np.zeros((3, x.shape[1])) if i < 0 else pool[i] if i < n_pool else tails[i - n_pool]
        e = np.concatenate([start, x[t:t + n]])
        tails.append(e[n:])
        out.append((t, e))
        t += n
    return out, np.stack(tails)


def conv_fwd(x, w, bias, lens, pool=None, idx=None, silu=True):
    docs, tails = _extended(x, lens, pool, idx)
    u = np.zeros_like(x)
    for t, e in docs:
        n = len(e) - 3
        u[t:t + n] = bias + sum(w[:, m] * e[m:m + n] for m in range(4))
    return (u * sigmoid(u) if silu else u), u, tails


def conv_bwd(x, w, lens, du, dtail=None, pool=None, idx=None):
    """From the gradient of u, the convolution's output before its activation."""
    docs, tails = _extended(x, lens, pool, idx)
    n_pool = 0 if pool is None else len(pool)
    g = np.zeros_like(tails) if dtail is None else dtail.copy()
    dx, dw = np.zeros_like(x), np.zeros_like(w)
    dinit = np.zeros((n_pool, 3, x.shape[1]))
    for d in range(len(lens) - 1, -1, -1):
        t, e = docs[d]
        n = len(e) - 3
        de = np.zeros_like(e)
        for m in range(4):
            de[m:m + n] += w[:, m] * du[t:t + n]
            dw[:, m] += (du[t:t + n] * e[m:m + n]).sum(0)
        de[n:] += g[d]
        dx[t:t + n] = de[3:]
        i = -1 if idx is None else idx[d]
        if i >= n_pool:
            g[i - n_pool] += de[:3]
        elif i >= 0:
            dinit[i] += de[:3]
    return dict(dx=dx, dw=dw, dbias=du.sum(0), dconv_init=dinit)


# ------------------------------------------------------------------------------ norm with its gate


def gnorm_fwd(x, z, w, group, eps, first):
    T, D = x.shape
    gate = z * sigmoid(z)
    u = (x if first == "norm" else x * gate).reshape(T, -1, group)
    hat = (u / np.sqrt((u * u).mean(2, keepdims=True) + eps)).reshape(T, D)
    y = hat * np.tile(w, D // len(w))
    return y * gate if first == "norm" else y


def gnorm_bwd(x, z, w, dy, group, eps, first):
    """dx, dz, dw and, for each, the sum of its terms' absolute values."""
    T, D = x.shape
    s = sigmoid(z)
    gate, slope = z * s, s * (1 + z * (1 - s))
    norm = first == "norm"
    u = x if norm else x * gate
    v = u.reshape(T, -1, group)
    rs = 1 / np.sqrt((v * v).mean(2, keepdims=True) + eps)
    hat = (v * rs).reshape(T, D)
    ww = np.tile(w, D // len(w))
    dn = dy * gate if norm else dy
    g = ww * dn

    def du(g, hat):
        m = (g * hat).reshape(T, -1, group).mean(2, keepdims=True)
        return (rs * g.reshape(T, -1, group)).reshape(T, D), (rs * hat.reshape(T, -1, group) * m).reshape(T, D)
    p, q = du(g, hat)
    pa, qa = du(np.abs(g), np.abs(hat))
    d, da = p - q, pa + qa
    sa = s * (1 + np.abs(z) * (1 - s))
    fold = lambda m: m.sum(0).reshape(-1, len(w)).sum(0)  # noqa: E731
    if norm:
        dx, dxa, dz, dza = d, da, dy * hat * ww * slope, np.abs(dy * hat * ww) * sa
    else:
        dx, dxa, dz, dza = d * gate, da * np.abs(gate), d * x * slope, da * np.abs(x) * sa
    return (dx, dz, fold(dn * hat)), (dxa, dza, fold(np.abs(dn * hat)))
