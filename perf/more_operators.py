"""Cases of a state-space block: the selective scan (prompts, gradients, single tokens), the short convolution in
front of it with its activation (the same three) and the gated norm behind it (forward, backward), with their plain
forms in 32 bits and their definitions in 64.

The scan, per channel c with states s, group g = c // (channels / groups):
    dt = softplus(dt_raw + dt_bias),  h_t = exp(dt_t a) h_{t-1} + dt_t b_t x_t,  y_t = sum_s c_t h_t + skip x_t,
    out = y silu(z)
per document, from a zero state or an entry of a pool of states. The convolution, per channel over the current
and the three preceding inputs: y_t = silu(bias + sum_m w_m x_{t-3+m}). The gated norm, for each group of columns:
    y = w x / sqrt(mean(x^2) + eps) silu(z),  or the same norm of x silu(z).
"""
import math
import random

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # a short prompt on its own: one document, latency counts
        {"name": "ssm_fwd_short", "op": "ssm_fwd", "T": 512, "N": 1, "C": 1024, "S": 16, "G": 1, "dtype": "bf16", "gate": True, "pool": 0},
        # continuations of cached prefixes: ragged documents, start states from a pool, an odd total
        {"name": "ssm_fwd_pool", "op": "ssm_fwd", "T": 9001, "N": 12, "C": 2048, "S": 16, "G": 1, "dtype": "fp16", "gate": True, "pool": 3},
        # one long prompt: nothing to run side by side but its channels and its own segments
        {"name": "ssm_fwd_long", "op": "ssm_fwd", "T": 32768, "N": 1, "C": 2048, "S": 16, "G": 1, "dtype": "bf16", "gate": True, "pool": 0},
        # gradients of a small fine-tuning batch with learned start states, in fp32, without the gate
        {"name": "ssm_bwd_small", "op": "ssm_bwd", "T": 1501, "N": 5, "C": 768, "S": 8, "G": 2, "dtype": "fp32", "gate": False, "pool": 2},
        # gradients of a long-context step: four documents
        {"name": "ssm_bwd_long", "op": "ssm_bwd", "T": 16384, "N": 4, "C": 2048, "S": 16, "G": 1, "dtype": "bf16", "gate": True, "pool": 0},
        # one user's next token
        {"name": "ssm_step_one", "op": "ssm_step", "B": 1, "C": 2048, "S": 16, "G": 1, "dtype": "bf16", "gate": True, "pool": 4},
        # the next token of a full serving batch
        {"name": "ssm_step_batch", "op": "ssm_step", "B": 200, "C": 8192, "S": 16, "G": 1, "dtype": "bf16", "gate": True, "pool": 256},
        # the convolution of a packed prefill batch, x a view into the fused projection
        {"name": "conv_fwd_packed", "op": "conv_fwd", "T": 32768, "N": 12, "C": 2048, "dtype": "bf16", "pool": 0},
        # its gradients in a training step, start tails from a pool
        {"name": "conv_bwd_packed", "op": "conv_bwd", "T": 16384, "N": 4, "C": 4096, "dtype": "bf16", "pool": 2},
        # its step for a full serving batch
        {"name": "conv_step_batch", "op": "conv_step", "B": 200, "C": 8192, "dtype": "fp16", "pool": 256},
        # the norm of each head's output before its gate, a prompt of 64 heads
        {"name": "gnorm_fwd_heads", "op": "gnorm_fwd", "T": 16384, "D": 8192, "group": 128, "shared": True, "first": "norm", "dtype": "bf16"},
        # the gate before the norm over all channels, gradients of a training step
        {"name": "gnorm_bwd_rows", "op": "gnorm_bwd", "T": 32768, "D": 2048, "group": 2048, "shared": False, "first": "gate", "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ssm_fwd", "ssm_fwd", "ssm_bwd", "ssm_bwd", "ssm_step", "conv_fwd", "conv_bwd", "conv_step",
                     "gnorm_fwd", "gnorm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("ssm_fwd", "ssm_bwd", "ssm_step"):
        S = rng.choice([5, 8, 16, 16, 16, 32, 64])
        G = rng.choice([1, 1, 2, 4])
        C = G * _log_int(rng, 16, 4096 // G)
        case = {"op": op, "C": C, "S": S, "G": G, "dtype": dtype, "gate": rng.random() < 0.7}
        if op == "ssm_step":
            case["B"] = _log_int(rng, 1, min(256, (1 << 24) // (C * S)))
            case["pool"] = case["B"] + rng.randrange(0, 17)
            return case
        T = _log_int(rng, 1, min(32768, (1 << (30 if op == "ssm_fwd" else 29)) // (C * S)))
        return {**case, "T": T, "N": _log_int(rng, 1, max(1, min(64, T // 8))), "pool": rng.choice([0, 0, 1, 5])}
    if op in ("conv_fwd", "conv_bwd", "conv_step"):
        C = 8 * _log_int(rng, 1, 1024)
        if op == "conv_step":
            B = _log_int(rng, 1, 256)
            return {"op": op, "B": B, "C": C, "dtype": dtype, "pool": B + rng.randrange(0, 17)}
        T = _log_int(rng, 1, min(32768, (1 << 26) // C))
        return {"op": op, "T": T, "N": _log_int(rng, 1, max(1, min(64, T // 8))), "C": C, "dtype": dtype,
                "pool": rng.choice([0, 0, 1, 5])}
    group = rng.choice([64, 128, 128, 256, _log_int(rng, 32, 8192)])
    D = group * _log_int(rng, 1, max(1, 8192 // group))
    T = _log_int(rng, 1, min(65536, (1 << 26) // D))
    return {"op": op, "T": T, "D": D, "group": group, "shared": rng.random() < 0.5, "first": rng.choice(["norm", "gate"]),
            "dtype": dtype}


def _lengths(case):
    """Ragged documents: N - 1 cuts at random places, the same for every seed."""
    T, N = case["T"], case["N"]
    r = random.Random(T * 1000003 + N)
    cuts = [0] + sorted(r.randint(0, T) for _ in range(N - 1)) + [T]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 29)
    dt = TYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32, by=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * by).to(dtype)

    s = {"op": case["op"]}
    if case["op"].startswith("gnorm"):
        T, Dm = case["T"], case["D"]
        s["x"] = normal(T, Dm, dtype=dt, by=2.0)
        s["z"] = normal(T, Dm, dtype=dt)
        s["w"] = (1.0 + normal(case["group"] if case["shared"] else Dm, by=0.1)).to(dt)
        s["group"], s["first"] = case["group"], case["first"]
        if case["op"] == "gnorm_bwd":
            s["dy"] = normal(T, Dm, dtype=dt)
        return s
    C, pool = case["C"], case["pool"]
    step = case["op"].endswith("step")
    T = case["B"] if step else case["T"]
    if step:
        s["state_idx"] = torch.randperm(pool, generator=gen, device=dev)[:T].to(torch.int32)
    else:
        cu = [0]
        for n in _lengths(case):
            cu.append(cu[-1] + n)
        s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["init_idx"] = torch.tensor([i % (pool + 1) - 1 for i in range(case["N"])], dtype=torch.int32, device=dev) if pool else None
    # the projection into the convolved channels and the gate; x and z are its halves
    fused = normal(T, 2 * C, dtype=dt)
    if case["op"].startswith("conv"):
        s["x"] = fused[:, :C]
        s["w"] = normal(C, 4, by=0.5)
        s["bias"] = normal(C, by=0.1)
        if step:
            s["tail_pool"] = normal(pool, 3, C, dtype=dt)
        else:
            s["conv_init"] = normal(pool, 3, C, dtype=dt) if pool else None
            if case["op"] == "conv_bwd":
                s["dy"] = normal(T, C, dtype=dt)
                s["dfinal_tail"] = normal(case["N"], 3, C, by=0.1) if pool else None
        return s
    S, G = case["S"], case["G"]
    # channels after the convolution's activation, time steps before the softplus, both maps views into a projection
    s["x"] = torch.nn.functional.silu(normal(T, C)).to(dt)
    s["z"] = fused[:, C:] if case["gate"] else None
    s["dt"] = normal(T, C, dtype=dt, by=0.5)
    rank = 8 * (-(-C // 128))
    maps = normal(T, rank + 2 * G * S, dtype=dt)
    s["b"] = maps[:, rank:rank + G * S].unflatten(1, (G, S))
    s["c"] = maps[:, rank + G * S:].unflatten(1, (G, S))
    # decays 1 .. S a unit of time, steps spread over 0.001 .. 0.1 by their bias
    s["a"] = -torch.arange(1, S + 1, device=dev).float()[None] * torch.exp(normal(C, S, by=0.1))
    steps = torch.exp(torch.rand(C, generator=gen, device=dev) * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = torch.log(torch.expm1(steps))
    s["skip"] = 1.0 + normal(C, by=0.1)
    if step:
        s["state_pool"] = normal(pool, C, S)
    else:
        s["initial_state"] = normal(pool, C, S, by=0.5) if pool else None
        if case["op"] == "ssm_bwd":
            s["dout"] = normal(T, C, dtype=dt)
            s["dfinal_state"] = normal(case["N"], C, S, by=0.1) if pool else None
    return s


# ------------------------------------------------------------------------------------------------ plain forms


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _silu_grad(x):
    p = _sigmoid(x)
    return p * (1.0 + x * (1.0 - p))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along the first dimension, from zero; blocks of tokens abreast, then carried on.
    Overwrites a and b; returns b."""
    T = a.shape[0]
    L = max(1, int(math.isqrt(T)))
    n = T // L
    head, rest = n * L, T - n * L
    av, bv = a[:head].unflatten(0, (n, L)), b[:head].unflatten(0, (n, L))
    for i in range(1, L):
        bv[:, i].addcmul_(av[:, i], bv[:, i - 1])
        av[:, i].mul_(av[:, i - 1])
    for j in range(1, n):
        bv[j].addcmul_(av[j], bv[j - 1, L - 1])
    for i in range(head, head + rest):
        b[i].addcmul_(a[i], b[i - 1])
    return b


def _starts(cu, idx, init):
    """The tokens that begin a document, the ones that end it, and each document's start from the pool or None."""
    live = cu[1:] > cu[:-1]
    first, last = cu[:-1].long()[live], cu[1:].long()[live] - 1
    if init is None:
        return live, first, last, None
    x = idx.long()
    start = torch.where((x >= 0).view(-1, *[1] * (init.dim() - 1)), init.float()[x.clamp(min=0)], 0.0)
    return live, first, last, start


def _per_channel(x, C):
    return x.float().repeat_interleave(C // x.shape[1], dim=1)  # [T, G, S] -> [T, C, S]


def _ssm_parts(s):
    x = s["x"].float()
    raw = s["dt"].float() + s["dt_bias"]
    delta = _softplus(raw)
    b, c = _per_channel(s["b"], x.shape[1]), _per_channel(s["c"], x.shape[1])
    return x, raw, delta, b, c


def _states(s, x, delta, b, start, first):
    a = torch.exp(delta[..., None] * s["a"])
    h = (delta * x)[..., None] * b
    if start is not None:
        h[first] += a[first] * start
    work = a.clone()
    work[first] = 0.0
    return a, _recur(work, h)


def _gated(s, y):
    return y if s["z"] is None else y * s["z"].float() * _sigmoid(s["z"].float())


def _ssm_fwd(s):
    x, _, delta, b, c = _ssm_parts(s)
    live, first, last, start = _starts(s["cu_seqlens"], s["init_idx"], s["initial_state"])
    _, h = _states(s, x, delta, b, None if start is None else start[live], first)
    y = (h * c).sum(2) + s["skip"] * x
    final = torch.zeros(live.numel(), *h.shape[1:], device=x.device) if start is None else start.clone()
    final[live] = h[last]
    return {"out": _gated(s, y).to(s["x"].dtype), "final_state": final}


def _ssm_bwd(s):
    x, raw, delta, b, c = _ssm_parts(s)
    live, first, last, start = _starts(s["cu_seqlens"], s["init_idx"], s["initial_state"])
    a, h = _states(s, x, delta, b, None if start is None else start[live], first)
    T, C, S = h.shape
    G = s["b"].shape[1]
    dt_ = s["x"].dtype
    dout = s["dout"].float()
    out = {}
    dy = dout
    if s["z"] is not None:
        z = s["z"].float()
        y = (h * c).sum(2) + s["skip"] * x
        out["dz"] = (dout * y * _silu_grad(z)).to(dt_)
        dy = dout * z * _sigmoid(z)
    groups = lambda m: m.view(T, G, C // G, S).sum(2).to(s["b"].dtype)  # noqa: E731
    out["dc"] = groups(dy[..., None] * h)
    g = dy[..., None] * c
    if s["dfinal_state"] is not None:
        g[last] += s["dfinal_state"][live]
    nxt = torch.zeros_like(a)
    nxt[:-1] = a[1:]
    nxt[last] = 0.0
    g = _recur(nxt.flip(0), g.flip(0)).flip(0)  # the gradient of h
    out["db"] = groups(g * (delta * x)[..., None])
    du = (g * b).sum(2)
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[first] = 0.0 if start is None else start[live]
    v = g * a * before
    ddelta = x * du + (v * s["a"]).sum(2)
    out["da"] = (v * delta[..., None]).sum(0)
    out["dx"] = (delta * du + s["skip"] * dy).to(dt_)
    ddt = ddelta * _sigmoid(raw)
    out["ddt"] = ddt.to(dt_)
    out["ddt_bias"] = ddt.sum(0)
    out["dskip"] = (dy * x).sum(0)
    if start is not None:
        dstart = torch.zeros_like(start) if s["dfinal_state"] is None else s["dfinal_state"].clone()
        dstart[live] = (a * g)[first]
        i = s["init_idx"].long()
        out["dinit"] = torch.zeros_like(s["initial_state"]).index_add_(
            0, i.clamp(min=0), torch.where((i >= 0)[:, None, None], dstart, 0.0))
    return out


def _ssm_step(s):
    x, _, delta, b, c = _ssm_parts(s)
    i = s["state_idx"].long()
    h = torch.exp(delta[..., None] * s["a"]) * s["state_pool"][i] + (delta * x)[..., None] * b
    s["state_pool"][i] = h
    y = (h * c).sum(2) + s["skip"] * x
    return {"out": _gated(s, y).to(s["x"].dtype), "states": s["state_pool"]}


def _conv_rows(s):
    """All tokens, each document's three inputs before its first in front of it: rows [T + 3 N, C], and each
    token's row."""
    cu, x = s["cu_seqlens"].long(), s["x"].float()
    N, T = cu.numel() - 1, x.shape[0]
    doc = torch.searchsorted(cu[1:], torch.arange(T, device=x.device), right=True)
    at = torch.arange(T, device=x.device) + 3 * (doc + 1)
    ext = torch.zeros(T + 3 * N, x.shape[1], device=x.device)
    ext[at] = x
    front = (cu[:-1] + 3 * torch.arange(N, device=x.device))[:, None] + torch.arange(3, device=x.device)
    if s["conv_init"] is not None:
        ext[front] = _starts(s["cu_seqlens"], s["init_idx"], s["conv_init"])[3]
    back = (cu[1:] + 3 * torch.arange(N, device=x.device))[:, None] + torch.arange(3, device=x.device)
    return ext, at, front, back


def _conv_taps(s, ext, at):
    return s["bias"] + sum(s["w"][:, m] * ext[at - 3 + m] for m in range(4))


def _conv_fwd(s):
    ext, at, _, back = _conv_rows(s)
    u = _conv_taps(s, ext, at)
    return {"y": (u * _sigmoid(u)).to(s["x"].dtype), "final_tail": ext[back].to(s["x"].dtype)}


def _conv_bwd(s):
    ext, at, front, back = _conv_rows(s)
    du = s["dy"].float() * _silu_grad(_conv_taps(s, ext, at))
    dext = torch.zeros_like(ext)
    dw = []
    for m in range(4):
        dext[at - 3 + m] += s["w"][:, m] * du
        dw.append((du * ext[at - 3 + m]).sum(0))
    if s["dfinal_tail"] is not None:
        dext[back] += s["dfinal_tail"]
    out = {"dx": dext[at], "dw": torch.stack(dw, 1), "dbias": du.sum(0)}
    if s["conv_init"] is not None:
        i = s["init_idx"].long()
        out["dconv_init"] = torch.zeros(s["conv_init"].shape, device=ext.device).index_add_(
            0, i.clamp(min=0), torch.where((i >= 0)[:, None, None], dext[front], 0.0))
    return out


def _conv_step(s):
    i = s["state_idx"].long()
    rows = torch.cat([s["tail_pool"][i], s["x"][:, None]], 1)  # [B, 4, C]
    u = s["bias"] + (s["w"].t() * rows.float()).sum(1)
    s["tail_pool"][i] = rows[:, 1:]
    return {"y": (u * _sigmoid(u)).to(s["x"].dtype), "tails": s["tail_pool"]}


def _gnorm_fwd(s):
    x, z = s["x"].float(), s["z"].float()
    gate = z * _sigmoid(z)
    u = (x if s["first"] == "norm" else x * gate).unflatten(1, (-1, s["group"]))
    y = (u * torch.rsqrt(u.square().mean(2, keepdim=True) + EPS)).flatten(1)
    y = y * s["w"].float().repeat(x.shape[1] // s["w"].numel())
    return {"y": (y * gate if s["first"] == "norm" else y).to(s["x"].dtype)}


def _gnorm_bwd(s):
    x, z, dy = s["x"].float(), s["z"].float(), s["dy"].float()
    p = _sigmoid(z)
    gate, slope = z * p, p * (1.0 + z * (1.0 - p))
    norm_first = s["first"] == "norm"
    u = (x if norm_first else x * gate).unflatten(1, (-1, s["group"]))
    rs = torch.rsqrt(u.square().mean(2, keepdim=True) + EPS)
    w = s["w"].float().repeat(x.shape[1] // s["w"].numel())
    hat = (u * rs).flatten(1)
    dn = dy * gate if norm_first else dy
    g = (w * dn).unflatten(1, (-1, s["group"]))
    du = (rs * g - u * rs ** 3 * (g * u).mean(2, keepdim=True)).flatten(1)
    dx, dz = (du, dy * hat * w * slope) if norm_first else (du * gate, du * x * slope)
    dw = (dn * hat).sum(0).view(-1, s["w"].numel()).sum(0)
    return {"dx": dx.to(s["x"].dtype), "dz": dz.to(s["x"].dtype), "dw": dw}


def run(s):
    if not own:
        return {"ssm_fwd": _ssm_fwd, "ssm_bwd": _ssm_bwd, "ssm_step": _ssm_step, "conv_fwd": _conv_fwd,
                "conv_bwd": _conv_bwd, "conv_step": _conv_step, "gnorm_fwd": _gnorm_fwd, "gnorm_bwd": _gnorm_bwd}[s["op"]](s)
    import linear_attention_varlen_gb300 as gdn
    if s["op"] == "ssm_fwd":
        out, final = gdn.ssm_scan_fwd(s["x"], s["dt"], s["a"], s["b"], s["c"], s["cu_seqlens"], skip=s["skip"], z=s["z"],
                                      dt_bias=s["dt_bias"], init_idx=s["init_idx"], initial_state=s["initial_state"])
        return {"out": out, "final_state": final}
    if s["op"] == "ssm_bwd":
        g = gdn.ssm_scan_bwd(s["x"], s["dt"], s["a"], s["b"], s["c"], s["cu_seqlens"], s["dout"],
                             dfinal_state=s["dfinal_state"], skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"],
                             init_idx=s["init_idx"], initial_state=s["initial_state"])
        return {k: v for k, v in g.items() if v is not None}
    if s["op"] == "ssm_step":
        out = gdn.ssm_decode_step(s["x"], s["dt"], s["a"], s["b"], s["c"], s["state_pool"], s["state_idx"], skip=s["skip"],
                                  z=s["z"], dt_bias=s["dt_bias"])
        return {"out": out, "states": s["state_pool"]}
    if s["op"] == "conv_fwd":
        y, tail = gdn.conv_fwd(s["x"], s["w"], s["cu_seqlens"], bias=s["bias"], init_idx=s["init_idx"],
                               conv_init=s["conv_init"], activation="silu")
        return {"y": y, "final_tail": tail}
    if s["op"] == "conv_bwd":
        g = gdn.conv_bwd(s["x"], s["w"], s["cu_seqlens"], s["dy"], bias=s["bias"], init_idx=s["init_idx"],
                         conv_init=s["conv_init"], dfinal_tail=s["dfinal_tail"], activation="silu")
        return {k: v for k, v in g.items() if v is not None}
    if s["op"] == "conv_step":
        y = gdn.conv_decode_step(s["x"], s["w"], s["tail_pool"], s["state_idx"], bias=s["bias"], activation="silu")
        return {"y": y, "tails": s["tail_pool"]}
    if s["op"] == "gnorm_fwd":
        return {"y": gdn.gated_rmsnorm_fwd(s["x"], s["z"], s["w"], group=s["group"], eps=EPS, first=s["first"])}
    dx, dz, dw = gdn.gated_rmsnorm_bwd(s["x"], s["z"], s["w"], s["dy"], group=s["group"], eps=EPS, first=s["first"])
    return {"dx": dx, "dz": dz, "dw": dw}


def work(case):
    op, e = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op.startswith("gnorm"):
        n = case["T"] * case["D"]
        w = case["group"] if case["shared"] else case["D"]
        # x, z read, y written; in the backward dy read too, dx, dz written
        return {"bytes": n * e * (3 if op == "gnorm_fwd" else 5) + w * (e if op == "gnorm_fwd" else e + 4),
                "flops": n * (12 if op == "gnorm_fwd" else 30)}
    C, pool = case["C"], case["pool"]
    rows = case["B"] if op.endswith("step") else case["T"]
    n = rows * C
    if op == "conv_fwd":
        return {"bytes": 2 * n * e + 3 * C * e * (case["N"] + pool) + 20 * C, "flops": 13 * n}
    if op == "conv_bwd":  # x, dy read, dx written in fp32
        tails = 3 * C * (case["N"] * 4 + pool * (e + 4)) if pool else 0
        return {"bytes": n * (2 * e + 4) + tails + 40 * C, "flops": 35 * n}
    if op == "conv_step":
        return {"bytes": n * e * 8 + 20 * C, "flops": 13 * n}
    S, G, gate = case["S"], case["G"], 1 if case["gate"] else 0
    params = C * (4 * S + 8)
    maps = 2 * rows * G * S * e
    if op == "ssm_fwd":
        return {"bytes": n * e * (3 + gate) + maps + params + 4 * C * S * (case["N"] + pool), "flops": n * (7 * S + 20)}
    if op == "ssm_step":
        return {"bytes": n * e * (3 + gate) + maps + params + 8 * n * S, "flops": n * (7 * S + 20)}
    # x, dt, dout (and z) read, dx, ddt (and dz) written; the maps and their gradients; the parameters and theirs
    states = 4 * C * S * (case["N"] + 2 * pool) if pool else 0
    return {"bytes": n * e * (5 + 2 * gate) + 2 * maps + 2 * params + states, "flops": n * (22 * S + 50)}


# ------------------------------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in prepare(case, seed).items()}
    if case["op"].startswith("gnorm"):
        return _exact_gnorm(case, s)
    if case["op"] == "conv_step":
        i = s["state_idx"].long()
        old = s["tail_pool"][i]
        u = s["bias"] + s["w"][:, 3] * s["x"]
        for m in range(3):
            u = u + s["w"][:, m] * old[:, m]
        s["tail_pool"][i] = torch.stack([old[:, 1], old[:, 2], s["x"]], 1)
        return {"y": u / (1 + (-u).exp()), "tails": s["tail_pool"]}
    if case["op"] in ("conv_fwd", "conv_bwd"):
        return _exact_conv(case, s)
    C, S = case["C"], case["S"]
    group = torch.arange(C, device=s["x"].device) // (C // case["G"])
    delta = torch.log1p(torch.exp(s["dt"] + s["dt_bias"]))
    if case["op"] == "ssm_step":
        i = s["state_idx"].long()
        h = s["state_pool"][i] * (delta.unsqueeze(2) * s["a"]).exp() + torch.einsum(
            "tc,tcs->tcs", delta * s["x"], s["b"][:, group])
        s["state_pool"][i] = h
        y = torch.einsum("tcs,tcs->tc", h, s["c"][:, group]) + s["skip"] * s["x"]
        return {"out": y if s["z"] is None else y * s["z"] / (1 + (-s["z"]).exp()), "states": s["state_pool"]}
    return _exact_scan(case, s, group, delta)


def _exact_scan(case, s, group, delta):
    """The recurrence token by token, all documents abreast (the longest first)."""
    lens, C, S, G = _lengths(case), case["C"], case["S"], case["G"]
    N, T, dev = len(lens), case["T"], delta.device
    order = sorted(range(N), key=lambda i: -lens[i])
    at = torch.tensor([sum(lens[:i]) for i in order], device=dev)
    long = [lens[i] for i in order]
    live, k = [], N
    for j in range(long[0]):
        while long[k - 1] <= j:
            k -= 1
        live.append(k)
    grad = case["op"] == "ssm_bwd"
    idx = [-1] * N if s["init_idx"] is None else s["init_idx"].tolist()
    H = torch.zeros(N, C, S, dtype=torch.float64, device=dev)
    for r, i in enumerate(order):
        if idx[i] >= 0:
            H[r] = s["initial_state"][idx[i]]
    x, a, u = s["x"], s["a"], delta * s["x"]
    y = s["skip"] * x
    seen = torch.empty(T, C, S, dtype=torch.float64, device=dev) if grad else None  # the states before each token
    for j, k in enumerate(live):
        t = at[:k] + j
        if grad:
            seen[t] = H[:k]
        H[:k].mul_((delta[t].unsqueeze(2) * a).exp()).addcmul_(u[t].unsqueeze(2), s["b"][t][:, group])
        y[t] += (H[:k] * s["c"][t][:, group]).sum(2)
    gate = None if s["z"] is None else s["z"] / (1 + (-s["z"]).exp())
    back = torch.empty(N, dtype=torch.long, device=dev)
    back[torch.tensor(order, device=dev)] = torch.arange(N, device=dev)
    if not grad:
        return {"out": y if gate is None else y * gate, "final_state": H[back]}
    out, dy = {}, s["dout"]
    if gate is not None:
        q = 1 / (1 + (-s["z"]).exp())
        out["dz"] = s["dout"] * y * (q + gate * (1 - q))
        dy = s["dout"] * gate
    K = torch.zeros(N, C, S, dtype=torch.float64, device=dev)  # the gradient of the state after the token
    if s["dfinal_state"] is not None:
        K.copy_(s["dfinal_state"][torch.tensor(order, device=dev)])
    dx, ddelta, da = s["skip"] * dy, torch.zeros_like(delta), torch.zeros_like(a)
    db, dc = (torch.zeros(T, G, S, dtype=torch.float64, device=dev) for _ in range(2))
    for j in range(long[0] - 1, -1, -1):
        k = live[j]
        t = at[:k] + j
        e = (delta[t].unsqueeze(2) * a).exp()
        bt, ct = s["b"][t][:, group], s["c"][t][:, group]
        kept = e * seen[t]
        dc[t] = (dy[t].unsqueeze(2) * (kept + u[t].unsqueeze(2) * bt)).view(k, G, -1, S).sum(2)
        K[:k].addcmul_(dy[t].unsqueeze(2), ct)
        db[t] = (K[:k] * u[t].unsqueeze(2)).view(k, G, -1, S).sum(2)
        kb = (K[:k] * bt).sum(2)
        through = K[:k] * kept
        dx[t] += delta[t] * kb
        ddelta[t] = x[t] * kb + (through * a).sum(2)
        da += (through * delta[t].unsqueeze(2)).sum(0)
        K[:k].mul_(e)
    ddt = ddelta / (1 + (-(s["dt"] + s["dt_bias"])).exp())
    out.update(dc=dc, db=db, da=da, dx=dx, ddt=ddt, ddt_bias=ddt.sum(0), dskip=(dy * x).sum(0))
    if s["initial_state"] is not None:
        out["dinit"] = torch.zeros_like(s["initial_state"])
        K = K[back]
        for i, p in enumerate(idx):
            if p >= 0:
                out["dinit"][p] += K[i]
    return out


def _exact_conv(case, s):
    """Document by document."""
    lens, C, dev = _lengths(case), case["C"], s["x"].device
    idx = [-1] * len(lens) if s["init_idx"] is None else s["init_idx"].tolist()
    y, tails, dx = [], [], torch.zeros(case["T"], C, dtype=torch.float64, device=dev)
    dw, dbias = torch.zeros(C, 4, dtype=torch.float64, device=dev), torch.zeros(C, dtype=torch.float64, device=dev)
    dinit = None if s["conv_init"] is None else torch.zeros_like(s["conv_init"])
    t = 0
    for i, n in enumerate(lens):
        start = torch.zeros(3, C, dtype=torch.float64, device=dev) if idx[i] < 0 else s["conv_init"][idx[i]]
        e = torch.cat([start, s["x"][t:t + n]])
        u = s["bias"] + e[0:n] * s["w"][:, 0] + e[1:n + 1] * s["w"][:, 1] + e[2:n + 2] * s["w"][:, 2] + e[3:n + 3] * s["w"][:, 3]
        if case["op"] == "conv_fwd":
            y.append(u / (1 + (-u).exp()))
            tails.append(e[n:])
        else:
            p = 1 / (1 + (-u).exp())
            du = s["dy"][t:t + n] * (p + u * p * (1 - p))
            de = torch.zeros_like(e)
            for m in range(4):
                de[m:m + n] += du * s["w"][:, m]
                dw[:, m] += (du * e[m:m + n]).sum(0)
            dbias += du.sum(0)
            if s["dfinal_tail"] is not None:
                de[n:] += s["dfinal_tail"][i]
            dx[t:t + n] = de[3:]
            if idx[i] >= 0:
                dinit[idx[i]] += de[:3]
        t += n
    if case["op"] == "conv_fwd":
        return {"y": torch.cat(y), "final_tail": torch.stack(tails)}
    out = {"dx": dx, "dw": dw, "dbias": dbias}
    return out if dinit is None else {**out, "dconv_init": dinit}


def _exact_gnorm(case, s):
    T, n, norm_first = case["T"], case["group"], case["first"] == "norm"
    x, z = s["x"].view(T, -1, n), s["z"].view(T, -1, n)
    w = s["w"].view(-1, n)
    p = 1 / (1 + (-z).exp())
    gate = z * p
    u = x if norm_first else x * gate
    ms = (u * u).sum(2, keepdim=True) / n + EPS
    if case["op"] == "gnorm_fwd":
        y = w * u / ms.sqrt()
        return {"y": (y * gate if norm_first else y).reshape(T, -1)}
    dy = s["dy"].view(T, -1, n)
    dn = dy * gate if norm_first else dy
    du = (w * dn - u * (u * w * dn).sum(2, keepdim=True) / (n * ms)) / ms.sqrt()
    slope = p + gate * (1 - p)
    dz = dy * w * u / ms.sqrt() * slope if norm_first else du * x * slope
    dw = (dn * u / ms.sqrt()).sum(0)
    return {"dx": (du if norm_first else du * gate).reshape(T, -1), "dz": dz.reshape(T, -1),
            "dw": dw.sum(0) if case["shared"] else dw.reshape(-1)}
