"""Cases of the decayed linear attention (prompts, gradients, single tokens) and of the root-mean-square
norm with the residual's addition, with their plain forms in 32 bits and their definitions in 64.

Linear attention, per value head h with log-decay g_h <= 0 (lam = exp(g_h), key head h // (Hv // Hk)):
    S_t = lam S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t
per document, from a zero state or an entry of a pool of states. The norm, per row:
    h = x + r,  y = w h / sqrt(mean(h^2) + eps),  y in the inputs' type, or in e4m3 with a scale amax / 448
for each row or each 128 columns.
"""
import math
import random

import torch

own = False

D = 128  # head size, key and value
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # a short prompt on its own: one document, few heads, latency counts
        {"name": "la_fwd_short", "op": "la_fwd", "T": 512, "N": 1, "Hk": 2, "Hv": 2, "decay": "slopes", "pool": 0},
        # a packed training or prefill batch: ragged documents, four value heads to a key head
        {"name": "la_fwd_packed", "op": "la_fwd", "T": 16384, "N": 12, "Hk": 2, "Hv": 8, "decay": "slopes", "pool": 0},
        # continuations of cached prefixes: start states from a pool, an odd total, heads not shared
        {"name": "la_fwd_pool", "op": "la_fwd", "T": 9001, "N": 16, "Hk": 16, "Hv": 16, "decay": "retention", "pool": 3},
        # one long prompt: nothing to run side by side but its own segments
        {"name": "la_fwd_long", "op": "la_fwd", "T": 32768, "N": 1, "Hk": 2, "Hv": 8, "decay": "retention", "pool": 0},
        # gradients of a small fine-tuning batch with learned start states
        {"name": "la_bwd_small", "op": "la_bwd", "T": 1501, "N": 5, "Hk": 4, "Hv": 4, "decay": "retention", "pool": 2},
        # gradients of a long-context step: four documents, shared key heads
        {"name": "la_bwd_long", "op": "la_bwd", "T": 65536, "N": 4, "Hk": 2, "Hv": 8, "decay": "slopes", "pool": 0},
        # one user's next token
        {"name": "la_step_one", "op": "la_step", "B": 1, "Hk": 2, "Hv": 8, "dtype": "bf16", "decay": "slopes", "pool": 4},
        # the next token of a full serving batch
        {"name": "la_step_batch", "op": "la_step", "B": 200, "Hk": 16, "Hv": 64, "dtype": "fp16", "decay": "slopes", "pool": 256},
        # the norm in front of a projection in 8 bits, for a few tokens being decoded
        {"name": "norm_fwd_few", "op": "norm_fwd", "T": 7, "D": 2048, "dtype": "bf16", "residual": True, "quant": "row"},
        # the same for a prompt, scales for each 128 columns
        {"name": "norm_fwd_prompt", "op": "norm_fwd", "T": 16384, "D": 8192, "dtype": "bf16", "residual": True, "quant": "group"},
        # the backward of a small step, at a width that is no multiple of anything
        {"name": "norm_bwd_odd", "op": "norm_bwd", "T": 777, "D": 1001, "dtype": "fp32", "residual": True},
        # the backward of a long-context training step
        {"name": "norm_bwd_long", "op": "norm_bwd", "T": 65536, "D": 1024, "dtype": "bf16", "residual": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["la_fwd", "la_fwd", "la_bwd", "la_bwd", "la_step", "norm_fwd", "norm_fwd", "norm_bwd"])
    if op in ("la_fwd", "la_bwd"):
        Hk = rng.choice([1, 2, 4, 8])
        Hv = Hk * rng.choice([1, 1, 2, 4])
        T = _log_int(rng, 1, min(65536, 262144 // Hv))
        N = _log_int(rng, 1, max(1, min(64, T // 8)))
        return {"op": op, "T": T, "N": N, "Hk": Hk, "Hv": Hv, "decay": rng.choice(["slopes", "retention"]),
                "pool": rng.choice([0, 0, 1, 5])}
    if op == "la_step":
        Hk = rng.choice([1, 2, 4, 8, 16])
        B = _log_int(rng, 1, 192)
        return {"op": op, "B": B, "Hk": Hk, "Hv": Hk * rng.choice([1, 2, 4]), "dtype": rng.choice(["bf16", "fp16"]),
                "decay": rng.choice(["slopes", "retention"]), "pool": B + rng.randrange(0, 17)}
    Dm = _log_int(rng, 64, 8192)
    Dm = rng.choice([Dm, -(-Dm // 8) * 8, -(-Dm // 128) * 128])
    T = _log_int(rng, 1, min(65536, (1 << 26) // Dm))
    case = {"op": op, "T": T, "D": Dm, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "residual": rng.random() < 0.75}
    if op == "norm_fwd":
        case["quant"] = rng.choice(["none", "none", "row", "group"])
    return case


def _lengths(case):
    """Ragged documents: N - 1 cuts at random places, the same for every seed."""
    T, N = case["T"], case["N"]
    r = random.Random(T * 1000003 + N)
    cuts = [0] + sorted(r.randint(0, T) for _ in range(N - 1)) + [T]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _log_decay(case):
    h = torch.arange(case["Hv"], dtype=torch.float64)
    if case["decay"] == "slopes":  # geometric slopes 2^(-8 (h + 1) / Hv)
        g = -torch.exp2(-8.0 * (h + 1) / case["Hv"])
    else:  # 1 - 2^(-5 - h'), h' spread over 0 .. 7
        g = torch.log1p(-torch.exp2(-5.0 - 7.0 * h / max(1, case["Hv"] - 1)))
    return g.float()


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)

    def normal(*shape, dtype=torch.float32, by=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * by).to(dtype)

    s = {"op": case["op"]}
    if case["op"] in ("la_fwd", "la_bwd"):
        T, N, Hk, Hv, pool = (case[x] for x in ("T", "N", "Hk", "Hv", "pool"))
        # queries and keys after their activation, values as projected
        s["q"] = torch.nn.functional.silu(normal(T, Hk, D)).to(torch.bfloat16)
        s["k"] = torch.nn.functional.silu(normal(T, Hk, D)).to(torch.bfloat16)
        s["v"] = normal(T, Hv, D, dtype=torch.bfloat16)
        s["log_decay"] = _log_decay(case).to(dev)
        s["scale"] = D ** -0.5
        cu = [0]
        for n in _lengths(case):
            cu.append(cu[-1] + n)
        s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["initial_state"] = normal(pool, Hv, D, D, by=0.5) if pool else None
        s["init_idx"] = torch.tensor([i % (pool + 1) - 1 for i in range(N)], dtype=torch.int32, device=dev) if pool else None
        if case["op"] == "la_bwd":
            s["dout"] = normal(T, Hv, D, dtype=torch.bfloat16)
            s["dfinal_state"] = normal(N, Hv, D, D, by=0.1) if pool else None
    elif case["op"] == "la_step":
        B, Hk, Hv, pool = (case[x] for x in ("B", "Hk", "Hv", "pool"))
        dt = TYPES[case["dtype"]]
        s["q"] = torch.nn.functional.silu(normal(B, Hk, D)).to(dt)
        s["k"] = torch.nn.functional.silu(normal(B, Hk, D)).to(dt)
        s["v"] = normal(B, Hv, D, dtype=dt)
        s["log_decay"] = _log_decay(case).to(dev)
        s["scale"] = D ** -0.5
        s["state_pool"] = normal(pool, Hv, D, D)
        s["state_idx"] = torch.randperm(pool, generator=gen, device=dev)[:B].to(torch.int32)
    else:
        T, Dm, dt = case["T"], case["D"], TYPES[case["dtype"]]
        s["w"] = (1.0 + normal(Dm, by=0.1)).to(dt)
        s["x"] = normal(T, Dm, dtype=dt)
        s["r"] = normal(T, Dm, dtype=dt, by=3.0) if case["residual"] else None
        s["quant"] = case.get("quant", "none")
        if case["op"] == "norm_bwd":
            s["dy"] = normal(T, Dm, dtype=dt)
    return s


# ------------------------------------------------------------------------------------------------ plain forms

C = 128  # tokens to a block of the plain form


def _blocks(cu, T, rev):
    """Blocks of C tokens of each document, in the order of its time (or from its end): token indices [M, C], which
    of them are tokens, each block's document, place in it and token count."""
    lens = (cu[1:] - cu[:-1]).long()
    N, dev = lens.numel(), cu.device
    upto = torch.cumsum((lens + C - 1) // C, 0)
    M = T // C + N
    c = torch.arange(M, device=dev)
    doc = torch.searchsorted(upto, c, right=True)
    live = doc < N
    doc = doc.clamp(max=N - 1)
    p0 = (c - upto[doc] + (lens[doc] + C - 1) // C) * C
    n = torch.where(live, (lens[doc] - p0).clamp(min=0, max=C), torch.zeros_like(p0))
    i = torch.arange(C, device=dev)
    ok = i[None] < n[:, None]
    pos = p0[:, None] + i[None]
    tok = cu[1:].long()[doc][:, None] - 1 - pos if rev else cu[:-1].long()[doc][:, None] + pos
    return tok.clamp(min=0, max=max(0, T - 1)), ok, doc, p0, n, lens


def _decayed(q, k, v, g, cu, start, rev):
    """sum_{s <= t} lam^(t - s) (q_t . k_s) v_s over each document, and its state's part, heads as v's;
    reversed in time where `rev` (then a token's own step does not decay the start state)."""
    T, H = v.shape[0], v.shape[1]
    own_step = 0 if rev else 1
    tok, ok, doc, p0, n, lens = _blocks(cu, T, rev)
    m = ok[:, :, None, None]
    take = lambda x: torch.where(m, x[tok].float(), 0.0).repeat_interleave(H // x.shape[1], dim=2).transpose(1, 2)  # noqa: E731
    qb, kb, vb = take(q), take(k), take(v)  # [M, H, C, D]
    i = torch.arange(C, device=v.device)
    gap = (i[:, None] - i[None]).float()
    mask = torch.where(gap >= 0, torch.exp(g[:, None, None] * gap.clamp(min=0)), 0.0)
    o = ((qb @ kb.transpose(2, 3)) * mask) @ vb
    left = (n[:, None] - i[None] - own_step).clamp(min=0).float()
    kv = (kb * torch.exp(g[None, :, None] * left[:, None, :])[..., None]).transpose(2, 3) @ vb  # [M, H, D, D]
    between = (p0[:, None] - p0[None] - n[None]).float()
    same = (doc[:, None] == doc[None]) & (p0[:, None] > p0[None]) & (n[None] > 0)
    carry = torch.where(same, torch.exp(g[:, None, None] * between.clamp(min=0)), 0.0)  # [H, M, M]
    S = torch.einsum("hab,bhx->ahx", carry, kv.flatten(2)).unflatten(2, (D, D))
    if start is not None:
        S = S + torch.exp(g[None] * p0[:, None].float())[..., None, None] * start[doc]
    o = o + torch.exp(g[None, :, None] * (i[None, None] + own_step).float())[..., None] * (qb @ S)
    after = (lens[None] - p0[:, None] - n[:, None]).float()
    ends = (doc[:, None] == torch.arange(lens.numel(), device=v.device)[None]) & (n[:, None] > 0)
    last = torch.where(ends, torch.exp(g[:, None, None] * after.clamp(min=0)), 0.0)  # [H, M, N]
    final = torch.einsum("hbn,bhx->nhx", last, kv.flatten(2)).unflatten(2, (D, D))
    if start is not None:
        final = final + torch.exp(g[None] * lens[:, None].float())[..., None, None] * start
    out = torch.zeros(T + 1, H, o.shape[3], device=v.device)
    out[torch.where(ok, tok, T).flatten()] = o.transpose(1, 2).flatten(0, 1)
    return out[:T], final


def _start(s):
    if s["initial_state"] is None:
        return None
    x = s["init_idx"].long()
    return torch.where((x >= 0)[:, None, None, None], s["initial_state"][x.clamp(min=0)], 0.0)


def _heads(x, H):
    return x.repeat_interleave(H // x.shape[1], dim=1)


def _la_fwd(s):
    o, final = _decayed(s["q"], s["k"], s["v"], s["log_decay"], s["cu_seqlens"], _start(s), False)
    return {"out": (o * s["scale"]).to(s["q"].dtype), "final_state": final}


def _la_bwd(s):
    q, k, v, do, g, cu, scale = (s[x] for x in ("q", "k", "v", "dout", "log_decay", "cu_seqlens", "scale"))
    T, Hk, Hv = q.shape[0], q.shape[1], v.shape[1]
    start, dfin = _start(s), s["dfinal_state"]
    t = lambda x: None if x is None else x.transpose(2, 3)  # noqa: E731
    dq, _ = _decayed(do, v, _heads(k, Hv), g, cu, t(start), False)
    sq = q.float() * scale
    dv, dstart = _decayed(_heads(k, Hv), sq, do, g, cu, dfin, True)
    dk, _ = _decayed(v, do, _heads(sq, Hv), g, cu, t(dfin), True)
    group = lambda x: x.view(T, Hk, Hv // Hk, D).sum(2)  # noqa: E731
    out = {"dq": (group(dq) * scale).to(q.dtype), "dk": group(dk).to(q.dtype), "dv": dv.to(q.dtype)}
    if start is not None:
        x = s["init_idx"].long()
        out["dinit"] = torch.zeros_like(s["initial_state"]).index_add_(
            0, x.clamp(min=0), torch.where((x >= 0)[:, None, None, None], dstart, 0.0))
    return out


def _la_step(s):
    x, Hv = s["state_idx"].long(), s["v"].shape[1]
    kv = _heads(s["k"].float(), Hv)[..., None] * s["v"].float()[..., None, :]
    S = torch.exp(s["log_decay"])[None, :, None, None] * s["state_pool"][x] + kv
    s["state_pool"][x] = S
    o = (_heads(s["q"].float(), Hv)[..., None, :] @ S)[..., 0, :]
    return {"out": (o * s["scale"]).to(s["q"].dtype), "states": s["state_pool"]}


def _norm_fwd(s):
    h = s["x"].float() if s["r"] is None else s["x"].float() + s["r"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    res = {} if s["r"] is None else {"h": h.to(s["x"].dtype)}
    if s["quant"] == "none":
        return {**res, "y": y.to(s["x"].dtype)}
    T, Dm = y.shape
    width = Dm if s["quant"] == "row" else 128
    parts = torch.nn.functional.pad(y, (0, -Dm % width)).view(T, -1, width)
    amax = parts.abs().amax(2)
    scales = torch.where(amax > 0, amax / 448.0, 1.0)
    y8 = (parts / scales[..., None]).view(T, -1)[:, :Dm].to(torch.float8_e4m3fn)
    return {**res, "y": y8.contiguous(), "scales": scales}


def _norm_bwd(s):
    # x is the sum that the forward left, r the gradient that reaches it beside the norm's
    h, dy = s["x"].float(), s["dy"].float()
    rs = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    wd = s["w"].float() * dy
    dx = rs * wd - h * (rs ** 3) * (wd * h).mean(1, keepdim=True)
    if s["r"] is not None:
        dx = dx + s["r"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * h * rs).sum(0)}


def run(s):
    if not own:
        return {"la_fwd": _la_fwd, "la_bwd": _la_bwd, "la_step": _la_step, "norm_fwd": _norm_fwd,
                "norm_bwd": _norm_bwd}[s["op"]](s)
    import linear_attention_varlen_gb300 as gdn
    if s["op"] == "la_fwd":
        out, final = gdn.la_chunk_fwd(s["q"], s["k"], s["v"], s["log_decay"], s["cu_seqlens"], s["init_idx"],
                                      s["initial_state"], scale=s["scale"])
        return {"out": out, "final_state": final}
    if s["op"] == "la_bwd":
        g = gdn.la_chunk_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["cu_seqlens"], s["dout"], s["dfinal_state"],
                             s["init_idx"], s["initial_state"], scale=s["scale"])
        return {x: g[x] for x in ("dq", "dk", "dv", "dinit") if g[x] is not None}
    if s["op"] == "la_step":
        out = gdn.la_decode_step(s["q"], s["k"], s["v"], s["log_decay"], s["state_pool"], s["state_idx"], scale=s["scale"])
        return {"out": out, "states": s["state_pool"]}
    if s["op"] == "norm_fwd":
        y, h, scales = gdn.rmsnorm_fwd(s["x"], s["w"], residual=s["r"], eps=EPS, quant=s["quant"])
        return {x: v for x, v in (("h", h), ("y", y), ("scales", scales)) if v is not None}
    dx, dw = gdn.rmsnorm_bwd(s["x"], s["w"], s["dy"], dh=s["r"], eps=EPS)
    return {"dx": dx, "dw": dw}


def work(case):
    if case["op"] in ("la_fwd", "la_bwd"):
        T, N, Hk, Hv, pool = (case[x] for x in ("T", "N", "Hk", "Hv", "pool"))
        state = Hv * D * D * 4
        if case["op"] == "la_fwd":  # q, k, v read, o and the final states written
            return {"bytes": 2 * T * D * (2 * Hk + 2 * Hv) + state * (N + pool), "flops": 4 * D * D * T * Hv}
        moved = 2 * T * D * (4 * Hk + 3 * Hv)  # q, k, v, do read, dq, dk, dv written
        return {"bytes": moved + state * (N + 2 * pool if pool else 0), "flops": 10 * D * D * T * Hv}
    if case["op"] == "la_step":
        B, Hk, Hv = case["B"], case["Hk"], case["Hv"]
        return {"bytes": B * (Hv * D * D * 8 + 2 * D * (2 * Hk + 2 * Hv)), "flops": 5 * D * D * B * Hv}
    T, Dm, e = case["T"], case["D"], 4 if case["dtype"] == "fp32" else 2
    n = T * Dm
    if case["op"] == "norm_fwd":
        groups = {"none": 0, "row": 1, "group": -(-Dm // 128)}[case["quant"]]
        y = n * e if not groups else n + 4 * T * groups
        return {"bytes": n * e * (3 if case["residual"] else 1) + y + Dm * e, "flops": 6 * n}
    return {"bytes": n * e * (4 if case["residual"] else 3) + Dm * (e + 4), "flops": 10 * n}


# ------------------------------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in prepare(case, seed).items()}
    if case["op"] in ("la_fwd", "la_bwd"):
        return _exact_tokens(case, s)
    if case["op"] == "la_step":
        Hv, r = s["v"].shape[1], s["v"].shape[1] // s["k"].shape[1]
        head = torch.arange(Hv, device=s["v"].device) // r
        pool, x = s["state_pool"], s["state_idx"].long()
        pool[x] = pool[x] * s["log_decay"].exp().view(1, -1, 1, 1) + torch.einsum("bhk,bhv->bhkv", s["k"][:, head], s["v"])
        return {"out": s["scale"] * torch.einsum("bhk,bhkv->bhv", s["q"][:, head], pool[x]), "states": pool}
    if case["op"] == "norm_bwd":
        h, w, dy, n = s["x"], s["w"], s["dy"], case["D"]
        ms = (h * h).sum(1, keepdim=True) / n + EPS
        dx = w * dy / ms.sqrt() - h * (h * w * dy).sum(1, keepdim=True) / (n * ms * ms.sqrt())
        return {"dx": dx if s["r"] is None else dx + s["r"], "dw": (h / ms.sqrt() * dy).sum(0)}
    h = s["x"] if s["r"] is None else s["x"] + s["r"]
    y = s["w"] * h / ((h * h).sum(1, keepdim=True) / case["D"] + EPS).sqrt()
    res = {"h": None if s["r"] is None else h}
    if case["quant"] == "none":
        return {**res, "y": y}
    if case["quant"] == "row":
        scales = y.abs().max(1, keepdim=True).values / 448
        return {**res, "y": y / scales, "scales": scales}
    group = torch.arange(case["D"], device=y.device) // 128
    scales = torch.stack([p.abs().max(1).values for p in y.split(128, 1)], 1) / 448
    return {**res, "y": y / scales[:, group], "scales": scales}


def _exact_tokens(case, s):
    """The recurrence token by token, all documents abreast (the longest first)."""
    lens, Hv, Hk, dev = _lengths(case), case["Hv"], case["Hk"], s["v"].device
    N = len(lens)
    order = sorted(range(N), key=lambda i: -lens[i])
    first = [sum(lens[:i]) for i in order]
    long = [lens[i] for i in order]
    head = torch.arange(Hv, device=dev) // (Hv // Hk)
    lam, scale = s["log_decay"].exp().view(1, -1, 1, 1), s["scale"]
    q, k, v = s["q"], s["k"], s["v"]
    S = torch.zeros(N, Hv, D, D, dtype=torch.float64, device=dev)
    idx = [-1] * N if s["init_idx"] is None else s["init_idx"].tolist()
    for a, i in enumerate(order):
        if idx[i] >= 0:
            S[a] = s["initial_state"][idx[i]]
    back = torch.empty(N, dtype=torch.long, device=dev)
    back[torch.tensor(order, device=dev)] = torch.arange(N, device=dev)
    at = torch.tensor(first, device=dev)
    live = [sum(1 for n in long if n > j) for j in range(long[0])] if N < 2 or long[0] < 4096 else None
    if live is None:
        live, a = [0] * long[0], N
        for j in range(long[0]):
            while long[a - 1] <= j:
                a -= 1
            live[j] = a
    grad = case["op"] == "la_bwd"
    o = torch.zeros_like(v) if not grad else None
    dqh = torch.zeros(v.shape[0], Hv, D, dtype=torch.float64, device=dev) if grad else None
    for j, a in enumerate(live):
        t = at[:a] + j
        S[:a].mul_(lam).addcmul_(k[t][:, head].unsqueeze(3), v[t].unsqueeze(2))
        if grad:
            dqh[t] = (S[:a] @ s["dout"][t].unsqueeze(3)).squeeze(3)
        else:
            o[t] = (q[t][:, head].unsqueeze(2) @ S[:a]).squeeze(2)
    if not grad:
        return {"out": o * scale, "final_state": S[back]}
    G = torch.zeros_like(S) if s["dfinal_state"] is None else s["dfinal_state"][torch.tensor(order, device=dev)]
    dv, dkh = torch.zeros_like(v), torch.zeros_like(dqh)
    for j in range(long[0] - 1, -1, -1):
        a = live[j]
        t = at[:a] + j
        G[:a].addcmul_(q[t][:, head].unsqueeze(3) * scale, s["dout"][t].unsqueeze(2))
        dv[t] = (k[t][:, head].unsqueeze(2) @ G[:a]).squeeze(2)
        dkh[t] = (G[:a] @ v[t].unsqueeze(3)).squeeze(3)
        G[:a].mul_(lam)
    shared = lambda x: x.view(-1, Hk, Hv // Hk, D).sum(2)  # noqa: E731
    out = {"dq": shared(dqh) * scale, "dk": shared(dkh), "dv": dv}
    if s["initial_state"] is not None:
        dinit, G = torch.zeros_like(s["initial_state"]), G[back]
        for i, x in enumerate(idx):
            if x >= 0:
                dinit[x] += G[i]
        out["dinit"] = dinit
    return out
