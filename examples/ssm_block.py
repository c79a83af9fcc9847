"""A pre-norm state-space block, trained and then run token by token.

    python examples/ssm_block.py

One block: h = x + residual; y = rmsnorm(h); u, z = one fused projection of y; v = silu(conv(u)); the scan's steps and maps
= a projection of v (the steps through a low rank); s = scan(v); out = gated_rmsnorm(s, z) Wo. Norms, convolution, scan
and their gradients are the library's, the projections torch's matrix products. After a few steps of gradient descent
the block answers a prompt in one call and goes on one token at a time from the tail and the state that the prompt
left.
"""
from __future__ import annotations

import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import linear_attention_varlen_gb300 as gdn  # noqa: E402


class ScanBlock:
    # what is learned in the projections' type, and what in fp32
    PROJECTIONS, PARAMETERS = ("norm", "w_in", "w_map", "w_dt", "gate_norm", "w_out"), ("conv_w", "conv_b", "a", "skip", "dt_bias")

    def __init__(self, width: int, channels: int, states: int = 16, rank: int = 16, dtype=torch.bfloat16, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.C, self.S, self.rank = channels, states, rank

        def normal(*shape, by):
            return torch.randn(*shape, generator=gen, device="cuda").mul_(by)
        self.norm = torch.ones(width, dtype=dtype, device="cuda")
        self.gate_norm = torch.ones(channels, dtype=dtype, device="cuda")
        self.w_in = normal(width, 2 * channels, by=width ** -0.5).to(dtype)
        self.w_map = normal(channels, rank + 2 * states, by=channels ** -0.5).to(dtype)
        self.w_dt = normal(rank, channels, by=0.5 * rank ** -0.5).to(dtype)
        self.w_out = normal(channels, width, by=channels ** -0.5).to(dtype)
        self.conv_w, self.conv_b = normal(channels, 4, by=0.5), normal(channels, by=0.1)
        self.a = -torch.arange(1, states + 1, device="cuda").float().repeat(channels, 1)
        self.skip = torch.ones(channels, device="cuda")
        steps = torch.exp(torch.rand(channels, generator=gen, device="cuda") * math.log(100.0) + math.log(1e-3))
        self.dt_bias = torch.log(torch.expm1(steps))

    def _maps(self, v):
        """The scan's inputs beside v: steps, and the two maps as views into their projection."""
        m = v @ self.w_map
        r, S = self.rank, self.S
        return m, m[:, :r] @ self.w_dt, m[:, r:r + S].unflatten(1, (1, S)), m[:, r + S:].unflatten(1, (1, S))

    def forward(self, x, residual, cu_seqlens):
        """Packed documents: (out, h, final tails and states, what the backward needs)."""
        y, h, _ = gdn.rmsnorm_fwd(x, self.norm, residual=residual)
        uz = y @ self.w_in
        u, z = uz[:, :self.C], uz[:, self.C:]  # views: the library takes tokens that lie apart
        v, tail = gdn.conv_fwd(u, self.conv_w, cu_seqlens, bias=self.conv_b, activation="silu")
        m, dt, b, c = self._maps(v)
        s, state = gdn.ssm_scan_fwd(v, dt, self.a, b, c, cu_seqlens, skip=self.skip, dt_bias=self.dt_bias)
        n = gdn.gated_rmsnorm_fwd(s, z, self.gate_norm, first="gate")
        return n @ self.w_out, h, tail, state, (y, h, u, z, v, m, dt, b, c, s, n, cu_seqlens)

    def backward(self, saved, dout, dh=None):
        """Gradients of all that is learned, and of x (the residual's is the same)."""
        y, h, u, z, v, m, dt, b, c, s, n, cu = saved
        ds, dz, dgate = gdn.gated_rmsnorm_bwd(s, z, self.gate_norm, dout @ self.w_out.t(), first="gate")
        g = gdn.ssm_scan_bwd(v, dt, self.a, b, c, cu, ds, skip=self.skip, dt_bias=self.dt_bias)
        dm = torch.cat([g["ddt"] @ self.w_dt.t(), g["db"].flatten(1), g["dc"].flatten(1)], dim=1)
        dv = g["dx"] + dm @ self.w_map.t()
        k = gdn.conv_bwd(u, self.conv_w, cu, dv, bias=self.conv_b, activation="silu")
        duz = torch.cat([k["dx"].to(dz.dtype), dz], dim=1)
        dx, dnorm = gdn.rmsnorm_bwd(h, self.norm, duz @ self.w_in.t(), dh=dh)
        return dict(x=dx, norm=dnorm, w_in=y.t() @ duz, conv_w=k["dw"], conv_b=k["dbias"], w_map=v.t() @ dm,
                    w_dt=m[:, :self.rank].t() @ g["ddt"], a=g["da"], skip=g["dskip"], dt_bias=g["ddt_bias"],
                    gate_norm=dgate, w_out=n.t() @ dout)

    def step(self, x, residual, tails, states, index):
        """One token of each sequence, in place on the pools of tails and states."""
        y, h, _ = gdn.rmsnorm_fwd(x, self.norm, residual=residual)
        uz = y @ self.w_in
        v = gdn.conv_decode_step(uz[:, :self.C], self.conv_w, tails, index, bias=self.conv_b, activation="silu")
        _, dt, b, c = self._maps(v)
        s = gdn.ssm_decode_step(v, dt, self.a, b, c, states, index, skip=self.skip, dt_bias=self.dt_bias)
        return gdn.gated_rmsnorm_fwd(s, uz[:, self.C:], self.gate_norm, first="gate") @ self.w_out, h


def train(block, x, residual, cu_seqlens, target, steps=8, rate=1e-2):
    """A few steps of gradient descent on the squared error, each as long as `rate` of the weight's norm (halved step by
    step); returns the losses."""
    losses = []
    for i in range(steps):
        out, _, _, _, saved = block.forward(x, residual, cu_seqlens)
        err = out.float() - target.float()
        losses.append(float(err.square().mean()))
        grads = block.backward(saved, (err / err.norm()).to(out.dtype))
        for name in block.PROJECTIONS + block.PARAMETERS:
            w, g = getattr(block, name), grads[name].float()
            w -= (g * (rate * 0.5 ** i * w.float().norm() / g.norm())).to(w.dtype)
    return losses


def main():
    torch.manual_seed(0)
    width, lens = 256, [300, 77, 1, 134]
    block = ScanBlock(width, 512)
    T = sum(lens)
    x, residual, target = (torch.randn(T, width, device="cuda").to(torch.bfloat16) for _ in range(3))
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    losses = train(block, x, residual, cu, target)
    print("losses", " ".join(f"{v:.4f}" for v in losses))

    # the first document but for its last eight tokens as a prompt, then those one at a time
    n, tail = lens[0], 8
    whole = block.forward(x[:n], residual[:n], cu[:2])[0]
    prompt = torch.tensor([0, n - tail], dtype=torch.int32, device="cuda")
    _, _, tails, states, _ = block.forward(x[:n - tail], residual[:n - tail], prompt)
    first = torch.zeros(1, dtype=torch.int32, device="cuda")
    steps = [block.step(x[t:t + 1], residual[t:t + 1], tails, states, first)[0] for t in range(n - tail, n)]
    off = (torch.cat(steps).float() - whole[n - tail:].float()).norm() / whole[n - tail:].float().norm()
    print(f"token by token against the whole document: relative difference {float(off):.1e}")
    return losses, float(off)


if __name__ == "__main__":
    main()
