"""A pre-norm block of decayed linear attention, trained and then run token by token.

    python examples/decay_block.py

One block: h = x + residual; y = rmsnorm(h); q, k, v = one fused projection of y; a = decayed attention over
the packed documents; out = a Wo; the next block's residual is h. The norm, the attention and their gradients
are the library's, the projections torch's matrix products. After a few steps of gradient descent the block
answers a prompt in one call and goes on one token at a time from the state that the prompt left.
"""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import linear_attention_varlen_gb300 as gdn  # noqa: E402

D_HEAD = 128


class DecayBlock:
    def __init__(self, width: int, Hk: int, Hv: int, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.Hk, self.Hv, self.scale = Hk, Hv, D_HEAD ** -0.5
        self.norm = torch.ones(width, **bf16)
        self.w_in = torch.randn(width, (2 * Hk + Hv) * D_HEAD, generator=gen, device="cuda").mul_(width ** -0.5).to(torch.bfloat16)
        self.w_out = torch.randn(Hv * D_HEAD, width, generator=gen, device="cuda").mul_((Hv * D_HEAD) ** -0.5).to(torch.bfloat16)
        # decays 1 - 2^-5, 1 - 2^-6, ... : constants of the heads
        self.log_decay = torch.log1p(-torch.exp2(-5.0 - torch.arange(Hv, device="cuda", dtype=torch.float32)))

    def _project(self, x, residual):
        y, h, _ = gdn.rmsnorm_fwd(x, self.norm, residual=residual)
        qkv = (y @ self.w_in).view(-1, 2 * self.Hk + self.Hv, D_HEAD)
        # views into the fused projection: the library takes tokens that lie apart
        return y, h, qkv[:, :self.Hk], qkv[:, self.Hk:2 * self.Hk], qkv[:, 2 * self.Hk:]

    def forward(self, x, residual, cu_seqlens, init_idx=None, initial_state=None):
        """Packed documents: (out, h, final states, what the backward needs)."""
        y, h, q, k, v = self._project(x, residual)
        a, state = gdn.la_chunk_fwd(q, k, v, self.log_decay, cu_seqlens, init_idx, initial_state, scale=self.scale)
        return a.flatten(1) @ self.w_out, h, state, (y, h, q, k, v, a, cu_seqlens)

    def backward(self, saved, dout, dh=None):
        """Gradients of the weights and of x (the residual's is the same)."""
        y, h, q, k, v, a, cu_seqlens = saved
        da = (dout @ self.w_out.t()).view(a.shape)
        g = gdn.la_chunk_bwd(q, k, v, self.log_decay, cu_seqlens, da, scale=self.scale)
        dqkv = torch.cat([g["dq"], g["dk"], g["dv"]], dim=1).flatten(1)
        dx, dnorm = gdn.rmsnorm_bwd(h, self.norm, dqkv @ self.w_in.t(), dh=dh)
        return dict(w_out=a.flatten(1).t() @ dout, w_in=y.t() @ dqkv, norm=dnorm, x=dx)

    def step(self, x, residual, state_pool, state_idx):
        """One token of each sequence, in place on the pool of states."""
        _, h, q, k, v = self._project(x, residual)
        a = gdn.la_decode_step(q, k, v, self.log_decay, state_pool, state_idx, scale=self.scale)
        return a.flatten(1) @ self.w_out, h


def train(block, x, residual, cu_seqlens, target, steps=8, rate=2e-2):
    """A few steps of gradient descent on the squared error, each as long as `rate` of the weight's norm (halved
    step by step); returns the losses."""
    losses = []
    for i in range(steps):
        out, _, _, saved = block.forward(x, residual, cu_seqlens)
        err = out.float() - target.float()
        losses.append(float(err.square().mean()))
        grads = block.backward(saved, (err / err.norm()).to(torch.bfloat16))
        for name in ("w_out", "w_in", "norm"):
            w, g = getattr(block, name), grads[name].float()
            w -= (g * (rate * 0.5 ** i * w.float().norm() / g.norm())).to(w.dtype)
    return losses


def main():
    torch.manual_seed(0)
    width, lens = 512, [300, 77, 1, 134]
    block = DecayBlock(width, Hk=2, Hv=4)
    T = sum(lens)
    x, residual, target = (torch.randn(T, width, device="cuda").to(torch.bfloat16) for _ in range(3))
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    losses = train(block, x, residual, cu, target)
    print("losses", " ".join(f"{v:.4f}" for v in losses))

    # the first document but for its last eight tokens as a prompt, then those one at a time
    n, tail = lens[0], 8
    whole, _, _, _ = block.forward(x[:n], residual[:n], cu[:2])
    prompt = torch.tensor([0, n - tail], dtype=torch.int32, device="cuda")
    _, _, states, _ = block.forward(x[:n - tail], residual[:n - tail], prompt)
    first = torch.zeros(1, dtype=torch.int32, device="cuda")
    steps = [block.step(x[t:t + 1], residual[t:t + 1], states, first)[0] for t in range(n - tail, n)]
    off = (torch.cat(steps).float() - whole[n - tail:].float()).norm() / whole[n - tail:].float().norm()
    print(f"token by token against the whole document: relative difference {float(off):.1e}")
    return losses, float(off)


if __name__ == "__main__":
    main()
