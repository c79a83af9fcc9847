"""The example block: its gradients against autograd of the same block in fp64, and its token-by-token form
against the packed one. Tolerances: a dozen roundings to bf16 (relative root mean square at most 1.7e-3 each)
lie between the inputs and a gradient: sqrt(12) 1.7e-3 = 6e-3, bound 1e-2; the two forms of the attention share
all roundings but three of the attention's own and the output's: bound 5e-3."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from examples import decay_block  # noqa: E402


def reference(block, x, residual, lens):
    """The block in fp64 with autograd: (out, leaves)."""
    leaf = {n: getattr(block, n).double().requires_grad_() for n in ("norm", "w_in", "w_out")}
    leaf["x"] = x.double().requires_grad_()
    h = leaf["x"] + residual.double()
    y = h * leaf["norm"] * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6)
    qkv = (y @ leaf["w_in"]).view(len(x), -1, 128)
    Hk, Hv = block.Hk, block.Hv
    q, k = (t.repeat_interleave(Hv // Hk, dim=1) for t in (qkv[:, :Hk], qkv[:, Hk:2 * Hk]))
    out, t0 = [], 0
    for n in lens:
        s = slice(t0, t0 + n)
        gap = torch.arange(n, device="cuda")[:, None] - torch.arange(n, device="cuda")[None]
        m = torch.where(gap >= 0, torch.exp(block.log_decay.double()[:, None, None] * gap.clamp(min=0)), 0.0)
        p = torch.einsum("thd,shd->hts", q[s], k[s]) * m * block.scale
        out.append(torch.einsum("hts,shd->thd", p, qkv[s, 2 * Hk:]))
        t0 += n
    return torch.cat(out).flatten(1) @ leaf["w_out"], leaf


def test_gradients_of_the_block():
    torch.manual_seed(1)
    lens = [150, 1, 37]
    block = decay_block.DecayBlock(256, 2, 4, seed=3)
    x, r, do = (torch.randn(sum(lens), 256, device="cuda").to(torch.bfloat16) for _ in range(3))
    cu = torch.tensor([0, 150, 151, 188], dtype=torch.int32, device="cuda")
    out, h, _, saved = block.forward(x, r, cu)
    g = block.backward(saved, do)
    ref, leaf = reference(block, x, r, lens)
    ref.backward(do.double())
    for name, got, want in [("out", out, ref.detach())] + [(n, g[n], leaf[n].grad) for n in ("w_out", "w_in", "norm", "x")]:
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= 1e-2, (name, rel)
    assert torch.equal(h, x + r)


def test_example_trains_and_continues_token_by_token():
    losses, off = decay_block.main()
    assert all(b < a for a, b in zip(losses, losses[1:])) and off <= 5e-3
