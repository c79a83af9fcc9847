"""The example block: norm, convolution, scan, gated norm and their gradients together, against autograd of the same block
in fp64, and its token-by-token form against the packed one.

Tolerances. In fp32 a term of any operator or product passes at most K + 64 roundings of 2^-21 (K = 128 terms of a matrix
product or tokens of a document), eight of them lie between the inputs and a gradient, and forward errors pass on through
the backward once more: 16 (128 + 64) 2^-21 = 1.5e-3 of the terms' size, as a bound on relative norms (terms cancel by less
than errors, which are random, do: neither side is anywhere near it). In bf16 two forms of the block share all roundings
but those of eight tensors (1.7e-3 each, root mean square): sqrt(8) 1.7e-3 = 5e-3, twice that as the bound."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from examples import ssm_block  # noqa: E402


def reference(block, x, residual, lens):
    """The block in fp64 with autograd, token by token: (out, leaves)."""
    leaf = {n: getattr(block, n).double().requires_grad_() for n in block.PROJECTIONS + block.PARAMETERS}
    leaf["x"] = x.double().requires_grad_()
    silu = torch.nn.functional.silu
    rms = lambda u: u * torch.rsqrt(u.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
    uz = (rms(leaf["x"] + residual.double()) * leaf["norm"]) @ leaf["w_in"]
    C, S, r = block.C, block.S, block.rank
    u, z = uz[:, :C], uz[:, C:]
    v, t0 = [], 0
    for n in lens:
        e = torch.cat([torch.zeros(3, C, dtype=torch.float64, device="cuda"), u[t0:t0 + n]])
        v.append(silu(leaf["conv_b"] + sum(leaf["conv_w"][:, k] * e[k:k + n] for k in range(4))))
        t0 += n
    v = torch.cat(v)
    m = v @ leaf["w_map"]
    delta = torch.nn.functional.softplus(m[:, :r] @ leaf["w_dt"] + leaf["dt_bias"])
    b, c = m[:, r:r + S], m[:, r + S:]
    s, t = [], 0
    for n in lens:
        h = torch.zeros(C, S, dtype=torch.float64, device="cuda")
        for t in range(t, t + n):
            h = torch.exp(delta[t][:, None] * leaf["a"]) * h + (delta[t] * v[t])[:, None] * b[t]
            s.append(h @ c[t] + leaf["skip"] * v[t])
        t += 1
    return (rms(torch.stack(s) * silu(z)) * leaf["gate_norm"]) @ leaf["w_out"], leaf


def test_gradients_of_the_block():
    torch.manual_seed(1)
    lens = [60, 1, 37]
    block = ssm_block.ScanBlock(64, 128, states=8, rank=8, dtype=torch.float32, seed=3)
    x, r, do = (torch.randn(sum(lens), 64, device="cuda") for _ in range(3))
    cu = torch.tensor([0, 60, 61, 98], dtype=torch.int32, device="cuda")
    out, h, _, _, saved = block.forward(x, r, cu)
    g = block.backward(saved, do)
    ref, leaf = reference(block, x, r, lens)
    ref.backward(do.double())
    assert set(g) == set(leaf)
    for name, got, want in [("out", out, ref.detach())] + [(n, g[n], leaf[n].grad) for n in leaf]:
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= 1.5e-3, (name, rel)
    assert torch.equal(h, x + r)


def test_example_runs_and_continues_token_by_token():
    losses, off = ssm_block.main()
    assert all(v == v and v < float("inf") for v in losses) and off <= 1e-2
