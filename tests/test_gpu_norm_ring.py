"""The norm's backward over so many rows that each team of warps refills its ring of row buffers several times, and
that teams end on different buffers. GPU only, against the formula in fp64; the rows off alignment, which come
without a ring, give the same bits. Tolerances as in tests/test_gpu_norm.py."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402

TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "fp16": (torch.float16, 2.0 ** -11), "fp32": (torch.float32, 0.0)}


def off_alignment(t):
    return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)


# teams of one warp to sixteen; about 2400 rows at a time for one warp, 150 for sixteen
@pytest.mark.parametrize("dtype,T,D", [("bf16", 12003, 1024), ("fp16", 30011, 200), ("bf16", 7001, 2048), ("bf16", 3333, 4096),
                                       ("bf16", 1501, 8192), ("fp16", 701, 16384), ("fp32", 12007, 512), ("fp32", 1499, 4096),
                                       ("fp32", 653, 8192)])
def test_many_rows(dtype, T, D):
    dt, half = TYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    h, dy, dh = (torch.randn(T, D, generator=gen, device="cuda").mul_(1 + i).to(dt) for i in range(3))
    w = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt)
    hd, wd, gd = h.double(), w.double(), dy.double()
    rs = torch.rsqrt(hd.square().mean(1, keepdim=True) + 1e-5)
    rx = rs * wd * gd - hd * rs ** 3 * (wd * gd * hd).mean(1, keepdim=True)
    scale = (rs * wd * gd).abs().amax(1, keepdim=True)
    terms = gd * hd * rs
    rw, bound_w = terms.sum(0), 1e-5 * terms.abs().sum(0)
    tiny = 2.0 ** -24 if dt == torch.float16 else 0.0
    for e in (None, dh):
        dx, dw = gdn.rmsnorm_bwd(h, w, dy, dh=e, eps=1e-5)
        want = rx if e is None else rx + dh.double()
        assert bool(((dx.double() - want).abs() <= half * want.abs() + 1e-5 * scale + tiny).all())
        assert bool(((dw.double() - rw).abs() <= bound_w).all())
        u, v = gdn.rmsnorm_bwd(off_alignment(h), off_alignment(w), off_alignment(dy), dh=e if e is None else off_alignment(e),
                               eps=1e-5)
        assert torch.equal(u, dx) and torch.equal(v, dw)
        for place in (dy, e):  # dx in the place of either
            if place is None:
                continue
            c = place.clone()
            u, v = gdn.rmsnorm_bwd(h, w, c if place is dy else dy, dh=c if place is e else e, dx=c, eps=1e-5)
            assert torch.equal(u, dx) and torch.equal(v, dw)
