"""Rows of the RMS norm that are not aligned: they are read and written in whole 16-byte pieces, and nothing
beside the tensor, or of another row, may change for that. GPU only."""
import pytest
import torch

import linear_attention_varlen_gb300 as gdn

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
# rows of one piece and less, of a warp, of several warps and vectors a thread, of the longest kind
SHAPES = [(1, 1), (3, 5), (5, 7), (2, 9), (9, 250), (33, 257), (7, 1023), (5, 2049), (3, 4100), (2, 20001)]


def inside(t, offset):
    """A copy of t that starts `offset` elements into a larger buffer; and the buffer."""
    buf = torch.full((t.numel() + offset + 24,), 77.0, device="cuda").to(t.dtype)
    view = buf[offset:offset + t.numel()].view(t.shape)
    view.copy_(t)
    return view, buf


def around(buf, offset, n):
    return torch.cat([buf[:offset], buf[offset + n:]]).float()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("offset", [1, 3])
def test_in_place_and_nothing_beside(T, D, dtype, offset):
    gen = torch.Generator(device="cuda").manual_seed(T * 131 + D + offset)
    x, r, dy, dh = (torch.randn(T, D, generator=gen, device="cuda").to(dtype) for _ in range(4))
    w = torch.randn(D, generator=gen, device="cuda").to(dtype)
    y0, h0, _ = gdn.rmsnorm_fwd(x, w, r)
    dx0, dw0 = gdn.rmsnorm_bwd(h0, w, dy, dh)
    n = T * D
    xv, xb = inside(x, offset)
    rv, rb = inside(r, offset + 1)
    wv, wb = inside(w, offset)
    y, h, _ = gdn.rmsnorm_fwd(xv, wv, rv, y=xv, residual_out=rv)
    assert torch.equal(y, y0) and torch.equal(h, h0)
    for buf, off in ((xb, offset), (rb, offset + 1)):
        assert (around(buf, off, n) == 77).all()
    for other in ("dy", "dh"):  # dx in the place of either
        gv, gb = inside(dy, offset)
        ev, eb = inside(dh, offset + 1)
        dx, dw = gdn.rmsnorm_bwd(rv, wv, gv, ev, dx=gv if other == "dy" else ev)
        assert torch.equal(dx, dx0) and torch.equal(dw, dw0)
        assert (around(gb, offset, n) == 77).all() and (around(eb, offset + 1, n) == 77).all()
    assert torch.equal(wv, w) and (around(wb, offset, D) == 77).all()


@pytest.mark.parametrize("quant", ["row", "group"])
@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("offset", [1, 6])
def test_bytes_beside_stay(T, D, quant, offset):
    gen = torch.Generator(device="cuda").manual_seed(T * 131 + D + offset)
    x = torch.randn(T, D, generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.randn(D, generator=gen, device="cuda")
    y0, _, s0 = gdn.rmsnorm_fwd(x, w, quant=quant)
    buf = torch.full((T * D + offset + 24,), 77, dtype=torch.uint8, device="cuda")
    y = buf[offset:offset + T * D].view(torch.float8_e4m3fn).view(T, D)
    _, _, s = gdn.rmsnorm_fwd(inside(x, 1)[0], w, quant=quant, y=y)
    assert torch.equal(y.view(torch.uint8), y0.view(torch.uint8)) and torch.equal(s, s0)
    assert (around(buf, offset, T * D) == 77).all()
