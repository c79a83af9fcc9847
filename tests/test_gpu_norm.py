"""Root-mean-square norm with the residual's addition, and its backward, against the fp64 definition
(tests/la_ref.py). Tolerances: a bf16 or fp16 output is one rounding of an fp32 value (half a unit in the
last place, plus 1e-5 relative for the fp32 sums); fp32 outputs 1e-5 of the row's (dw: the column's)
largest term; an e4m3 value is within half a unit (2^-4 of itself, 2^-10 at least) of the scaled value."""
import numpy as np
import pytest

from tests import la_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0}
SIZES = [(1, 1), (3, 7), (5, 64), (9, 130), (4, 256), (2, 513), (6, 1000), (1, 1024), (3, 1025), (2, 2048), (2, 5003),
         (3, 8192), (1, 12345), (1, 32768)]


def inputs(seed, T, D, dtype, n, wdtype=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = [torch.randn((T, D), generator=gen, device="cuda").mul_(1 + 2 * i).to(dtype) for i in range(n)]
    w = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(wdtype or dtype)
    return t, w


def f64(x):
    return x.double().cpu().numpy()


def close(got, ref, dtype, name, terms=None):
    scale = np.abs(ref if terms is None else terms).max(1, keepdims=True)
    tiny = 2.0 ** -24 if dtype == torch.float16 else 0.0  # half the smallest fp16 value
    bound = HALF_ULP[dtype] * np.abs(ref) + 1e-5 * scale + tiny
    assert (np.abs(f64(got) - ref) <= bound).all(), f"{name}: {np.abs(f64(got) - ref).max()}"


@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_forward(T, D, dtype):
    dt = TYPES[dtype]
    (x, r), w = inputs(T * 100003 + D, T, D, dt, 2)
    for res in (None, r):
        y, h, sc = gdn.rmsnorm_fwd(x, w, residual=res, eps=1e-5)
        ry, rh = la_ref.rms_fwd(f64(x), f64(w), None if res is None else f64(res), 1e-5)
        assert y.dtype == dt and sc is None
        close(y, ry, dt, "y")
        if res is None:
            assert h is None
        else:
            close(h, rh, dt, "h")


@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("quant", ["row", "group"])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_forward_in_8_bits(T, D, quant, dtype):
    dt = TYPES[dtype]
    (x, r), w = inputs(T * 100003 + D + 1, T, D, dt, 2)
    x[0, :min(D, 130)] = 0  # a group of zeros where D has two
    r[0, :min(D, 130)] = 0
    y, h, sc = gdn.rmsnorm_fwd(x, w, residual=r, quant=quant)
    ry, _ = la_ref.rms_fwd(f64(x), f64(w), f64(r))
    width = D if quant == "row" else 128
    groups = -(-D // width)
    assert y.dtype == torch.float8_e4m3fn and sc.shape == (T, groups)
    pad = np.pad(ry, ((0, 0), (0, groups * width - D))).reshape(T, groups, width)
    amax = np.abs(pad).max(2)
    rs = np.where(amax > 0, amax / 448, 1.0)
    assert (np.abs(f64(sc) - rs) <= 1e-5 * rs).all()
    scaled = (pad / rs[:, :, None]).reshape(T, -1)[:, :D]
    assert (np.abs(f64(y.float()) - scaled) <= (2.0 ** -4 + 1e-4) * np.abs(scaled) + 2.0 ** -10 + 1e-5).all()


@pytest.mark.parametrize("T,D", SIZES + [(3000, 192), (700, 2056)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_backward(T, D, dtype):
    dt = TYPES[dtype]
    (h, dy, dh), w = inputs(T * 100003 + D + 2, T, D, dt, 3)
    for e in (None, dh):
        dx, dw = gdn.rmsnorm_bwd(h, w, dy, dh=e, eps=1e-5)
        rx, rw = la_ref.rms_bwd(f64(h), f64(w), f64(dy), None if e is None else f64(e), 1e-5)
        rs = 1 / np.sqrt((f64(h) ** 2).mean(1, keepdims=True) + 1e-5)
        close(dx, rx, dt, "dx", terms=rs * f64(w) * f64(dy))
        terms = np.abs(f64(dy) * f64(h) * rs).sum(0)
        assert dw.dtype == torch.float32 and (np.abs(f64(dw) - rw) <= 1e-5 * terms + 1e-30).all()


def test_views_off_alignment_and_mixed_weight_types():
    """Rows that start off a 16-byte boundary take the narrow path and give the same values."""
    for dt, wdt in ((torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16), (torch.float16, torch.float32)):
        (x, r), w = inputs(77, 4, 1024, dt, 2, wdt)
        shift = lambda t: torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)  # noqa: E731
        a = gdn.rmsnorm_fwd(x, w, residual=r, quant="group")
        b = gdn.rmsnorm_fwd(shift(x), shift(w), residual=shift(r), quant="group")
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
        c, d = gdn.rmsnorm_bwd(x, w, r), gdn.rmsnorm_bwd(shift(x), shift(w), shift(r))
        assert torch.equal(c[0], d[0]) and torch.equal(c[1], d[1])


def test_in_place_and_same_bits_on_another_stream():
    (x, r, dy), w = inputs(78, 33, 2048, torch.bfloat16, 3)
    y, h, _ = gdn.rmsnorm_fwd(x, w, residual=r)
    r2, x2 = r.clone(), x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2, h2, _ = gdn.rmsnorm_fwd(x2, w, residual=r2, residual_out=r2, y=x2)
    side.synchronize()
    assert h2 is r2 and y2 is x2 and torch.equal(y, y2) and torch.equal(h, h2)
    dx, dw = gdn.rmsnorm_bwd(h, w, dy, dh=r)
    keep = r.clone()
    dx2, dw2 = gdn.rmsnorm_bwd(h, w, dy, dh=keep, dx=keep)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_non_finite_rows_and_zero_rows():
    (x, r), w = inputs(79, 5, 300, torch.bfloat16, 2)
    x[1, 7], x[3, 250] = float("nan"), float("inf")
    x[4], r[4] = 0, 0
    for quant in (None, "row", "group"):
        y, h, sc = gdn.rmsnorm_fwd(x, w, residual=r, quant=quant)
        y, ok = y.float(), gdn.rmsnorm_fwd(x[[0, 2, 4]].contiguous(), w, residual=r[[0, 2, 4]].contiguous(), quant=quant)
        assert torch.equal(y[[0, 2, 4]], ok[0].float()) and not y[4].any() and bool(torch.isnan(y[1]).all())
        assert bool(torch.isnan(y[3, 250])) and not bool(torch.isnan(y[3, :128]).any())
    assert bool((sc[4] == 1).all())


def test_no_rows_and_refusals():
    (x, r), w = inputs(80, 4, 64, torch.bfloat16, 2)
    y, h, sc = gdn.rmsnorm_fwd(x[:0], w, residual=r[:0], quant="row")
    assert y.shape == (0, 64) and sc.shape == (0, 1)
    dx, dw = gdn.rmsnorm_bwd(x[:0], w, r[:0])
    assert dx.shape == (0, 64) and not dw.any()
    for kw in (dict(x=x.double()), dict(x=x.t()), dict(w=w[:63]), dict(residual=r.float()), dict(residual=r[:3]),
               dict(quant="tile"), dict(y=torch.empty_like(x), quant="row"), dict(scales=torch.empty(4, 1, device="cuda")),
               dict(residual_out=torch.empty_like(x))):
        with pytest.raises(ValueError):
            gdn.rmsnorm_fwd(**(dict(x=x, w=w) | kw))
    with pytest.raises(gdn.GdnError) as e:
        gdn.rmsnorm_fwd(x, w, eps=-1.0)
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    big = torch.zeros((1, 32776), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gdn.GdnError) as e:
        gdn.rmsnorm_fwd(big, big[0])
    assert e.value.status == gdn.GDN_ERR_UNSUPPORTED
    with pytest.raises(gdn.GdnError) as e:
        gdn.rmsnorm_bwd(x, w, r, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == gdn.GDN_ERR_WORKSPACE
