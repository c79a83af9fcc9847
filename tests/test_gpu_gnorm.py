"""The norm of groups of columns with its gate, and its backward, against the fp64 definition (tests/ssm_ref.py).
Tolerances: half a unit of the output's type; the fp32 arithmetic behind it 2^-21 of the sum of the terms' absolute
values for each rounding in a row: 16 an element (exponential, reciprocal, root, a handful of products), and for a sum
of n terms log2 of the threads and n / threads in a row, at most 16 + 8 within a group (its half counts, through the
root); dw one for each row."""
import numpy as np
import pytest

from tests import ssm_ref
from tests.test_gpu_ssm import TYPES, near

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402

EPS = 1e-5
SHAPES = [(1, 1, 1), (3, 7, 1), (5, 8, 3), (9, 64, 2), (4, 128, 5), (300, 128, 2), (2, 130, 3), (7, 256, 1), (6, 257, 2),
          (3, 512, 2), (2, 1000, 1), (5, 1024, 1), (3, 2048, 2), (2, 2056, 1), (2, 4096, 1), (1, 5003, 1), (2, 8192, 1),
          (1, 8193, 1), (1, 16384, 1)]  # rows, columns of a group, groups


def inputs(seed, T, D, group, dtype, shared, wdtype=None, apart=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[dtype]

    def rows(by):
        t = torch.randn((T, D), generator=gen, device="cuda").mul_(by).to(dt)
        if apart:
            t = torch.full((T, D + 8 + apart), 9.0, dtype=dt, device="cuda")[:, 8:8 + D].copy_(t)
        return t
    w = (1 + 0.2 * torch.randn(group if shared else D, generator=gen, device="cuda")).to(wdtype or dt)
    return rows(2.0), rows(1.0), w, rows(1.0)


def f64(t):
    return t.double().cpu().numpy()


def check(x, z, w, dy, group, first):
    a = [f64(t) for t in (x, z, w, dy)]
    y = gdn.gated_rmsnorm_fwd(x, z, w, group=group, eps=EPS, first=first)
    ref = ssm_ref.gnorm_fwd(*a[:3], group, EPS, first)
    assert y.dtype == x.dtype
    near("y", y, ref, np.abs(ref), 28)
    got = gdn.gated_rmsnorm_bwd(x, z, w, dy, group=group, eps=EPS, first=first)
    refs, mags = ssm_ref.gnorm_bwd(*a, group, EPS, first)
    assert got[2].shape == w.shape and got[2].dtype == torch.float32
    for name, g, r, m, n in zip(("dx", "dz", "dw"), got, refs, mags, (40, 40, 40 + x.shape[0] * (x.shape[1] // w.numel()))):
        near(name, g, r, m, n)


@pytest.mark.parametrize("T,group,ng", SHAPES)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("first", ["norm", "gate"])
def test_shapes(T, group, ng, dtype, first):
    check(*inputs(T + group, T, group * ng, group, dtype, group % 3 == 0), group, first)


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("wdtype", list(TYPES))
@pytest.mark.parametrize("dtype", list(TYPES))
def test_weights(shared, wdtype, dtype):
    check(*inputs(3, 20, 512, 128, dtype, shared, TYPES[wdtype]), 128, "norm")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("apart", [8, 3])  # rows on 16 bytes and off them
@pytest.mark.parametrize("group", [64, 192])
def test_views_into_wider_rows(dtype, apart, group):
    check(*inputs(5, 9, 384, group, dtype, True, apart=apart), group, "gate")


def test_more_rows_than_teams():
    check(*inputs(6, 20001, 16, 8, "bf16", True), 8, "norm")
    check(*inputs(7, 3001, 1024, 1024, "fp32", True), 1024, "gate")


def test_whole_row_by_default():
    x, z, w, _ = inputs(8, 5, 96, 96, "fp32", True)
    assert torch.equal(gdn.gated_rmsnorm_fwd(x, z, w), gdn.gated_rmsnorm_fwd(x, z, w, group=96))


@pytest.mark.parametrize("first", ["norm", "gate"])
@pytest.mark.parametrize("group", [128, 2048, 16384])
def test_in_place(first, group):
    x, z, w, dy = inputs(9, 6, 16384, group, "bf16", True)
    want = gdn.gated_rmsnorm_fwd(x, z, w, group=group, first=first)
    for t in (x.clone(), z.clone()):
        a, b = (t, z) if torch.equal(t, x) else (x, t)
        assert gdn.gated_rmsnorm_fwd(a, b, w, group=group, first=first, y=t) is t and torch.equal(t, want)
    wx, wz, ww = gdn.gated_rmsnorm_bwd(x, z, w, dy, group=group, first=first)
    a, b = x.clone(), dy.clone()
    gx, gz, gw = gdn.gated_rmsnorm_bwd(a, z, w, b, group=group, first=first, dx=b, dz=a)
    assert torch.equal(gx, wx) and torch.equal(gz, wz) and torch.equal(gw, ww)


def test_rows_and_groups_keep_what_is_not_finite():
    x, z, w, dy = inputs(10, 6, 512, 128, "fp32", True)
    want = gdn.gated_rmsnorm_fwd(x, z, w, group=128)
    x[2, 200] = float("nan")
    got = gdn.gated_rmsnorm_fwd(x, z, w, group=128)
    keep = torch.ones_like(x, dtype=torch.bool)
    keep[2, 128:256] = False
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[~keep]).all()
    z[4] = -float("inf")  # the gate is 0
    assert (gdn.gated_rmsnorm_fwd(x, z, w, group=128)[4] == 0).all()
    assert (gdn.gated_rmsnorm_fwd(x, z, w, group=128, first="gate")[4] == 0).all()  # a group of zeros over sqrt(eps)


def test_the_same_bits_every_time():
    x, z, w, dy = inputs(11, 5000, 1024, 128, "bf16", True)
    first = gdn.gated_rmsnorm_bwd(x, z, w, dy, group=128)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, gdn.gated_rmsnorm_bwd(x, z, w, dy, group=128)))


def test_no_rows():
    x, z, w, dy = inputs(1, 0, 64, 32, "bf16", True)
    assert gdn.gated_rmsnorm_fwd(x, z, w, group=32).shape == (0, 64)
    dx, dz, dw = gdn.gated_rmsnorm_bwd(x, z, w, dy, group=32)
    assert dx.shape == (0, 64) and (dw == 0).all()


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("group", [1, 128])
def test_no_rows_of_more_groups_than_teams(shared, group):
    D = 80000 if group == 1 else 128 * 5000  # 77824 threads to teams of one and of sixteen
    x, z, w, dy = inputs(2, 0, D, group, "bf16", shared)
    ws = torch.full((256 + 4 * D,), 63, dtype=torch.uint8, device="cuda")  # an earlier call's
    dw = torch.full(w.shape, 5.0, device="cuda")
    gdn.gated_rmsnorm_bwd(x, z, w, dy, group=group, workspace=ws, dw=dw)
    assert (dw == 0).all() and gdn.workspace_status(ws) == gdn.GDN_OK
