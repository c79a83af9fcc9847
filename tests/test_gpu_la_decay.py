"""Decayed linear attention over long documents whose earlier tokens still count although their decay is deep: the
values fall as fast as the state does, so that every token of a period has the same weight in the state at its end.
GPU only, against the quadratic form in fp64.

Tolerance: a row carries the roundings of tests/test_gpu_la.py (2.9e-3 of it in the 2-norm, over its 128 elements);
bound 1e-2 of each row's norm. States 1e-5 of their norm."""
import numpy as np
import pytest

from tests import la_quad, la_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from tests.test_gpu_la import SCALE, run_bwd, run_fwd, to_dev  # noqa: E402


def falling(x, g, period, rev):
    """x [T, H, 128], token t of head h multiplied by exp(g_h (t mod period_h)); from the end if rev."""
    t = np.arange(len(x))[::-1] if rev else np.arange(len(x))
    return la_ref.bf16(x * np.exp(g[None] * (t[:, None] % period[None]))[:, :, None])


def rows_near(name, got, ref):
    off = (got.double() - ref).norm(dim=2) / ref.norm(dim=2)
    assert bool((off <= 1e-2).all()), f"{name}: rows {(off > 1e-2).nonzero()[:4].tolist()}, error {float(off.max()):.3e}"


@pytest.mark.parametrize("which", ["v", "do"])  # not both at once: their products would leave fp32's range
def test_tokens_behind_a_deep_decay_still_count(which):
    T, H = 16384, 8
    g = np.where(np.arange(H) % 2 == 0, -0.12, -0.06).astype(np.float32).astype(np.float64)
    period = np.where(np.arange(H) % 2 == 0, 500, 1000)  # 60 e-folds to a period
    p = la_ref.problem(21, [T], H, H, g)
    p[which] = falling(p[which], g, period, which == "do")
    d = to_dev(p)
    ref = la_quad.packed(d, [T], None, SCALE)
    out, fin = run_fwd(d)
    rows_near("out", out, ref["out"])
    for h in range(H):
        assert float((fin[0, h].double() - ref["fin"][0, h]).norm() / ref["fin"][0, h].norm()) <= 1e-5
    r = run_bwd(d)
    for name, x in (("dq", "dqh"), ("dk", "dkh"), ("dv", "dv")):
        rows_near(name, r[name], ref[x])
