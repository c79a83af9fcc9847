"""Decayed linear attention at the ends of its range: large finite values and a long tail of zeros in heads whose
decay within a chunk is deep. GPU only, against the quadratic form in fp64, each head by itself; tolerances as
in tests/test_gpu_la.py (rows: 1e-2 of the row's norm, three times what its roundings come to)."""
import numpy as np
import pytest

from tests import la_quad, la_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from tests.test_gpu_la import SCALE, near, run_bwd, run_fwd, to_dev  # noqa: E402

# e-folds of a 128-token chunk from nothing to far below fp32's range
DECAYS = [0.0, -0.01, -0.1, -0.2, -0.46, -0.5, -0.9, -5.0]


def by_head(got, ref):
    """One key head to a value head: every output of each head against its own reference."""
    for name, x in got.items():
        for h in range(x.shape[1]):
            near(f"{name} of head {h}", x[:, h], ref[name][:, h].cpu().numpy(), states=name in ("fin", "dpool"))


@pytest.mark.parametrize("big", ["v", "qk", "do"])
def test_large_finite_values(big):
    lens, H = [300, 77], len(DECAYS)
    p = la_ref.problem(31, lens, H, H, DECAYS, n_pool=1, dfin=True)
    if big == "v":
        for x in ("v", "pool"):
            p[x] = p[x] * 2.0 ** 90
    elif big == "do":
        for x in ("do", "dfin"):
            p[x] = p[x] * 2.0 ** 90
    else:
        p["q"], p["k"] = p["q"] * 2.0 ** 45, p["k"] * 2.0 ** 45
        p["pool"], p["dfin"] = p["pool"] * 2.0 ** 45, p["dfin"] * 2.0 ** 45
    d = to_dev(p)
    ref = la_quad.packed(d, lens, [0, -1], SCALE)
    out, fin = run_fwd(d, [0, -1])
    by_head(dict(out=out, fin=fin), ref)
    r = run_bwd(d, [0, -1])
    by_head(dict(dqh=r["dq"], dkh=r["dk"], dv=r["dv"], dpool=r["dinit"]), ref)


def test_rows_that_only_the_start_state_reaches():
    """Values of zero (masked padding) after the start: what is left of the state is all that a row holds."""
    lens, H = [200, 90], len(DECAYS)
    p = la_ref.problem(32, lens, H, H, DECAYS, n_pool=1)
    p["v"][:] = 0
    d = to_dev(p)
    ref = la_quad.packed(d, lens, [0, 0], SCALE)["out"]
    out, _ = run_fwd(d, [0, 0])
    off, size = (out.double() - ref).norm(dim=2), ref.norm(dim=2)
    seen = size > 2.0 ** -100  # rows that fp32 holds with room to spare
    assert bool((off[seen] <= 1e-2 * size[seen]).all()), float((off / size)[seen].max())
    assert bool((off[~seen] <= 2.0 ** -100).all()) and int(seen.sum()) > 1500 and int((~seen).sum()) > 100
    assert np.isfinite(out.float().cpu().numpy()).all()
