"""Decayed linear attention, every head by itself: heads of slow and of strong decay differ in size, so one norm over
all of them would hide an error in the small ones. Cut documents with eight heads over two, 64 heads, the
planner's longer segments, a decay above zero. GPU only, against the quadratic form in fp64 (tests/la_quad.py);
tolerances as in tests/test_gpu_la.py, a head at a time (dq and dk: a key head at a time)."""
import numpy as np
import pytest

from tests import la_quad, la_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from tests.test_gpu_la import SCALE, near, run_bwd, run_fwd, to_dev  # noqa: E402


def slopes(H):
    return -np.exp2(-8.0 * (np.arange(H) + 1) / H)


def retention(H):
    return np.log1p(-np.exp2(-5.0 - 7.0 * np.arange(H) / (H - 1)))


CASES = [([5000, 1300], 2, 8, slopes(8), None, 0), ([9000, 3], 2, 8, retention(8), [1, 0], 2),
         ([700, 1, 130], 8, 64, slopes(64), [0, -1, 0], 1), ([16001], 1, 4, slopes(4), None, 0),
         ([300, 40], 1, 2, [0.02, 0.004], [0, -1], 1)]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_each_head_by_itself(i):
    lens, Hk, Hv, g, idx, n_pool = CASES[i]
    p = la_ref.problem(500 + i, lens, Hk, Hv, np.asarray(g).astype(np.float32), n_pool, dfin=True)
    d = to_dev(p)
    ref = la_quad.packed(d, lens, idx, SCALE)
    group = lambda x: x.view(len(x), Hk, Hv // Hk, 128).sum(2)  # noqa: E731
    out, fin = run_fwd(d, idx)
    r = run_bwd(d, idx)
    pairs = [("out", out, ref["out"]), ("final_state", fin, ref["fin"]), ("dv", r["dv"], ref["dv"]),
             ("dq", r["dq"], group(ref["dqh"])), ("dk", r["dk"], group(ref["dkh"]))]
    if n_pool:
        pairs.append(("dinit", r["dinit"], ref["dpool"]))
    for name, got, want in pairs:
        for h in range(want.shape[1]):
            near(f"{name} of head {h}", got[:, h], want[:, h].cpu().numpy(), states=name in ("final_state", "dinit"))
