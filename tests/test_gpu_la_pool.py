"""A pool of more entries than a grid has rows: the gradient of every entry is written."""
import pytest

from tests import la_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402
from tests.test_gpu_la import SCALE, near, run_bwd, run_fwd, to_dev  # noqa: E402


def test_gradients_of_a_large_pool():
    lens, n, used = [40, 3, 129], 65537, [65536, 0, 65536]
    p = la_ref.problem(51, lens, 1, 1, -0.01, n_pool=2, dfin=True)
    d = to_dev(p)
    pool = torch.zeros(n, 1, 128, 128, device="cuda")
    pool[[0, 65536]] = d["pool"]
    d["pool"] = pool
    small = [1, 0, 1]
    out, _ = run_fwd(d, used)
    ro, _, _ = la_ref.la_fwd(p["q"], p["k"], p["v"], p["g"], lens, small, p["pool"], SCALE)
    near("out", out, ro)
    g = run_bwd(d, used)
    ref = la_ref.la_bwd(p["q"], p["k"], p["v"], p["g"], lens, p["do"], p["dfin"], small, p["pool"], SCALE)
    near("dinit", g["dinit"][[0, 65536]], ref[3], states=True)
    assert not bool(g["dinit"][1:65536].any())


def test_more_entries_than_any_grid_are_refused_before_anything_runs():
    p = la_ref.problem(52, [5], 1, 1, -0.01, n_pool=1)
    d = to_dev(p)
    out = {x: torch.full_like(d["q"], 3) for x in ("dq", "dk", "dv")}
    dinit = torch.empty_like(d["pool"])
    ws = torch.empty(gdn.la_workspace_size(1, 5, 1, 1, False, True), dtype=torch.uint8, device="cuda")
    ptr = lambda t: t.data_ptr()  # noqa: E731
    rc = gdn.load().gdn_la_bwd(ptr(d["q"]), ptr(d["k"]), ptr(d["v"]), ptr(d["g"]), ptr(d["cu"]), 1, 5, 1, 1, 128, None, None,
                               ptr(d["pool"]), 1 << 28, SCALE, ptr(d["do"]), None, *(ptr(t) for t in out.values()), ptr(dinit),
                               ptr(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == gdn.GDN_ERR_INVALID_ARG and all(bool((t == 3).all()) for t in out.values())
