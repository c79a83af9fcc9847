"""A decay that is NaN reaches every output of its head, in the chunked form as in the step, and no other head."""
import pytest

from tests import la_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402
from tests.test_gpu_la import run_bwd, run_fwd, to_dev  # noqa: E402


@pytest.mark.parametrize("lens,idx", [([130, 40], None), ([3000, 1, 200], [0, -1, 1]), ([70, 300], [0, 1])])
def test_nan_decay_is_seen(lens, idx):
    p = la_ref.problem(41, lens, 2, 2, [-0.05, -0.3], n_pool=1, dfin=True)
    d = to_dev(p)
    (out, fin), g = run_fwd(d, idx), run_bwd(d, idx)
    d["g"] = torch.tensor([float("nan"), -0.3], device="cuda")
    (out2, fin2), g2 = run_fwd(d, idx), run_bwd(d, idx)
    pairs = [(out, out2), (fin, fin2), (g["dq"], g2["dq"]), (g["dk"], g2["dk"]), (g["dv"], g2["dv"])]
    if idx is not None:
        pairs.append((g["dinit"], g2["dinit"]))
    for clean, got in pairs:
        assert bool(torch.isnan(got[:, 0]).all()) and torch.equal(got[:, 1], clean[:, 1])
    pool = d["pool"].clone()
    o = gdn.la_decode_step(d["q"][:1], d["k"][:1], d["v"][:1], d["g"], pool, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert bool(torch.isnan(o[:, 0]).all()) and bool(torch.isnan(pool[0, 0]).all()) and not bool(torch.isnan(pool[0, 1]).any())


def test_empty_documents_hand_states_on_all_the_same():
    p = la_ref.problem(42, [0, 0], 1, 1, -0.1, n_pool=1, dfin=True)
    d = to_dev(p)
    d["g"] = torch.full((1,), float("nan"), device="cuda")
    for idx in ([0, -1], [0, 1]):  # the second forks the first
        _, fin = run_fwd(d, idx)
        g = run_bwd(d, idx)
        fork = idx[1] == 1
        assert torch.equal(fin[0], d["pool"][0]) and torch.equal(fin[1], fin[0] if fork else torch.zeros_like(fin[1]))
        assert torch.equal(g["dinit"][0], d["dfin"].sum(0) if fork else d["dfin"][0])
