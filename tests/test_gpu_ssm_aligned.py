"""The selective scan where every row of every block of channels lies on 16 bytes, for each padded number of states (8, 16,
32, 64), states that fill it and that do not, channels of one block and of several; and its step. Against the fp64
definition with the tolerances that tests/test_gpu_ssm.py derives (none of these has more than 96 channels to a sum).
Aligned views into wider rows go the same way as contiguous tensors, so they give the same bits."""
import numpy as np
import pytest

from tests import ssm_ref
from tests.test_gpu_ssm import TYPES, check, int32, near, on_gpu, run_bwd, run_fwd

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402

SHAPES = [(64, 5, 2), (64, 8, 1), (96, 12, 1), (48, 24, 2), (64, 32, 1), (96, 32, 1), (32, 18, 1), (64, 64, 1), (80, 48, 2),
          (48, 51, 1)]  # C, S, G: channels to a group are a multiple of 8


@pytest.mark.parametrize("C,S,G", SHAPES)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_shapes(C, S, G, dtype):
    check(ssm_ref.problem(C * 103 + S, [37, 0, 1, 90], C, S, G, n_pool=2, dfin=True), dtype, [1, -1, 2 + 0, 0])


@pytest.mark.parametrize("C,S", [(32, 32), (64, 64)])
def test_documents_of_many_segments(C, S):
    check(ssm_ref.problem(23, [1200, 40, 0, 900], C, S, n_pool=1, dfin=True), "bf16", [0, 1 + 0, 1 + 1, 1 + 0])


def aligned_views(d, names):
    """The same tensors as views into rows that lie a multiple of 16 bytes apart, on 16 bytes."""
    v = dict(d)
    for i, k in enumerate(names):
        t = d[k]
        wide = torch.full((t.shape[0], t[0].numel() + 16 + 8 * i), float("nan"), dtype=t.dtype, device="cuda")
        v[k] = wide[:, 8:8 + t[0].numel()].unflatten(1, t.shape[1:]).copy_(t)
        assert not v[k].is_contiguous()
    return v


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("C,S,G", [(64, 8, 1), (64, 16, 2), (64, 32, 1), (64, 64, 1)])
def test_aligned_views(dtype, C, S, G):
    idx = [0, -1, 1 + 0]
    d, _ = on_gpu(ssm_ref.problem(8, [50, 3, 20], C, S, G, n_pool=1, dfin=True), dtype)
    v = aligned_views(d, ("x", "dt", "z", "b", "c", "dout"))
    assert all(torch.equal(a, b) for a, b in zip(run_fwd(d, idx), run_fwd(v, idx)))
    want, got = run_bwd(d, idx), run_bwd(v, idx)
    assert all(torch.equal(want[k], got[k]) for k in want)


STEPS = [(5, 64, 8, 1), (2, 32, 12, 1), (4, 64, 16, 2), (3, 40, 20, 1), (3, 48, 32, 1), (2, 32, 48, 2), (2, 64, 64, 1)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,C,S,G", STEPS)
def test_single_tokens(dtype, B, C, S, G):
    d, r = on_gpu(ssm_ref.problem(B + C, [1] * B, C, S, G, n_pool=B + 2), dtype)
    idx = np.random.default_rng(B).permutation(B + 2)[:B]
    q = ssm_ref.terms(r)
    m = ssm_ref.magnitudes(q)
    pools = [d["pool"].clone(), d["pool"].clone()]
    outs = [gdn.ssm_decode_step(s["x"], s["dt"], s["a"], s["b"], s["c"], p, int32(idx.tolist()), skip=s["skip"], z=s["z"],
                                dt_bias=s["dt_bias"]) for s, p in zip((d, aligned_views(d, ("x", "dt", "z", "b", "c"))), pools)]
    ref, _, _, _, fin = ssm_ref.scan_fwd(q, idx)
    mout, _, _, _, mfin = ssm_ref.scan_fwd(m, idx)
    near("out", outs[0], ref, mout, 65)
    near("states", pools[0][idx], fin, mfin, 65)
    assert torch.equal(outs[0], outs[1]) and torch.equal(pools[0], pools[1])
