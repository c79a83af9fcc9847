"""Decayed linear attention and the norm as a program calls them: captured in a CUDA graph, one workspace for calls of
different layouts, and a batch whose planner works in several passes. GPU only; tolerances as in
tests/test_gpu_la.py."""
import numpy as np
import pytest

from tests import la_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402
from tests.test_gpu_la import SCALE, near, run_bwd, run_fwd, to_dev  # noqa: E402


def test_captured_in_a_graph():
    lens = [300, 0, 1500, 77]
    d = to_dev(la_ref.problem(11, lens, 2, 4, -0.01, dfin=True))
    T, N = sum(lens), len(lens)
    w = torch.randn(512, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    pool = torch.randn(3, 4, 128, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    idx = torch.tensor([2, 0], dtype=torch.int32, device="cuda")

    def block(state):
        out, fin = gdn.la_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], scale=SCALE)
        g = gdn.la_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["do"], d["dfin"], scale=SCALE)
        y, h, _ = gdn.rmsnorm_fwd(out.view(T, 512), w, residual=d["v"].view(T, 512))
        dx, dw = gdn.rmsnorm_bwd(h, w, y)
        o = gdn.la_decode_step(d["q"][:2], d["k"][:2], d["v"][:2], d["g"], state, idx)
        return [out, fin, g["dq"], g["dk"], g["dv"], y, h, dx, dw, o, state]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(pool.clone())  # attributes are set and the allocator is warm before the capture
    torch.cuda.current_stream().wait_stream(side)
    state = pool.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(state)
    for turn in range(2):
        d["q"].mul_(-1), d["v"].add_(turn)  # other values in the captured places
        want = block(pool.clone())
        state.copy_(pool)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_one_workspace_for_other_layouts():
    calls = [([1500, 40, 1100], 1, 2, None), ([5], 1, 1, None), ([260, 130, 0, 400], 1, 2, [-1, 0, 1, -1])]
    sizes = [gdn.la_workspace_size(len(n), sum(n), hk, hv, idx is not None, True) for n, hk, hv, idx in calls]
    ws = torch.full((max(sizes),), 255, dtype=torch.uint8, device="cuda")
    for lens, hk, hv, idx in calls * 2:
        d = to_dev(la_ref.problem(sum(lens), lens, hk, hv, -0.003, dfin=True))
        x = None if idx is None else torch.tensor(idx, dtype=torch.int32, device="cuda")
        want, want_fin = run_fwd(d, idx)
        want_g = run_bwd(d, idx)
        out, fin = gdn.la_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], x, scale=SCALE, workspace=ws)
        g = gdn.la_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["do"], d["dfin"], x, scale=SCALE, workspace=ws)
        assert torch.equal(out, want) and torch.equal(fin, want_fin)
        assert all(torch.equal(g[n], want_g[n]) for n in ("dq", "dk", "dv"))


def test_many_documents_with_a_long_one_and_forks():
    lens = [int(n) for n in np.random.default_rng(6).integers(0, 4, 1100)]
    lens[700] = 4000
    idx = [-1] * 1100
    idx[3] = 0  # the pool's entry; then forks of the first document, of the long one, and of its fork
    idx[20], idx[701], idx[1099] = 1 + 0, 1 + 700, 1 + 701
    p = la_ref.problem(7, lens, 1, 2, [-0.002, -0.2], n_pool=1, dfin=True)
    d = to_dev(p)
    a = (p["q"], p["k"], p["v"], p["g"], p["lens"])
    out, fin = run_fwd(d, idx)
    ref_out, ref_fin, _ = la_ref.la_fwd(*a, idx=idx, pool=p["pool"], scale=SCALE)
    near("out", out, ref_out)
    near("final", fin, ref_fin, states=True)
    g = run_bwd(d, idx)
    ref = la_ref.la_bwd(*a, p["do"], p["dfin"], idx=idx, pool=p["pool"], scale=SCALE)
    for name, x in zip(("dq", "dk", "dv", "dinit"), ref):
        near(name, g[name], x, states=name == "dinit")
