"""Decayed linear attention with a tile that never comes (a test hook leaves its copy out): every role's wait gives up
after the limit, the CTA lets its copies and products end and frees its tensor memory, and the host reads
GDN_ERR_TIMEOUT. The GPU stays usable: the next ordinary call gives the bits of one before. Nothing here faults,
traps or hangs the GPU: every wait involved is bounded."""
import time

import pytest

from tests import la_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402
from tests.test_gpu_la import run_bwd, run_fwd, to_dev  # noqa: E402

# a key, query or value tile of the first chunk, one of a later chunk; uncut documents (the output walk alone), a cut
# one and forks (both walks), a decay that takes the extra pass
LAYOUTS = [([200, 77], -0.05, None), ([129, 300], -0.5, [-1, 0]), ([3000], -0.001, None)]


@pytest.mark.parametrize("lens,g,idx", LAYOUTS)
@pytest.mark.parametrize("copy", [1, 2, 3, 5])
def test_tile_that_never_comes(lens, g, idx, copy):
    d = to_dev(la_ref.problem(71, lens, 1, 2, g, dfin=True))
    out, fin = run_fwd(d, idx)
    grads = run_bwd(d, idx)
    x = None if idx is None else torch.tensor(idx, dtype=torch.int32, device="cuda")
    T, N = sum(lens), len(lens)
    for bwd in (False, True):
        ws = torch.zeros(gdn.la_workspace_size(N, T, 1, 2, idx is not None, bwd), dtype=torch.uint8, device="cuda")
        t0 = time.perf_counter()
        with gdn.withheld_copy(copy):
            if bwd:
                gdn.la_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["do"], d["dfin"], x, workspace=ws)
            else:
                gdn.la_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], x, workspace=ws)
        assert gdn.workspace_status(ws) == gdn.GDN_ERR_TIMEOUT
        assert time.perf_counter() - t0 < 10.0
    out2, fin2 = run_fwd(d, idx)
    again = run_bwd(d, idx)
    assert torch.equal(out, out2) and torch.equal(fin, fin2)
    assert all(torch.equal(grads[n], again[n]) for n in ("dq", "dk", "dv"))
