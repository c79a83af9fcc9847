"""Bounded waits for bulk copies that run out: a test hook leaves one copy out, the wait for it gives up after its limit,
the kernel lets its other copies land, returns, and the host reads GDN_ERR_TIMEOUT from the status word. The GPU stays
usable: the next ordinary call gives the bits of one before. Nothing here faults, traps or hangs the GPU: every wait
involved is bounded."""
import time

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402


def norm_problem(T, D, dtype):
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    h, dy, dh = (torch.randn(T, D, generator=gen, device="cuda").to(dtype) for _ in range(3))
    w = torch.randn(D, generator=gen, device="cuda").to(dtype)
    code = {torch.bfloat16: gdn.DTYPE_BF16, torch.float32: gdn.DTYPE_FP32}[dtype]
    ws = torch.full((gdn.load().gdn_rmsnorm_workspace_size(T, D, code),), 255, dtype=torch.uint8, device="cuda")
    return h, w, dy, dh, ws


# teams of one warp (a first fill, a later refill), of eight, of two; the last row
@pytest.mark.parametrize("T,D,dtype,row", [(40, 1024, torch.bfloat16, 0), (12003, 1024, torch.bfloat16, 9000),
                                           (1501, 8192, torch.bfloat16, 700), (5000, 1024, torch.float32, 4999)])
def test_norm_row_that_never_comes(T, D, dtype, row):
    h, w, dy, dh, ws = norm_problem(T, D, dtype)
    dx, dw = gdn.rmsnorm_bwd(h, w, dy, dh, workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_OK
    t0 = time.perf_counter()
    with gdn.withheld_copy(row + 1):
        lost, _ = gdn.rmsnorm_bwd(h, w, dy, dh, dx=torch.full_like(dx, 77), workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 10.0
    # nothing was made of what had not arrived, and other teams' rows are as ever
    assert bool((lost[row] == 77).all()) and torch.equal(lost[row - 1 if row else 1], dx[row - 1 if row else 1])
    dx2, dw2 = gdn.rmsnorm_bwd(h, w, dy, dh, workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_OK and torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("T,D", [(0, 64), (3, 7), (5, 1024), (2, 20000), (2, 32768)])
def test_norm_status_word_of_every_form(T, D):
    h, w, dy, _, ws = norm_problem(T, D, torch.bfloat16)
    gdn.rmsnorm_bwd(h, w, dy, workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_OK


def test_withholding_is_of_its_block():
    with pytest.raises(gdn.GdnError):
        with gdn.withheld_copy(-1):
            pass
    h, w, dy, dh, ws = norm_problem(33, 512, torch.bfloat16)
    with pytest.raises(KeyError):
        with gdn.withheld_copy(1):
            raise KeyError
    gdn.rmsnorm_bwd(h, w, dy, dh, workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_OK
