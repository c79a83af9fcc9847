"""Selective scan (forward, backward, single tokens) against its fp64 definition (tests/ssm_ref.py).

Tolerances: half a unit of the output's type (eps / 2 of the value; fp16 outputs also half of its smallest value, 2^-25),
and for the fp32 arithmetic behind it 2^-21 of the sum of the terms' absolute values for each rounding in a row. A term
passes one token's step with at most one exponential (2 ulp = 2^-22), its argument's two roundings (2^-23 |arg|, and |arg|
e^-|arg| < 0.37 of what entered) and two roundings of a product and a sum (2^-24 each): together below 2^-21. So LONG + 64
of them, LONG being the tokens of the longest chain of documents, and 64 for the sums over states, channels and segments,
the softplus, the gate and a document's carries. fp32 ends at 2^-126, below which a sigmoid (or an exponential) is 0: it
is off by that much at most, and what it is multiplied with stays below 2^11 in these tests (a gate of 300 by a y of 5, and
an output's gradient): 2^-115 absolute."""
import numpy as np
import pytest

from tests import ssm_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 2.0 ** -21


def near(name, got, ref, terms, roundings):
    assert got is not None, name
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -115
    assert got.shape == ref.shape, name
    err = np.abs(got.double().cpu().numpy() - ref)
    bound = (half * np.abs(ref) + EPS * roundings * terms) * (1 + half) + tiny
    worst = float((err / bound).max()) if err.size else 0.0  # NaN fails
    assert worst <= 1, f"{name}: {worst} of the bound"


def on_gpu(p, dtype, apart=False):
    """The problem on the GPU, and the same with its inputs as the GPU has them, in fp64."""
    d, r = {}, dict(p)
    for k in ("x", "dt", "z", "b", "c", "dout"):
        if p[k] is None:
            d[k] = None
            continue
        t = torch.from_numpy(p[k]).to("cuda", TYPES[dtype])
        r[k] = t.double().cpu().numpy()
        if apart:  # a view into a wider row
            wide = torch.full((t.shape[0], t[0].numel() + 24 + len(d)), 7.0, dtype=t.dtype, device="cuda")
            view = wide[:, 8 + len(d):8 + len(d) + t[0].numel()].unflatten(1, t.shape[1:]) if t.shape[0] else t
            t = view.copy_(t) if t.shape[0] else t
        d[k] = t
    for k in ("a", "skip", "dt_bias", "pool", "dfin"):
        d[k] = None if p[k] is None else torch.from_numpy(p[k]).float().cuda()
        r[k] = None if p[k] is None else d[k].double().cpu().numpy()
    cu = np.concatenate([[0], np.cumsum(p["lens"])])
    d["cu"] = torch.from_numpy(cu).to("cuda", torch.int32)
    return d, r


def int32(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


def run_fwd(d, idx=None, softplus=True, **kw):
    return gdn.ssm_scan_fwd(d["x"], d["dt"], d["a"], d["b"], d["c"], d["cu"], skip=d["skip"], z=d["z"],
                            dt_bias=d["dt_bias"], init_idx=int32(idx), initial_state=d["pool"], dt_softplus=softplus, **kw)


def run_bwd(d, idx=None, softplus=True, **kw):
    return gdn.ssm_scan_bwd(d["x"], d["dt"], d["a"], d["b"], d["c"], d["cu"], d["dout"], dfinal_state=d["dfin"],
                            skip=d["skip"], z=d["z"], dt_bias=d["dt_bias"], init_idx=int32(idx),
                            initial_state=d["pool"], dt_softplus=softplus, **kw)


def chain(lens, idx, n_pool):
    longest = []
    for i, n in enumerate(lens):
        j = -1 if idx is None else idx[i] - n_pool
        longest.append(n + (longest[j] if j >= 0 else 0))
    return max(longest)


def check(p, dtype, idx=None, apart=False, bwd=True, fwd=True):
    d, r = on_gpu(p, dtype, apart)
    q = ssm_ref.terms(r)
    m = ssm_ref.magnitudes(q)
    n = chain(p["lens"], idx, 0 if p["pool"] is None else len(p["pool"])) + 64
    if fwd:
        out, fin = run_fwd(d, idx, p["softplus"])
        ref, _, _, _, rfin = ssm_ref.scan_fwd(q, idx)
        mout, _, _, _, mfin = ssm_ref.scan_fwd(m, idx)
        near("out", out, ref, mout, n)
        near("final", fin, rfin, mfin, n)
    if bwd:
        g = run_bwd(d, idx, p["softplus"])
        ref = ssm_ref.scan_bwd(q, r["dout"], r["dfin"], idx)
        mag = ssm_ref.scan_bwd(m, np.abs(r["dout"]), None if r["dfin"] is None else np.abs(r["dfin"]), idx)
        for key in ("dx", "ddt", "da", "db", "dc"):
            near(key, g[key], ref[key], mag[key], 2 * n)  # a term passes the states forward and their gradients back
        for key, of in (("dz", "z"), ("dskip", "skip"), ("ddt_bias", "dt_bias"), ("dinit", "pool")):
            if p[of] is None:
                assert g[key] is None
            else:
                near(key, g[key], ref[key], mag[key], 2 * n)


SHAPES = [  # C, S, G
    (1, 1, 1), (3, 2, 1), (64, 16, 1), (65, 16, 1), (130, 16, 2), (48, 8, 3), (70, 5, 2), (33, 32, 1), (36, 20, 2),
    (40, 64, 2), (17, 51, 1), (256, 16, 4)]


@pytest.mark.parametrize("C,S,G", SHAPES)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_shapes(C, S, G, dtype):
    check(ssm_ref.problem(C * 101 + S, [37, 0, 1, 90], C, S, G), dtype)


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [63, 64, 65], [0, 0, 3], [4, 8, 1, 0], [400]])
@pytest.mark.parametrize("S", [8, 16, 64])
def test_lengths(lens, S):
    check(ssm_ref.problem(sum(lens) + S, lens, 36, S), "fp32")


@pytest.mark.parametrize("gate,skip,bias,softplus", [(False, True, True, True), (True, False, True, True),
                                                      (True, True, False, True), (False, False, False, False),
                                                      (True, True, True, False)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_parts_left_out(gate, skip, bias, softplus, dtype):
    check(ssm_ref.problem(9, [80, 21], 40, 16, 2, gate, skip, bias, softplus=softplus), dtype)


@pytest.mark.parametrize("idx", [[-1, 0, 1, 1, -1, 0], [2, -1, 3 + 0, 3 + 2, 3 + 1, 3 + 2], [-1, 3, 3, -1, 3 + 3, 2]])
@pytest.mark.parametrize("S", [5, 16])
@pytest.mark.parametrize("dfin", [True, False])
def test_pools_and_forks(idx, S, dfin):
    """Start states from a pool (one entry used twice, one not at all), forks of long, empty and forked documents."""
    check(ssm_ref.problem(17, [150, 70, 0, 9, 1, 33], 40, S, 2, n_pool=3, dfin=dfin), "fp32", idx)


def test_forks_without_a_pool():
    check(ssm_ref.problem(18, [40, 0, 25, 90, 1], 24, 16, dfin=True), "fp32", [-1, 0, 1, 2, 0])


def test_pool_without_indices():
    p = ssm_ref.problem(4, [20, 5], 16, 8, n_pool=2, dfin=True)
    check(p, "fp32")  # every document starts from zero, dinit is zero


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("C,S,G", [(64, 16, 1), (50, 7, 2)])
def test_views_into_wider_rows(dtype, C, S, G):
    check(ssm_ref.problem(8, [50, 3, 20], C, S, G, n_pool=1, dfin=True), dtype, [0, -1, 1 + 0], apart=True)


@pytest.mark.parametrize("lens", [[3000], [1200, 40, 0, 900]])
@pytest.mark.parametrize("S,C", [(16, 70), (64, 12)])
def test_documents_of_many_segments(lens, S, C):
    idx = None if len(lens) == 1 else [0, 1 + 0, 1 + 1, 1 + 0]
    check(ssm_ref.problem(21, lens, C, S, n_pool=1, dfin=True), "fp32", idx)


def test_many_documents():
    lens = [int(n) for n in np.random.default_rng(3).integers(0, 6, 1500)]
    lens[700] = 500
    idx = [-1] * 1500
    idx[5], idx[20], idx[701], idx[1499] = 0, 1 + 3, 1 + 700, 1 + 701
    check(ssm_ref.problem(2, lens, 20, 8, n_pool=1, dfin=True), "fp32", idx)


def test_steep_decays_and_far_steps():
    """exp(dt a) from one that underflows to one that stays at 1, steps of tens and near zero."""
    p = ssm_ref.problem(6, [120, 30], 24, 16)
    p["a"] = -np.geomspace(1e-4, 300.0, 24 * 16).reshape(24, 16)
    p["dt"][::3] += 30.0
    p["dt"][1::3] -= 15.0
    check(p, "fp32")
    p["a"][:] = 0.0  # no decay at all
    check(ssm_ref.problem(6, [64], 24, 16) | {"a": p["a"]}, "fp32")


def test_extreme_gates_keep_their_limits():
    p = ssm_ref.problem(12, [40], 16, 8)
    p["z"][::2] = np.where(np.arange(16) % 2, 300.0, -300.0)
    check(p, "fp32")
    d, _ = on_gpu(p, "bf16")
    d["z"][:] = -float("inf")  # silu(-inf) = 0
    out, _ = run_fwd(d)
    assert (out == 0).all()
    g = run_bwd(d)
    assert all((g[k] == 0).all() for k in ("dx", "ddt", "db", "dc", "da"))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_document_and_channel(value):
    p = ssm_ref.problem(13, [70, 90, 40], 40, 16)
    d, _ = on_gpu(p, "fp32")
    want, wfin = run_fwd(d)
    wg = run_bwd(d)
    d["x"][80, 7] = value
    out, fin = run_fwd(d)
    g = run_bwd(d)
    touched = torch.zeros(200, 40, dtype=torch.bool, device="cuda")
    touched[70:160, 7] = True
    assert torch.equal(out[~touched], want[~touched]) and not torch.isfinite(out[80:160, 7]).any()
    assert torch.equal(out[70:80], want[70:80])  # tokens before it
    assert torch.equal(fin[[0, 2]], wfin[[0, 2]]) and not torch.isfinite(fin[1, 7]).any()
    for k in ("dx", "ddt", "dz"):
        assert torch.equal(g[k][~touched], wg[k][~touched]), k
    for k in ("db", "dc"):
        assert torch.equal(g[k][:70], wg[k][:70]) and torch.equal(g[k][160:], wg[k][160:]), k


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,C,S,G", [(1, 64, 16, 1), (5, 70, 5, 2), (4, 33, 64, 1), (9, 256, 16, 4), (3, 8, 20, 1),
                                     (2, 1, 1, 1), (300, 24, 32, 3)])
def test_single_tokens(dtype, B, C, S, G):
    p = ssm_ref.problem(B + C, [1] * B, C, S, G, n_pool=B + 3)
    d, r = on_gpu(p, dtype, apart=True)
    idx = np.random.default_rng(B).permutation(B + 3)[:B]
    q = ssm_ref.terms(r)
    m = ssm_ref.magnitudes(q)
    before = d["pool"].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gdn.ssm_decode_step(d["x"], d["dt"], d["a"], d["b"], d["c"], d["pool"], int32(idx.tolist()), skip=d["skip"],
                              z=d["z"], dt_bias=d["dt_bias"], status=status)
    ref, _, _, _, fin = ssm_ref.scan_fwd(q, idx)
    mout, _, _, _, mfin = ssm_ref.scan_fwd(m, idx)
    near("out", out, ref, mout, 65)
    near("states", d["pool"][idx], fin, mfin, 65)
    rest = [i for i in range(B + 3) if i not in set(idx.tolist())]
    assert torch.equal(d["pool"][rest], before[rest]) and status.item() == 0


def test_steps_follow_a_prompt():
    """A prompt, then tokens one at a time: the same as the whole document, to the tolerance of either."""
    p = ssm_ref.problem(31, [60], 48, 16, 2)
    d, r = on_gpu(p, "fp32")
    q = ssm_ref.terms(r)
    m = ssm_ref.magnitudes(q)
    cut = {k: (v[:50] if k in ("x", "dt", "z", "b", "c") else v) for k, v in d.items()}
    cut["cu"] = int32([0, 50])
    _, state = run_fwd(cut)
    at = int32([0])
    for t in range(50, 60):
        o = gdn.ssm_decode_step(d["x"][t:t + 1], d["dt"][t:t + 1], d["a"], d["b"][t:t + 1], d["c"][t:t + 1], state, at,
                                skip=d["skip"], z=d["z"][t:t + 1], dt_bias=d["dt_bias"])
        near("out", o, ssm_ref.scan_fwd(q)[0][t:t + 1], ssm_ref.scan_fwd(m)[0][t:t + 1], 60 + 64)
    near("state", state, ssm_ref.scan_fwd(q)[4], ssm_ref.scan_fwd(m)[4], 60 + 64)


def test_step_skips_and_reports_bad_entries():
    p = ssm_ref.problem(2, [1] * 4, 40, 16, n_pool=3)
    d, _ = on_gpu(p, "bf16")
    before = d["pool"].clone()
    for bad in (3, -1, 2 ** 31 - 1):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        d["pool"].copy_(before)
        out = gdn.ssm_decode_step(d["x"], d["dt"], d["a"], d["b"], d["c"], d["pool"], int32([1, bad, 0, 2]), skip=d["skip"],
                                  z=d["z"], dt_bias=d["dt_bias"], status=status)
        assert status.item() == gdn.GDN_ERR_INVALID_ARG and (out[1] == 0).all() and (out[[0, 2, 3]] != 0).any(1).all()
        assert (d["pool"] != before).flatten(1).any(1).all()


@pytest.mark.parametrize("cu,idx", [([0, 9, 5, 20], None), ([1, 5, 9, 20], None), ([0, 5, 9, 21], None),
                                    ([0, 5, 9, 19], None), ([0, 5, 9, 20], [-2, 0, 0]), ([0, 5, 9, 20], [-1, -1, 2 + 2])])
def test_bad_layouts_are_reported(cu, idx):
    p = ssm_ref.problem(1, [5, 4, 11], 16, 8, n_pool=2)
    d, _ = on_gpu(p, "bf16")
    d["cu"] = int32(cu)
    out = torch.full((20, 16), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(gdn.ssm_workspace_size(3, 20, 16, 8, 1, True), dtype=torch.uint8, device="cuda")
    run_fwd(d, idx, out=out, workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_ERR_INVALID_ARG and (out == 3.0).all()
    run_bwd(d, idx, workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_ERR_INVALID_ARG
    d["cu"] = int32([0, 5, 9, 20])
    run_fwd(d, None, workspace=ws)
    assert gdn.workspace_status(ws) == gdn.GDN_OK


def test_the_same_bits_every_time():
    p = ssm_ref.problem(44, [700, 80, 3, 260], 130, 16, 2, n_pool=2, dfin=True)
    d, _ = on_gpu(p, "bf16")
    idx = [0, 2 + 0, 1, 0]
    first, firstg = run_fwd(d, idx), run_bwd(d, idx)
    for _ in range(3):
        again, g = run_fwd(d, idx), run_bwd(d, idx)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        assert all(torch.equal(firstg[k], g[k]) for k in g if g[k] is not None)


def test_no_tokens_at_all():
    p = ssm_ref.problem(3, [0, 0], 12, 8, n_pool=1, dfin=True)
    d, r = on_gpu(p, "bf16")
    out, fin = run_fwd(d, [0, -1])
    assert out.shape == (0, 12) and torch.equal(fin[0], d["pool"][0]) and (fin[1] == 0).all()
    g = run_bwd(d, [0, -1])
    assert torch.equal(g["dinit"][0], d["dfin"][0])
    assert all((g[k] == 0).all() for k in ("da", "dskip", "ddt_bias"))


@pytest.mark.parametrize("T", [1, 33])
def test_nothing_beside_the_outputs_is_written(T):
    p = ssm_ref.problem(T, [T], 35, 12, 1)
    d, _ = on_gpu(p, "bf16")
    guard = 64

    def fenced(shape, dtype):
        n = int(np.prod(shape))
        flat = torch.full((n + 2 * guard,), 5.0, dtype=dtype, device="cuda")
        return flat, flat[guard:guard + n].view(shape)
    shapes = dict(dx=(T, 35), ddt=(T, 35), dz=(T, 35), db=(T, 1, 12), dc=(T, 1, 12))
    flats, grads = {}, {}
    for k, s in shapes.items():
        flats[k], grads[k] = fenced(s, torch.bfloat16)
    for k, s in dict(da=(35, 12), dskip=(35,), ddt_bias=(35,)).items():
        flats[k], grads[k] = fenced(s, torch.float32)
    flats["out"], out = fenced((T, 35), torch.bfloat16)
    flats["fin"], fin = fenced((1, 35, 12), torch.float32)
    run_fwd(d, out=out, final_state=fin)
    run_bwd(d, grads=grads)
    for k, f in flats.items():
        assert (f[:guard] == 5).all() and (f[-guard:] == 5).all(), k
        assert (f[guard:-guard] != 5).all(), k
