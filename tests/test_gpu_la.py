"""Decayed linear attention on the GPU against its fp64 definition (tests/la_ref.py).

Tolerances, derived from the roundings: one rounding to bf16 has a relative root-mean-square error of at
most 2^-9 / sqrt(1) ~ 1.7e-3 on such data; out, dq, dk and dv carry three of them (the map, the state the
rows read, the result), independent: sqrt(3) 1.7e-3 = 2.9e-3 in the 2-norm, bound 4e-3. An element: 2^-8 of
itself for its own rounding and eight root-mean-squares of the others, 8 x 2.4e-3 of the tensor's. The
states carry the second bf16 term's rounding, 2^-18 an element, and fp32 sums: bound 1e-5."""
import numpy as np
import pytest

from tests import la_ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402

SCALE = 128 ** -0.5


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), device="cuda")


def to_dev(p):
    d = {k: torch.from_numpy(p[k]).to("cuda", torch.bfloat16) for k in ("q", "k", "v", "do")}
    d |= {k: None if p[k] is None else torch.from_numpy(p[k]).to("cuda", torch.float32) for k in ("g", "pool", "dfin")}
    return d | {"cu": cu_of(p["lens"])}


def near(name, got, ref, states=False):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape and np.isfinite(got).all(), name
    if not ref.size:
        return
    n = np.linalg.norm(ref)
    rel = np.linalg.norm(got - ref) / n if n else np.linalg.norm(got)
    assert rel <= (1e-5 if states else 4e-3), f"{name}: relative error {rel:.3e}"
    if not states:
        bound = 2.0 ** -8 * np.abs(ref) + 8 * 2.4e-3 * np.sqrt((ref ** 2).mean())
        assert (np.abs(got - ref) <= bound).all(), f"{name}: largest error {np.abs(got - ref).max():.3e}"


def run_fwd(d, idx=None, scale=SCALE, **kw):
    x = None if idx is None else torch.tensor(idx, dtype=torch.int32, device="cuda")
    T, Hk, Hv, N = d["q"].shape[0], d["q"].shape[1], d["v"].shape[1], d["cu"].shape[0] - 1
    ws = torch.empty(gdn.la_workspace_size(N, T, Hk, Hv, x is not None), dtype=torch.uint8, device="cuda")
    out, fin = gdn.la_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], x, d["pool"], scale=scale, workspace=ws, **kw)
    assert gdn.workspace_status(ws) == gdn.GDN_OK
    return out, fin


def run_bwd(d, idx=None, scale=SCALE, **kw):
    x = None if idx is None else torch.tensor(idx, dtype=torch.int32, device="cuda")
    T, Hk, Hv, N = d["q"].shape[0], d["q"].shape[1], d["v"].shape[1], d["cu"].shape[0] - 1
    ws = torch.empty(gdn.la_workspace_size(N, T, Hk, Hv, x is not None, True), dtype=torch.uint8, device="cuda")
    g = gdn.la_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["do"], d["dfin"], x, d["pool"], scale=scale,
                         workspace=ws, **kw)
    assert gdn.workspace_status(ws) == gdn.GDN_OK
    return g


SLOW = -np.exp2(-np.arange(4.0) * 2 - 2)
LAYOUTS = [
    ([1], 1, 1, -0.1, None, 0),
    ([2, 1, 3], 1, 2, -0.1, None, 0),
    ([127], 1, 1, -0.01, None, 0),
    ([128], 2, 2, -0.01, None, 0),
    ([129], 1, 4, SLOW, None, 0),
    ([0], 1, 1, -0.5, None, 0),
    ([0, 130, 0, 1, 257, 0], 2, 4, SLOW, None, 0),
    ([300, 700], 1, 2, 0.0, [1, 0], 2),
    # one long document: cut into segments, the scan over them, an odd tail
    ([2601], 1, 1, -0.002, None, 0),
    ([1500, 40, 1100], 1, 2, [-0.0005, -0.3], [0, -1, 0], 1),
    # forks: of an uncut document, of a cut one, of an empty one, of a fork
    ([200, 130, 0, 77, 600, 129], 1, 2, [-0.01, -0.4], [0, 1, 2, 3, -1, 5], 1),
    ([900, 300, 515], 1, 1, -0.001, [-1, 0, 0], 0),
    # row factors below the cut, decays of zero and of everything
    ([400, 3], 1, 4, [-0.47, -0.7, -5.0, -np.inf], None, 0),
    ([260], 1, 2, [-1e9, -60.0], [0], 1),
]


@pytest.mark.parametrize("i", range(len(LAYOUTS)))
def test_forward(i):
    lens, Hk, Hv, g, idx, n_pool = LAYOUTS[i]
    p = la_ref.problem(100 + i, lens, Hk, Hv, g, n_pool)
    out, fin = run_fwd(to_dev(p), idx)
    ro, rf, _ = la_ref.la_fwd(p["q"], p["k"], p["v"], p["g"], lens, idx, p["pool"], SCALE)
    near("out", out, ro)
    near("final_state", fin, rf, states=True)


@pytest.mark.parametrize("i", range(len(LAYOUTS)))
def test_backward(i):
    lens, Hk, Hv, g, idx, n_pool = LAYOUTS[i]
    p = la_ref.problem(200 + i, lens, Hk, Hv, g, n_pool, dfin=i % 2 == 1)
    r = run_bwd(to_dev(p), idx)
    ref = la_ref.la_bwd(p["q"], p["k"], p["v"], p["g"], lens, p["do"], p["dfin"], idx, p["pool"], SCALE)
    for name, x in zip(("dq", "dk", "dv"), ref):
        near(name, r[name], x)
    if n_pool:
        near("dinit", r["dinit"], ref[3], states=True)
    else:
        assert r["dinit"] is None


def test_many_short_documents():
    lens = list(np.random.default_rng(5).integers(0, 4, 1500))
    p = la_ref.problem(300, lens, 1, 1, -0.2)
    d = to_dev(p)
    out, fin = run_fwd(d)
    ro, rf, _ = la_ref.la_fwd(p["q"], p["k"], p["v"], p["g"], lens, scale=SCALE)
    near("out", out, ro)
    near("final_state", fin, rf, states=True)
    r = run_bwd(d)
    for name, x in zip(("dq", "dk", "dv"), la_ref.la_bwd(p["q"], p["k"], p["v"], p["g"], lens, p["do"], scale=SCALE)):
        near(name, r[name], x)


def test_other_documents_nan_and_inf_stay_there():
    """Documents share chunks' tiles: what one holds must not reach its neighbours."""
    lens = [70, 100, 90]
    p = la_ref.problem(301, lens, 1, 2, [-0.05, -0.6])
    d = to_dev(p)
    clean, cfin = run_fwd(d)
    gclean = run_bwd(d)
    for x in ("q", "k", "v", "do"):
        d[x][70:120] = float("nan")
        d[x][120:170] = float("inf")
    out, fin = run_fwd(d)
    g = run_bwd(d)
    for a, b in [(out, clean)] + [(g[x], gclean[x]) for x in ("dq", "dk", "dv")]:
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[170:], b[170:])
    assert torch.equal(fin[0], cfin[0]) and torch.equal(fin[2], cfin[2])


def test_strided_views_of_a_fused_projection():
    p = la_ref.problem(302, [333], 2, 4, SLOW)
    d = to_dev(p)
    fused = torch.empty((333, 2 + 2 + 4, 128), dtype=torch.bfloat16, device="cuda")
    fused[:, :2], fused[:, 2:4], fused[:, 4:] = d["q"], d["k"], d["v"]
    s = d | {"q": fused[:, :2], "k": fused[:, 2:4], "v": fused[:, 4:]}
    assert not s["q"].is_contiguous()
    assert all(torch.equal(a, b) for a, b in zip(run_fwd(d), run_fwd(s)))
    a, b = run_bwd(d), run_bwd(s)
    assert all(torch.equal(a[x], b[x]) for x in ("dq", "dk", "dv"))


def test_same_bits_twice_and_on_another_stream():
    p = la_ref.problem(303, [1200, 300], 1, 4, SLOW, 1, dfin=True)
    d = to_dev(p)
    a, b = run_fwd(d, [0, 1]), run_bwd(d, [0, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c, e = run_fwd(d, [0, 1]), run_bwd(d, [0, 1])
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, c))
    assert all(torch.equal(b[x], e[x]) for x in ("dq", "dk", "dv", "dinit"))


def test_zero_tokens_pass_the_states_through():
    p = la_ref.problem(304, [0, 0], 1, 2, -0.1, 1, dfin=True)
    d = to_dev(p)
    out, fin = run_fwd(d, [0, -1])
    assert out.shape == (0, 2, 128) and torch.equal(fin[0], d["pool"][0]) and not fin[1].any()
    g = run_bwd(d, [0, -1])
    assert torch.equal(g["dinit"][0], d["dfin"][0])


def test_scale_enters_once():
    p = la_ref.problem(305, [260], 1, 1, -0.01, 1, dfin=True)
    d = to_dev(p)
    for scale in (0.0, -2.5):
        ro, rf, _ = la_ref.la_fwd(p["q"], p["k"], p["v"], p["g"], [260], [0], p["pool"], scale)
        out, fin = run_fwd(d, [0], scale)
        near("out", out, ro)
        near("final_state", fin, rf, states=True)
        r = run_bwd(d, [0], scale)
        ref = la_ref.la_bwd(p["q"], p["k"], p["v"], p["g"], [260], p["do"], p["dfin"], [0], p["pool"], scale)
        for name, x in zip(("dq", "dk", "dv"), ref):
            near(name, r[name], x)


@pytest.mark.parametrize("cu,idx", [([0, 5, 3, 10], None), ([1, 4, 10], None), ([0, 4, 9], None), ([0, 4, 11], None),
                                    ([0, -4, 10], None), ([0, 5, 10], [-2, 0]), ([0, 5, 10], [0, 2]), ([0, 5, 10], [1, 0])])
def test_bad_documents_are_reported_by_the_status_word(cu, idx):
    p = la_ref.problem(306, [10], 1, 1, -0.1, 1 if idx else 0)
    d = to_dev(p) | {"cu": torch.tensor(cu, dtype=torch.int32, device="cuda")}
    x = None if idx is None else torch.tensor(idx, dtype=torch.int32, device="cuda")
    for bwd in (False, True):
        ws = torch.empty(gdn.la_workspace_size(len(cu) - 1, 10, 1, 1, idx is not None, bwd), dtype=torch.uint8, device="cuda")
        if bwd:
            gdn.la_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["cu"], d["do"], None, x, d["pool"], workspace=ws)
        else:
            gdn.la_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], x, d["pool"], workspace=ws)
        assert gdn.workspace_status(ws) == gdn.GDN_ERR_INVALID_ARG


def test_refusals():
    p = la_ref.problem(307, [64], 2, 4, -0.1)
    d = to_dev(p)
    ok = dict(q=d["q"], k=d["k"], v=d["v"], log_decay=d["g"], cu_seqlens=d["cu"])
    for name, bad in [("q", d["q"].half()), ("q", d["q"].cpu()), ("k", d["k"][:, :1]), ("v", d["v"][:, :3]),
                      ("v", d["v"][:63]), ("log_decay", d["g"][:3]), ("log_decay", d["g"].double()),
                      ("cu_seqlens", d["cu"].long()), ("q", d["q"].transpose(0, 1).contiguous().transpose(0, 1))]:
        with pytest.raises((ValueError, gdn.GdnError)):
            gdn.la_chunk_fwd(**(ok | {name: bad}))
    with pytest.raises(gdn.GdnError) as e:
        gdn.la_chunk_fwd(**ok, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == gdn.GDN_ERR_WORKSPACE
    with pytest.raises(gdn.GdnError) as e:
        gdn.la_chunk_fwd(**ok, scale=float("nan"))
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    odd = torch.empty(64 * 2 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(64, 2, 128)
    with pytest.raises(gdn.GdnError) as e:
        gdn.la_chunk_fwd(**(ok | {"q": odd}))
    assert e.value.status == gdn.GDN_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        gdn.la_chunk_bwd(**ok, dout=None)


# ---------------------------------------------------------------------------------------- single tokens


@pytest.mark.parametrize("B,Hk,Hv,dtype", [(1, 1, 1, torch.bfloat16), (1, 2, 8, torch.float16), (33, 2, 8, torch.bfloat16),
                                           (70, 4, 4, torch.float16)])
def test_step(B, Hk, Hv, dtype):
    g = -np.exp2(-np.arange(float(Hv)))
    g[-1] = -np.inf if Hv > 1 else g[-1]
    rng = np.random.default_rng(B)
    idx = rng.permutation(B + 5)[:B].astype(np.int32)
    p = la_ref.problem(400 + B, [1] * B, Hk, Hv, g, B + 5)
    q, k, v = (torch.from_numpy(p[x]).to("cuda", dtype) for x in ("q", "k", "v"))
    pool = torch.from_numpy(p["pool"]).to("cuda", torch.float32)
    before, gd = pool.clone(), torch.from_numpy(p["g"]).to("cuda", torch.float32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gdn.la_decode_step(q, k, v, gd, pool, torch.from_numpy(idx).cuda(), scale=SCALE, status=st)
    assert out.dtype == dtype and int(st) == 0
    qd, kd, vd = (x.double().cpu().numpy() for x in (q, k, v))
    ro, rf, _ = la_ref.la_fwd(qd, kd, vd, p["g"], [1] * B, list(idx), p["pool"], SCALE)
    # one rounding: half a unit in the last place of the type, and fp32 sums of 128 terms
    got, unit = out.double().cpu().numpy(), 2.0 ** (-9 if dtype == torch.bfloat16 else -12)
    assert (np.abs(got - ro) <= 1.01 * 2 * unit * np.abs(ro) + 1e-5).all()
    near("states", pool[torch.from_numpy(idx).long().cuda()], rf, states=True)
    rest = torch.from_numpy(np.setdiff1d(np.arange(B + 5), idx)).cuda()
    assert torch.equal(pool[rest], before[rest])


def test_steps_continue_a_prompt():
    """A prompt through the chunked form, then tokens one at a time: the whole document."""
    p = la_ref.problem(450, [150], 2, 4, SLOW)
    d = to_dev(p)
    head = {x: d[x][:147] for x in ("q", "k", "v", "do")} | {"g": d["g"], "pool": None, "cu": cu_of([147])}
    out, pool = run_fwd(head)
    outs = [out]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in range(147, 150):
        outs.append(gdn.la_decode_step(d["q"][t:t + 1], d["k"][t:t + 1], d["v"][t:t + 1], d["g"], pool, zero, scale=SCALE))
    ro, rf, _ = la_ref.la_fwd(p["q"], p["k"], p["v"], p["g"], [150], scale=SCALE)
    near("out", torch.cat(outs), ro)
    near("state", pool, rf, states=True)


def test_step_strides_bad_index_and_refusals():
    p = la_ref.problem(451, [1] * 6, 1, 2, -0.3, 7)
    d = to_dev(p)
    idx = torch.tensor([3, 1, 9, 0, -1, 5], dtype=torch.int32, device="cuda")
    fused = torch.cat([d["q"], d["k"], d["v"]], dim=1)
    pool = d["pool"].clone()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gdn.la_decode_step(fused[:, :1], fused[:, 1:2], fused[:, 2:], d["g"], pool, idx, status=st)
    assert int(st) == gdn.GDN_ERR_INVALID_ARG and not out[2].any() and not out[4].any()
    keep = [0, 1, 3, 5]
    ro, rf, _ = la_ref.la_fwd(*(p[x][keep] for x in ("q", "k", "v")), p["g"], [1] * 4, [3, 1, 0, 5], p["pool"])
    near("out", out[keep], ro)
    near("states", pool[[3, 1, 0, 5]], rf, states=True)
    assert torch.equal(pool[[2, 4, 6]], d["pool"][[2, 4, 6]])
    assert gdn.la_decode_step(d["q"][:0], d["k"][:0], d["v"][:0], d["g"], pool, idx[:0]).shape == (0, 2, 128)
    for kw in (dict(q=d["q"].float()), dict(k=d["k"].half()), dict(v=d["v"][:5]), dict(state_pool=pool[:, :1]),
               dict(state_idx=idx.long())):
        args = dict(q=d["q"], k=d["k"], v=d["v"], log_decay=d["g"], state_pool=pool, state_idx=idx) | kw
        with pytest.raises(ValueError):
            gdn.la_decode_step(**args)
