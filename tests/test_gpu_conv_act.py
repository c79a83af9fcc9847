"""The convolution with its activation (forward, backward, single tokens) against its fp64 definition
(tests/ssm_ref.py). Tolerances: half a unit of the output's type, and 2^-21 of the sum of the terms' absolute values for
each of the few fp32 roundings behind it: 8 (four products summed, the activation's exponential, reciprocal and
product), for dx 8 more, for the sums over tokens one a token (tails: one a fork)."""
import numpy as np
import pytest

from tests import ssm_ref
from tests.test_gpu_ssm import TYPES, int32, near

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import linear_attention_varlen_gb300 as gdn  # noqa: E402


def inputs(seed, lens, C, dtype, n_pool=0, apart=0):
    rng = np.random.default_rng(seed)
    T, dt = sum(lens), TYPES[dtype]

    def rows(n):
        t = torch.from_numpy(rng.standard_normal((n, C))).to("cuda", dt)
        if apart and n:
            wide = torch.full((n, C + 8 + apart), 9.0, dtype=dt, device="cuda")
            t = wide[:, 8:8 + C].copy_(t)
        return t
    d = dict(x=rows(T), dy=rows(T), lens=lens)
    d["w"] = torch.from_numpy(0.5 * rng.standard_normal((C, 4))).float().cuda()
    d["bias"] = torch.from_numpy(0.3 * rng.standard_normal(C)).float().cuda()
    d["pool"] = torch.from_numpy(rng.standard_normal((n_pool, 3, C))).to("cuda", dt) if n_pool else None
    d["dtail"] = torch.from_numpy(rng.standard_normal((len(lens), 3, C))).float().cuda()
    d["cu"] = int32(np.concatenate([[0], np.cumsum(lens)]).tolist())
    return d


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def check(d, idx=None, act="silu", bias=True, dtail=True):
    b = d["bias"] if bias else None
    x, w, pool = f64(d["x"]), f64(d["w"]), f64(d["pool"])
    bb = f64(d["bias"]) if bias else np.zeros(x.shape[1])
    kw = dict(bias=b, init_idx=int32(idx), conv_init=d["pool"], activation=act)
    y, tail = gdn.conv_fwd(d["x"], d["w"], d["cu"], **kw)
    ry, u, rt = ssm_ref.conv_fwd(x, w, bb, d["lens"], pool, idx, act == "silu")
    mu = ssm_ref.conv_fwd(np.abs(x), np.abs(w), np.abs(bb), d["lens"], None if pool is None else np.abs(pool), idx, False)[1]
    near("y", y, ry, mu, 8)  # |silu'| < 1.1
    assert tail.dtype == d["x"].dtype and np.array_equal(f64(tail), rt)
    g = gdn.conv_bwd(d["x"], d["w"], d["cu"], d["dy"], dfinal_tail=d["dtail"] if dtail else None, **kw)
    dy, dt = f64(d["dy"]), f64(d["dtail"]) if dtail else None
    s = ssm_ref.sigmoid(u)
    slope = s * (1 + u * (1 - s)) if act == "silu" else np.ones_like(u)
    # |silu''| < 0.5 times the error of u, and the slope's own terms
    mdu = np.abs(dy) * ((s * (1 + np.abs(u) * (1 - s)) if act == "silu" else 1.0) + mu)
    ref = ssm_ref.conv_bwd(x, w, d["lens"], dy * slope, dt, pool, idx)
    mag = ssm_ref.conv_bwd(np.abs(x), np.abs(w), d["lens"], mdu, None if dt is None else np.abs(dt),
                           None if pool is None else np.abs(pool), idx)
    n = len(x) + 16 + len(d["lens"])
    near("dx", g["dx"], ref["dx"], mag["dx"], 16 + len(d["lens"]))
    near("dw", g["dw"], ref["dw"], mag["dw"], n)
    if bias:
        near("dbias", g["dbias"], ref["dbias"], mag["dbias"], n)
    else:
        assert g["dbias"] is None
    if pool is None:
        assert g["dconv_init"] is None
    else:
        near("dconv_init", g["dconv_init"], ref["dconv_init"], mag["dconv_init"], 16 + len(d["lens"]))


@pytest.mark.parametrize("lens", [[1], [2, 1, 3], [0, 4], [31, 32, 33], [63, 64, 65, 1], [200], [2, 2, 2, 0, 0, 60, 1, 1, 1]])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_lengths(lens, dtype):
    check(inputs(sum(lens), lens, 24, dtype))


@pytest.mark.parametrize("C", [8, 16, 1000, 1032, 4104])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_channels(C, dtype):
    check(inputs(C, [40, 3, 30], C, dtype))


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("dtail", [True, False])
def test_parts_left_out(act, bias, dtail):
    check(inputs(3, [70, 1, 2, 9], 16, "bf16", n_pool=2), [1, -1, 0, 0], act, bias, dtail)


@pytest.mark.parametrize("idx", [[-1, 0, 1, 1, 0, -1], [0, 2 + 0, 2 + 1, 2 + 2, 2 + 3, 2 + 1], [-1, 2, 2, -1, 2 + 1, 1]])
@pytest.mark.parametrize("lens", [[70, 5, 0, 1, 2, 66], [1, 0, 0, 1, 1, 3], [2, 1, 64, 128, 0, 1]])
def test_pools_and_forks(idx, lens):
    check(inputs(7, lens, 16, "fp32", n_pool=2), idx)
    check(inputs(8, lens, 16, "bf16", n_pool=2), idx)


def test_forks_without_a_pool():
    check(inputs(19, [40, 0, 2, 70, 1], 16, "fp32"), [-1, 0, 1, 2, 0])


@pytest.mark.parametrize("dtype", list(TYPES))
def test_views_into_wider_rows(dtype):
    check(inputs(5, [50, 0, 20], 40, dtype, n_pool=1, apart=16), [0, -1, 1 + 0])


def test_without_activation_as_the_plain_convolution():
    """bf16 and contiguous, activation "none": the same function as the call without the argument, to a rounding."""
    d = inputs(9, [33, 100, 2], 64, "bf16")
    old, old_tail = gdn.conv_fwd(d["x"], d["w"], d["cu"], bias=d["bias"])
    new, new_tail = gdn.conv_fwd(d["x"], d["w"], d["cu"], bias=d["bias"], activation="none")
    assert torch.equal(old_tail, new_tail)
    off = (old.double() - new.double()).abs()
    assert (off <= 2.0 ** -7 * old.double().abs() + 1e-5).all()  # two roundings to bf16


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_what_is_not_finite_stays_in_its_reach(value):
    d = inputs(11, [40, 30], 16, "fp32")
    want = gdn.conv_fwd(d["x"], d["w"], d["cu"], bias=d["bias"], activation="silu")[0]
    wdx = gdn.conv_bwd(d["x"], d["w"], d["cu"], d["dy"], bias=d["bias"], activation="silu")["dx"]
    d["x"][38, 5] = value
    got = gdn.conv_fwd(d["x"], d["w"], d["cu"], bias=d["bias"], activation="silu")[0]
    gdx = gdn.conv_bwd(d["x"], d["w"], d["cu"], d["dy"], bias=d["bias"], activation="silu")["dx"]
    keep = torch.ones(70, 16, dtype=torch.bool, device="cuda")
    keep[38:40, 5] = False  # the second document begins at 40
    assert torch.equal(got[keep], want[keep])
    keep[35:40, 5] = False
    assert torch.equal(gdx[keep], wdx[keep])
    u = -value if value == value else value
    if u == u:  # an infinite u: silu gives 0 or inf, its slope 0 or 1
        assert not torch.isnan(got[38, 5])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,C", [(1, 8), (3, 1032), (200, 64)])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_single_tokens(dtype, B, C, act):
    d = inputs(B + C, [1] * B, C, dtype, n_pool=B + 2, apart=8)
    idx = np.random.default_rng(B).permutation(B + 2)[:B]
    before = d["pool"].clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = gdn.conv_decode_step(d["x"], d["w"], d["pool"], int32(idx.tolist()), bias=d["bias"], activation=act, status=status)
    x, w, b = f64(d["x"]), f64(d["w"]), f64(d["bias"])
    ref, _, tails = ssm_ref.conv_fwd(x, w, b, [1] * B, f64(before), idx, act == "silu")
    mu = ssm_ref.conv_fwd(np.abs(x), np.abs(w), np.abs(b), [1] * B, np.abs(f64(before)), idx, False)[1]
    near("y", y, ref, mu, 8)
    assert np.array_equal(f64(d["pool"])[idx], tails) and status.item() == 0
    rest = [i for i in range(B + 2) if i not in set(idx.tolist())]
    assert torch.equal(d["pool"][rest], before[rest])


def test_steps_follow_a_prompt():
    d = inputs(4, [30], 16, "bf16")
    whole, end = gdn.conv_fwd(d["x"], d["w"], d["cu"], bias=d["bias"], activation="silu")
    _, tail = gdn.conv_fwd(d["x"][:20], d["w"], int32([0, 20]), bias=d["bias"], activation="silu")
    for t in range(20, 30):
        y = gdn.conv_decode_step(d["x"][t:t + 1], d["w"], tail, int32([0]), bias=d["bias"], activation="silu")
        assert torch.equal(y[0], whole[t])  # the same operations in the same order
    assert torch.equal(tail, end)


def test_step_skips_and_reports_bad_entries():
    d = inputs(2, [1] * 3, 16, "fp16", n_pool=2)
    for bad in (2, -1):
        before = d["pool"].clone()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = gdn.conv_decode_step(d["x"], d["w"], d["pool"], int32([1, bad, 0]), bias=d["bias"], status=status)
        assert status.item() == gdn.GDN_ERR_INVALID_ARG and (y[1] == 0).all() and (y[0] != 0).any()
        assert torch.equal(d["pool"][1, :2], before[1, 1:])


@pytest.mark.parametrize("cu,idx", [([0, 9, 5, 20], None), ([1, 5, 9, 20], None), ([0, 5, 9, 21], None),
                                    ([0, 5, 9, 20], [-2, 0, 0]), ([0, 5, 9, 20], [-1, -1, 2 + 2])])
def test_bad_layouts_are_reported(cu, idx):
    d = inputs(1, [5, 4, 11], 16, "bf16", n_pool=2)
    y = torch.full((20, 16), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(gdn.conv_workspace_size(3, 20, 16, True, "silu"), dtype=torch.uint8, device="cuda")
    kw = dict(bias=d["bias"], init_idx=int32(idx), conv_init=d["pool"], activation="silu", workspace=ws)
    gdn.conv_fwd(d["x"], d["w"], int32(cu), y=y, **kw)
    assert gdn.workspace_status(ws) == gdn.GDN_ERR_INVALID_ARG and (y == 3.0).all()
    gdn.conv_bwd(d["x"], d["w"], int32(cu), d["dy"], **kw)
    assert gdn.workspace_status(ws) == gdn.GDN_ERR_INVALID_ARG


def test_no_tokens_at_all():
    d = inputs(1, [0, 0], 16, "bf16", n_pool=1)
    y, tail = gdn.conv_fwd(d["x"], d["w"], d["cu"], bias=d["bias"], init_idx=int32([0, -1]), conv_init=d["pool"],
                           activation="silu")
    assert y.shape == (0, 16) and torch.equal(tail[0], d["pool"][0]) and (tail[1] == 0).all()
    g = gdn.conv_bwd(d["x"], d["w"], d["cu"], d["dy"], bias=d["bias"], init_idx=int32([0, -1]), conv_init=d["pool"],
                     dfinal_tail=d["dtail"], activation="silu")
    assert torch.equal(g["dconv_init"][0], d["dtail"][0]) and (g["dw"] == 0).all() and (g["dbias"] == 0).all()


def test_the_same_bits_every_time():
    d = inputs(6, [3000, 1, 500], 64, "bf16", n_pool=1)
    kw = dict(bias=d["bias"], init_idx=int32([0, 1, 0]), conv_init=d["pool"], activation="silu")
    first = gdn.conv_bwd(d["x"], d["w"], d["cu"], d["dy"], dfinal_tail=d["dtail"], **kw)
    for _ in range(3):
        again = gdn.conv_bwd(d["x"], d["w"], d["cu"], d["dy"], dfinal_tail=d["dtail"], **kw)
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_backward_of_a_large_batch_as_of_its_documents():
    """Enough rows for the backward's longer blocks: dx has the bits of calls on one document each (their blocks are
    shorter), dw and dbias differ by the order of their sums, 12000 roundings of 2^-24 of the terms."""
    lens, C = [5000, 1, 3499, 0, 3500], 4096
    d = inputs(21, lens, C, "bf16")
    g = gdn.conv_bwd(d["x"], d["w"], d["cu"], d["dy"], bias=d["bias"], dfinal_tail=d["dtail"], activation="silu")
    dw, db, size, t = 0.0, 0.0, 0.0, 0
    for i, n in enumerate(lens):
        if n == 0:
            continue
        a = gdn.conv_bwd(d["x"][t:t + n], d["w"], int32([0, n]), d["dy"][t:t + n], bias=d["bias"],
                         dfinal_tail=d["dtail"][i:i + 1], activation="silu")
        assert torch.equal(g["dx"][t:t + n], a["dx"])
        dw, db, t = dw + a["dw"].double(), db + a["dbias"].double(), t + n
    size = 12000 ** 0.5 * 12  # of sums of 12000 products of normal values, none of them above this by far
    assert float((g["dw"].double() - dw).abs().max()) <= 12000 * 2.0 ** -24 * size
    assert float((g["dbias"].double() - db).abs().max()) <= 12000 * 2.0 ** -24 * size


def test_backward_in_long_blocks():
    """Enough tokens and channels for the longer blocks of the backward, documents that end at their borders and around
    them. The reference is the definition in fp64 on the GPU; bounds as in `check`."""
    C = 4096
    lens = [124 * 30, 1, 0, 122, 3, 124 * 20 - 2, 2, 124 * 26]
    T = sum(lens)
    assert T >= 124 * 76  # eight CTAs to each SM: 16 blocks of channels, 152 SMs
    d = inputs(77, lens, C, "bf16")
    g = gdn.conv_bwd(d["x"], d["w"], d["cu"], d["dy"], bias=d["bias"], activation="silu")
    x, dy, w, b = (d[k].double() for k in ("x", "dy", "w", "bias"))
    ref = {k: torch.zeros_like(v, dtype=torch.float64) for k, v in g.items() if v is not None}
    mag = {k: torch.zeros_like(v) for k, v in ref.items()}
    t = 0
    for n in lens:
        e = torch.cat([torch.zeros_like(x[:3]), x[t:t + n]])
        u = b + sum(w[:, m] * e[m:m + n] for m in range(4))
        mu = b.abs() + sum((w[:, m] * e[m:m + n]).abs() for m in range(4))
        s = torch.sigmoid(u)
        du = dy[t:t + n] * s * (1 + u * (1 - s))
        mdu = dy[t:t + n].abs() * (s * (1 + u.abs() * (1 - s)) + mu)
        for out, v, wv, ev in ((ref, du, w, e), (mag, mdu, w.abs(), e.abs())):
            de = torch.zeros_like(e)
            for m in range(4):
                de[m:m + n] += wv[:, m] * v
                out["dw"][:, m] += (v * ev[m:m + n]).sum(0)
            out["dx"][t:t + n] = de[3:]
            out["dbias"] += v.sum(0)
        t += n
    for k, roundings in (("dx", 16 + len(lens)), ("dw", T + 16 + len(lens)), ("dbias", T + 16 + len(lens))):
        assert ((g[k].double() - ref[k]).abs() <= 2.0 ** -21 * roundings * mag[k] + 2.0 ** -115).all(), k
