"""What the state-space block's operators refuse, on the CPU: the library's checks come before it touches a GPU, the
binding's before it calls the library."""
import ctypes
import os

import pytest

import linear_attention_varlen_gb300 as gdn

P = ctypes.c_void_p
A = 1 << 20  # stands for an aligned device pointer; never read


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn.library_path()):
        from linear_attention_varlen_gb300 import build
        build.build()
    return gdn.load()


def ssm(lib, bwd=False, **kw):
    a = dict(x=A, dt=A, z=A, a=A, b=A, c=A, skip=A, bias=A, cu=A, N=1, T=64, C=64, S=16, G=1, dtype=0, strides=None,
             idx=None, pool=None, n_init=0, out=A, fin=A, ws=A, ws_bytes=1 << 40, dout=A, dfin=None, dx=A, ddt=A, dz=A, da=A,
             db=A, dc=A, dskip=A, dbias=A, dinit=None)
    a.update(kw)
    st = None if a["strides"] is None else (ctypes.c_int64 * 6)(*a["strides"])
    head = [P(a[k]) for k in ("x", "dt", "z", "a", "b", "c", "skip", "bias", "cu")]
    mid = [a["N"], a["T"], a["C"], a["S"], a["G"], a["dtype"], st, 1, P(a["idx"]), P(a["pool"]), a["n_init"]]
    if not bwd:
        return lib.gdn_ssm_fwd(*head, *mid, P(a["out"]), P(a["fin"]), P(a["ws"]), a["ws_bytes"], None)
    tail = [P(a[k]) for k in ("dout", "dfin", "dx", "ddt", "dz", "da", "db", "dc", "dskip", "dbias", "dinit", "ws")]
    return lib.gdn_ssm_bwd(*head, *mid, *tail, a["ws_bytes"], None)


@pytest.mark.parametrize("bwd", [False, True])
def test_scan_refusals(lib, bwd):
    bad = gdn.GDN_ERR_INVALID_ARG
    for kw in (dict(N=0), dict(N=(1 << 30) + 1), dict(T=-1), dict(T=2 ** 31 - 1), dict(C=0), dict(S=0), dict(S=65), dict(G=0), dict(G=3), dict(x=None), dict(dt=None),
               dict(a=None), dict(b=None), dict(c=None), dict(cu=None), dict(ws=None), dict(n_init=1), dict(n_init=-1),
               dict(x=A + 1), dict(a=A + 2), dict(cu=A + 1), dict(ws=A + 128), dict(strides=[8, 0, 0, 0, 0, 0]),
               dict(strides=[0, 0, 0, -16, 0, 0]), dict(strides=[0, 0, 0, 0, 1 << 41, 0])):
        assert ssm(lib, bwd, **kw) == bad, kw
    assert ssm(lib, bwd, dtype=3) == gdn.GDN_ERR_UNSUPPORTED
    need = gdn.ssm_workspace_size(1, 64, 64, 16, 1, bwd)
    assert ssm(lib, bwd, ws_bytes=need - 1) == gdn.GDN_ERR_WORKSPACE
    if bwd:
        for kw in (dict(dout=None), dict(dx=None), dict(ddt=None), dict(dz=None), dict(da=None), dict(db=None),
                   dict(dskip=None), dict(dbias=None), dict(n_init=1, pool=A), dict(dx=A + 1),
                   dict(strides=[0, 0, 0, 0, 0, 63])):
            assert ssm(lib, bwd, **kw) == bad, kw
    else:
        assert ssm(lib, fin=None) == bad and ssm(lib, out=None) == bad
    assert gdn.ssm_workspace_size(1, 64, 64, 65) == 0 and gdn.ssm_workspace_size(1, 64, 65, 16, 2) == 0


@pytest.mark.parametrize("dtype", [gdn.DTYPE_BF16, gdn.DTYPE_FP16, gdn.DTYPE_FP32])
def test_scan_outputs_are_aligned_to_their_types(lib, dtype):
    """Two bytes are enough for an output in 16 bits, not for one in fp32, whatever the inputs' type. The check comes before
    the workspace's, which tells a call that passed it from one that did not."""
    kw = dict(dtype=dtype, n_init=1, pool=A, idx=A, dinit=A, dfin=A, ws_bytes=0)
    typed = {False: ("out",), True: ("dx", "ddt", "dz", "db", "dc")}
    fp32 = {False: ("fin",), True: ("da", "dskip", "dbias", "dinit", "dfin")}
    by_two = gdn.GDN_ERR_INVALID_ARG if dtype == gdn.DTYPE_FP32 else gdn.GDN_ERR_WORKSPACE
    for bwd in (False, True):
        assert ssm(lib, bwd, **kw) == gdn.GDN_ERR_WORKSPACE
        for name in typed[bwd]:
            assert ssm(lib, bwd, **(kw | {name: A + 1})) == gdn.GDN_ERR_INVALID_ARG, name
            assert ssm(lib, bwd, **(kw | {name: A + 2})) == by_two, name
        for name in fp32[bwd]:
            for off in (1, 2, 3):
                assert ssm(lib, bwd, **(kw | {name: A + off})) == gdn.GDN_ERR_INVALID_ARG, (name, off)
            assert ssm(lib, bwd, **(kw | {name: A + 4})) == gdn.GDN_ERR_WORKSPACE, name


def test_scan_workspace_holds_the_largest_call(lib):
    sizes = [gdn.ssm_workspace_size(n, t, 2048, 16, 1, True) for n, t in ((1, 1), (1, 16384), (4, 16384), (4, 32768))]
    assert sizes == sorted(sizes) and gdn.ssm_workspace_size(1, 0, 1, 1) > 0


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("C,S,G", [(2048, 16, 1), (64, 16, 1), (1, 1, 1), (768, 8, 3), (8192, 64, 8), (200000, 8, 1)])
def test_scan_workspace_grows_with_tokens_and_documents(lib, C, S, G, bwd):
    """A workspace of the largest call holds every call of no more documents and tokens, on either side of each step of the
    segments' length."""
    size = lib.gdn_ssm_workspace_size
    tokens = sorted(set(range(0, 3000)) | {t + d for t in (int(1.07 ** k) for k in range(120, 300)) for d in (-1, 0, 1) if t < 2 ** 22}
                    | {16 * k + d for k in range(180, 20000, 97) for d in (0, 1)})
    for N in (1, 2, 5, 64, 1500):
        sizes = [size(N, t, C, S, G, bwd) for t in tokens]
        assert sizes[0] > 0 and sizes == sorted(sizes), N
    documents = [*range(1, 300), *range(300, 9000, 61)]
    for t in (0, 7, 16, 500, 1217, 9001, 32768, 300001):
        sizes = [size(n, t, C, S, G, bwd) for n in documents]
        assert sizes == sorted(sizes), t


def step(lib, **kw):
    a = dict(x=A, dt=A, z=A, a=A, b=A, c=A, skip=A, bias=A, B=2, C=64, S=16, G=1, dtype=0, strides=None, idx=A, pool=A,
             n_pool=4, out=A, status=None)
    a.update(kw)
    st = None if a["strides"] is None else (ctypes.c_int64 * 5)(*a["strides"])
    return lib.gdn_ssm_decode_step(*[P(a[k]) for k in ("x", "dt", "z", "a", "b", "c", "skip", "bias")], a["B"], a["C"], a["S"],
                                   a["G"], a["dtype"], st, 1, P(a["idx"]), P(a["pool"]), a["n_pool"], P(a["out"]),
                                   P(a["status"]), None)


def test_step_refusals(lib):
    for kw in (dict(B=-1), dict(B=65536), dict(C=0), dict(S=65), dict(S=0), dict(G=3), dict(x=None), dict(idx=None),
               dict(pool=None), dict(out=None), dict(n_pool=0), dict(pool=A + 2), dict(strides=[63, 0, 0, 0, 0]),
               dict(strides=[0, 0, 0, 15, 0]), dict(status=A + 2)):
        assert step(lib, **kw) == gdn.GDN_ERR_INVALID_ARG, kw
    assert step(lib, dtype=7) == gdn.GDN_ERR_UNSUPPORTED
    assert step(lib, B=0) == gdn.GDN_OK


def conv(lib, bwd=False, **kw):
    a = dict(x=A, xs=0, w=A, bias=A, cu=A, N=1, T=64, C=64, dtype=0, act=1, idx=None, pool=None, n_init=0, y=A, tail=A, ws=A,
             ws_bytes=1 << 40, dy=A, dys=0, dtail=None, dx=A, dw=A, dbias=A, dinit=None)
    a.update(kw)
    head = [P(a["x"]), a["xs"], P(a["w"]), P(a["bias"]), P(a["cu"]), a["N"], a["T"], a["C"], a["dtype"], a["act"],
            P(a["idx"]), P(a["pool"]), a["n_init"]]
    if not bwd:
        return lib.gdn_conv_act_fwd(*head, P(a["y"]), P(a["tail"]), P(a["ws"]), a["ws_bytes"], None)
    return lib.gdn_conv_act_bwd(*head, P(a["dy"]), a["dys"], *[P(a[k]) for k in ("dtail", "dx", "dw", "dbias", "dinit", "ws")],
                                a["ws_bytes"], None)


@pytest.mark.parametrize("bwd", [False, True])
def test_convolution_refusals(lib, bwd):
    for kw in (dict(N=0), dict(T=-1), dict(C=4), dict(C=12), dict(C=(1 << 23) + 8), dict(x=None), dict(w=None), dict(cu=None),
               dict(ws=None), dict(n_init=1), dict(n_init=-1), dict(x=A + 8), dict(w=A + 4), dict(ws=A + 16), dict(xs=56),
               dict(xs=68), dict(xs=-64), dict(T=2 ** 31 - 1, C=8)):
        assert conv(lib, bwd, **kw) == gdn.GDN_ERR_INVALID_ARG, kw
    assert conv(lib, bwd, dtype=3) == gdn.GDN_ERR_UNSUPPORTED and conv(lib, bwd, act=2) == gdn.GDN_ERR_UNSUPPORTED
    assert conv(lib, bwd, ws_bytes=255) == gdn.GDN_ERR_WORKSPACE
    extra = (dict(dy=None), dict(dx=None), dict(dw=None), dict(dys=60), dict(n_init=1, pool=A)) if bwd else \
        (dict(y=None), dict(tail=None), dict(y=A + 8))
    for kw in extra:
        assert conv(lib, bwd, **kw) == gdn.GDN_ERR_INVALID_ARG, kw
    assert gdn.conv_workspace_size(1, 10, 12, activation="silu") == 0


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("C", [8, 264, 4096, 65536, 1 << 23])
def test_convolution_workspace_grows_with_tokens_and_documents(lib, C, bwd):
    """As the scan's: the backward's blocks get longer from some length on, and fewer."""
    size = lib.gdn_conv_act_workspace_size
    tokens = sorted({*range(0, 3000), *range(3000, 20000, 7), *range(20000, 400000, 61), *range(150650, 150920)})
    tokens = [t for t in tokens if t * C <= 1 << 40]
    for N in (1, 33, 4000):
        sizes = [size(N, t, C, bwd) for t in tokens]
        assert sizes[0] > 0 and sizes == sorted(sizes), N
    sizes = [size(n, 9001, C, bwd) for n in range(1, 3000)]
    assert sizes == sorted(sizes)


def test_convolution_step_refusals(lib):
    def call(x=A, xs=0, w=A, B=2, C=64, dtype=0, act=1, idx=A, pool=A, n_pool=3, y=A, status=None):
        return lib.gdn_conv_decode_step(P(x), xs, P(w), None, B, C, dtype, act, P(idx), P(pool), n_pool, P(y), P(status), None)
    for kw in (dict(B=-1), dict(B=65536), dict(C=4), dict(x=None), dict(w=None), dict(idx=None), dict(pool=None), dict(y=None),
               dict(n_pool=0), dict(xs=60), dict(x=A + 2), dict(pool=A + 8), dict(status=A + 1)):
        assert call(**kw) == gdn.GDN_ERR_INVALID_ARG, kw
    assert call(dtype=5) == gdn.GDN_ERR_UNSUPPORTED and call(act=-1) == gdn.GDN_ERR_UNSUPPORTED
    assert call(B=0) == gdn.GDN_OK


def gnorm(lib, bwd=False, **kw):
    a = dict(x=A, xs=0, z=A, zs=0, w=A, dy=A, dys=0, T=4, D=256, group=128, shared=1, first=0, dtype=0, wdtype=0, eps=1e-6,
             y=A, dx=A, dz=A, dw=A, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    kinds = [a["T"], a["D"], a["group"], a["shared"], a["first"], a["dtype"], a["wdtype"], a["eps"]]
    if not bwd:
        return lib.gdn_gated_rmsnorm_fwd(P(a["x"]), a["xs"], P(a["z"]), a["zs"], P(a["w"]), *kinds, P(a["y"]), None)
    return lib.gdn_gated_rmsnorm_bwd(P(a["x"]), a["xs"], P(a["z"]), a["zs"], P(a["w"]), P(a["dy"]), a["dys"], *kinds,
                                     P(a["dx"]), P(a["dz"]), P(a["dw"]), P(a["ws"]), a["ws_bytes"], None)


@pytest.mark.parametrize("bwd", [False, True])
def test_gated_norm_refusals(lib, bwd):
    for kw in (dict(T=-1), dict(D=0), dict(group=0), dict(group=100), dict(x=None), dict(z=None), dict(w=None), dict(xs=255),
               dict(zs=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(x=A + 1), dict(T=1 << 40)):
        assert gnorm(lib, bwd, **kw) == gdn.GDN_ERR_INVALID_ARG, kw
    for kw in (dict(first=2), dict(dtype=3), dict(wdtype=-1), dict(D=16385, group=16385)):
        assert gnorm(lib, bwd, **kw) == gdn.GDN_ERR_UNSUPPORTED, kw
    if bwd:
        for kw in (dict(dy=None), dict(dx=None), dict(dz=None), dict(dw=None), dict(ws=None), dict(ws=A + 16), dict(dys=3)):
            assert gnorm(lib, bwd, **kw) == gdn.GDN_ERR_INVALID_ARG, kw
        assert gnorm(lib, bwd, ws_bytes=255) == gdn.GDN_ERR_WORKSPACE
    else:
        assert gnorm(lib, y=None) == gdn.GDN_ERR_INVALID_ARG
        assert gnorm(lib, T=0) == gdn.GDN_OK


def test_host_pointers_are_refused(lib):
    """Nothing here is device memory, so calls that pass every other check stop before a launch."""
    assert ssm(lib) != gdn.GDN_OK and ssm(lib, True) != gdn.GDN_OK and step(lib) != gdn.GDN_OK
    assert conv(lib) != gdn.GDN_OK and conv(lib, True) != gdn.GDN_OK
    assert gnorm(lib) != gdn.GDN_OK and gnorm(lib, True) != gdn.GDN_OK


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 16)
    cu = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: gdn.conv_fwd(x, x, cu, activation="relu"),
                 lambda: gdn.conv_decode_step(x, x, x, cu, activation="gelu"),
                 lambda: gdn.gated_rmsnorm_fwd(x, x, x[0], first="both"),
                 lambda: gdn.gated_rmsnorm_fwd(x, x, x[0], group=5),
                 lambda: gdn.gated_rmsnorm_bwd(x, x, x[0], None),
                 lambda: gdn.ssm_scan_bwd(x, x, x, x[:, None], x[:, None], cu, None),
                 lambda: gdn.ssm_scan_fwd(x, x, x, x[:, None], x[:, None], cu),   # not on a GPU
                 lambda: gdn.ssm_scan_fwd(x.int(), x, x, x[:, None], x[:, None], cu)):
        with pytest.raises(ValueError):
            call()


def test_refused_activations_name_the_allowed_ones():
    """The step has no call without an activation, whose default is None."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match='^activation: expected None, "none" or "silu"$'):
        gdn.conv_fwd(x, x, cu, activation="relu")
    for activation in (None, "relu"):
        with pytest.raises(ValueError, match='^activation: expected "none" or "silu"$'):
            gdn.conv_decode_step(x, x, x, cu, activation=activation)
