"""The fp64 definitions of tests/ssm_ref.py: their reverse modes against central differences, forks against the same
documents joined, and steps of one token against a whole document."""
import numpy as np
import pytest

from tests import ssm_ref

EPS = 1e-6  # central differences of smooth functions of order one: error about EPS^2 + 1e-16 / EPS = 1e-10


def differences(f, x, at):
    out = np.zeros(len(at))
    for k, i in enumerate(at):
        keep = x[i]
        x[i] = keep + EPS
        hi = f()
        x[i] = keep - EPS
        lo = f()
        x[i] = keep
        out[k] = (hi - lo) / (2 * EPS)
    return out


def some(rng, shape, n=6):
    return [tuple(rng.integers(0, s) for s in shape) for _ in range(n)]


@pytest.mark.parametrize("gate,softplus,G,idx", [(True, True, 1, None), (False, True, 2, [-1, 0, 2 + 0, 2 + 2, 1]),
                                                 (True, False, 2, [0, 0, 1, 2 + 1, -1])])
def test_scan_gradients_against_differences(gate, softplus, G, idx):
    lens = [7, 0, 5, 1, 9]
    p = ssm_ref.problem(5, lens, 6, 3, G, gate=gate, softplus=softplus, n_pool=2, dfin=True)
    g = ssm_ref.scan_bwd(ssm_ref.terms(p), p["dout"], p["dfin"], idx)

    def loss():
        out, _, _, _, fin = ssm_ref.scan_fwd(ssm_ref.terms(p), idx)
        return (out * p["dout"]).sum() + (fin * p["dfin"]).sum()
    rng = np.random.default_rng(1)
    for key, of in (("dx", "x"), ("ddt", "dt"), ("dz", "z"), ("da", "a"), ("db", "b"), ("dc", "c"), ("dskip", "skip"),
                    ("ddt_bias", "dt_bias"), ("dinit", "pool")):
        if p[of] is None:
            continue
        at = some(rng, p[of].shape)
        want = differences(loss, p[of], at)
        np.testing.assert_allclose([g[key][i] for i in at], want, rtol=1e-6, atol=1e-7, err_msg=key)


def test_scan_of_a_fork_and_of_joined_documents():
    p = ssm_ref.problem(3, [9, 6], 4, 5)
    q = ssm_ref.terms(p)
    out, _, _, _, fin = ssm_ref.scan_fwd(q, idx=[-1, 0])  # the second starts where the first ends
    q["lens"] = [15]
    joined, _, _, _, end = ssm_ref.scan_fwd(q)
    np.testing.assert_array_equal(out, joined)
    np.testing.assert_array_equal(fin[1], end[0])


@pytest.mark.parametrize("idx", [None, [-1, 0, 1, 2 + 0, 2 + 3, 2 + 1]])
def test_conv_gradients_against_differences(idx):
    rng = np.random.default_rng(2)
    lens, C = [5, 0, 1, 2, 1, 8], 3
    x, w, bias = rng.standard_normal((sum(lens), C)), rng.standard_normal((C, 4)), rng.standard_normal(C)
    pool, dy = rng.standard_normal((2, 3, C)), rng.standard_normal((sum(lens), C))
    dtail = rng.standard_normal((len(lens), 3, C))

    def loss():
        y, _, tails = ssm_ref.conv_fwd(x, w, bias, lens, pool, idx)
        return (y * dy).sum() + (tails * dtail).sum()
    u = ssm_ref.conv_fwd(x, w, bias, lens, pool, idx)[1]
    s = ssm_ref.sigmoid(u)
    g = ssm_ref.conv_bwd(x, w, lens, dy * s * (1 + u * (1 - s)), dtail, pool, idx)
    for key, of in (("dx", x), ("dw", w), ("dbias", bias), ("dconv_init", pool)):
        at = some(rng, of.shape, 10)
        np.testing.assert_allclose([g[key][i] for i in at], differences(loss, of, at), rtol=1e-6, atol=1e-7, err_msg=key)


@pytest.mark.parametrize("first", ["norm", "gate"])
@pytest.mark.parametrize("shared", [True, False])
def test_gated_norm_gradients_against_differences(first, shared):
    rng = np.random.default_rng(4)
    x, z, dy = (rng.standard_normal((3, 12)) for _ in range(3))
    w = rng.standard_normal(4 if shared else 12)

    def loss():
        return (ssm_ref.gnorm_fwd(x, z, w, 4, 1e-3, first) * dy).sum()
    (dx, dz, dw), bounds = ssm_ref.gnorm_bwd(x, z, w, dy, 4, 1e-3, first)
    for got, bound, of in zip((dx, dz, dw), bounds, (x, z, w)):
        at = some(rng, of.shape, 12)
        np.testing.assert_allclose([got[i] for i in at], differences(loss, of, at), rtol=1e-6, atol=1e-7)
        assert (np.abs(got) <= bound * (1 + 1e-12)).all()
