"""The fp64 definitions the GPU tests compare with, pinned by themselves: the quadratic form, packing,
forks, and central differences of the forward for every gradient."""
import numpy as np
import pytest

from tests import la_ref


def small(seed, lens, Hk, Hv, g, n_pool=0, d=3):
    rng = np.random.default_rng(seed)
    T = sum(lens)
    mk = lambda *s: rng.standard_normal(s)  # noqa: E731
    return dict(q=mk(T, Hk, d), k=mk(T, Hk, d), v=mk(T, Hv, d), g=np.asarray(g, float),
                pool=mk(n_pool, Hv, d, d) if n_pool else None, do=mk(T, Hv, d), dfin=mk(len(lens), Hv, d, d))


def test_forward_is_the_masked_quadratic_form():
    p = small(1, [7], 1, 2, [-0.3, 0.0], n_pool=1)
    out, fin, _ = la_ref.la_fwd(p["q"], p["k"], p["v"], p["g"], [7], [0], p["pool"], 0.5)
    t = np.arange(7)
    for h in range(2):
        gap = t[:, None] - t[None]
        m = np.where(gap >= 0, np.exp(p["g"][h] * gap), 0)
        ref = (p["q"][:, 0] @ p["k"][:, 0].T * m) @ p["v"][:, h]
        ref += np.exp(p["g"][h] * (t + 1))[:, None] * (p["q"][:, 0] @ p["pool"][0, h])
        np.testing.assert_allclose(out[:, h], 0.5 * ref, rtol=1e-12)
        w = np.exp(p["g"][h] * (6 - t))
        np.testing.assert_allclose(fin[0, h], np.exp(7 * p["g"][h]) * p["pool"][0, h] + (p["k"][:, 0] * w[:, None]).T @ p["v"][:, h],
                                   rtol=1e-12)


def test_packing_and_forks_equal_separate_runs():
    p = small(2, [4, 0, 3, 5], 2, 4, [-0.1, -1.0, -0.5, -0.01])
    lens, idx = [4, 0, 3, 5], [-1, 0, 1, -1]  # document 1 (empty) forks 0, document 2 forks 1
    out, fin, _ = la_ref.la_fwd(p["q"], p["k"], p["v"], p["g"], lens, idx)
    a, fa, _ = la_ref.la_fwd(p["q"][:7], p["k"][:7], p["v"][:7], p["g"], [7])
    np.testing.assert_array_equal(out[:7], a)
    np.testing.assert_array_equal(fin[2], fa[0])
    np.testing.assert_array_equal(fin[1], fin[0])
    b, _, _ = la_ref.la_fwd(p["q"][7:], p["k"][7:], p["v"][7:], p["g"], [5])
    np.testing.assert_array_equal(out[7:], b)


@pytest.mark.parametrize("lens,idx,n_pool", [([5, 3], None, 0), ([3, 0, 1, 4, 2], [1, 2, -1, 0, 4], 2)])
def test_gradients_against_central_differences(lens, idx, n_pool):
    p = small(3, lens, 2, 4, [-0.2, -0.9, 0.0, -0.05], n_pool)

    def loss():
        out, fin, _ = la_ref.la_fwd(p["q"], p["k"], p["v"], p["g"], lens, idx, p["pool"], 0.7)
        return (out * p["do"]).sum() + (fin * p["dfin"]).sum()
    grads = la_ref.la_bwd(p["q"], p["k"], p["v"], p["g"], lens, p["do"], p["dfin"], idx, p["pool"], 0.7)
    for name, got in zip(("q", "k", "v", "pool"), grads):
        if got is None:
            continue
        x, eps = p[name], 1e-5
        for i in np.ndindex(x.shape):
            at = x[i]
            x[i] = at + eps
            up = loss()
            x[i] = at - eps
            num = (up - loss()) / (2 * eps)
            x[i] = at
            # the loss is quadratic at most in one entry: the difference is exact up to fp64 cancellation
            assert abs(num - got[i]) <= 1e-7 * max(1.0, abs(num)), (name, i, num, got[i])


def test_norm_gradients_against_central_differences():
    rng = np.random.default_rng(4)
    x, r, w, dy, dh = rng.standard_normal((3, 5)), rng.standard_normal((3, 5)), rng.standard_normal(5), \
        rng.standard_normal((3, 5)), rng.standard_normal((3, 5))

    def loss():
        y, h = la_ref.rms_fwd(x, w, r, 1e-3)
        return (y * dy).sum() + (h * dh).sum()
    dx, dw = la_ref.rms_bwd(x + r, w, dy, dh, 1e-3)
    for arr, got in ((x, dx), (r, dx), (w, dw)):
        for i in np.ndindex(arr.shape):
            at = arr[i]
            arr[i] = at + 1e-5
            up = loss()
            arr[i] = at - 1e-5
            num = (up - loss()) / 2e-5
            arr[i] = at
            # third derivatives of order 1 at these inputs: a difference error of about 1e-10
            assert abs(num - got[i]) <= 1e-7 * max(1.0, abs(num))
