"""The quadratic form in fp64 (tests/la_quad.py) agrees with the token-by-token definition (tests/la_ref.py)."""
import numpy as np
import torch

from tests import la_quad, la_ref


def test_quadratic_form_is_the_recurrence():
    lens, idx, Hk, Hv = [7, 0, 5], [1, 0, -1], 1, 3
    p = la_ref.problem(1, lens, Hk, Hv, [-0.3, 0.0, -np.inf], n_pool=2, dfin=True)
    d = {x: torch.from_numpy(p[x]) for x in ("q", "k", "v", "do", "pool", "dfin", "g")}
    r = la_quad.packed(d, lens, idx, 0.5)
    out, fin, _ = la_ref.la_fwd(p["q"], p["k"], p["v"], p["g"], lens, idx, p["pool"], 0.5)
    dq, dk, dv, dpool = la_ref.la_bwd(p["q"], p["k"], p["v"], p["g"], lens, p["do"], p["dfin"], idx, p["pool"], 0.5)
    for got, want in ((r["out"], out), (r["fin"], fin), (r["dqh"].sum(1, keepdim=True), dq),
                      (r["dkh"].sum(1, keepdim=True), dk), (r["dv"], dv), (r["dpool"], dpool)):
        np.testing.assert_allclose(got.numpy(), want, rtol=1e-10, atol=1e-10)
