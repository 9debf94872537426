"""The oracle of the gated delta rule: its gradients against differences, and cases that have a closed form."""

import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from oracle import mixer as M  # noqa: E402


def make(B, T, H, Hk, dk, dv, seed=0):
    r = np.random.default_rng(seed)
    k = r.standard_normal((B, T, Hk, dk))
    x = dict(q=r.standard_normal((B, T, Hk, dk)), k=k / np.linalg.norm(k, axis=-1, keepdims=True), v=r.standard_normal((B, T, H, dv)),
             g=-np.abs(r.standard_normal((B, T, H))) * 0.2, beta=r.random((B, T, H)))
    return x, r.standard_normal((B, H, dk, dv)), r


@pytest.mark.parametrize("lens", [None, [5, 3]])
def test_gradients_against_differences(lens):
    x, state, r = make(2, 7, 4, 2, 3, 5)
    d_o, d_last = r.standard_normal((2, 7, 4, 5)), r.standard_normal(state.shape)
    scale = 0.7

    def loss(y, s):
        o, last, _, _ = M.gdr_forward(y["q"], y["k"], y["v"], y["g"], y["beta"], scale, s, lens)
        return (o * d_o).sum() + (last * d_last).sum()

    grads, _ = M.gdr_backward(d_o, x["q"], x["k"], x["v"], x["g"], x["beta"], scale, state, d_last, lens)
    for name, at in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("state", "dstate")):
        for i in r.integers(0, grads[at].size, 12):
            h, vals = 1e-5, []
            for sign in (1, -1):
                y, s = {n: t.copy() for n, t in x.items()}, state.copy()
                (s if name == "state" else y[name]).reshape(-1)[i] += sign * h
                vals.append(loss(y, s))
            # central differences of a smooth function: an error of h^2, and 64-bit rounding of the loss over h
            assert abs((vals[0] - vals[1]) / (2 * h) - grads[at].reshape(-1)[i]) < 1e-7, (name, i)


def test_closed_forms():
    x, state, _ = make(1, 6, 1, 1, 4, 3, seed=2)
    # beta 0: the state only decays, and every output reads it.
    o, last, _, _ = M.gdr_forward(x["q"], x["k"], x["v"], x["g"], 0 * x["beta"], 1.0, state)
    a = np.exp(x["g"][0, :, 0].cumsum())
    np.testing.assert_allclose(last[0, 0], a[-1] * state[0, 0], rtol=1e-13)
    np.testing.assert_allclose(o[0, :, 0], a[:, None] * (x["q"][0, :, 0] @ state[0, 0]), rtol=1e-12)
    # beta 1, no decay, keys of norm 1: after its token the state gives a key's value back exactly.
    o, _, _, _ = M.gdr_forward(x["k"], x["k"], x["v"], 0 * x["g"], 0 * x["beta"] + 1, 1.0, state)
    np.testing.assert_allclose(o, x["v"], rtol=1e-12, atol=1e-14)
    # A reset leaves nothing of the state, be it NaN.
    g = x["g"].copy()
    g[0, 3] = -np.inf
    both = M.gdr_forward(x["q"], x["k"], x["v"], g, x["beta"], 1.0, state * np.nan)[0][0, 3:]
    alone = M.gdr_forward(x["q"][:, 3:], x["k"][:, 3:], x["v"][:, 3:], x["g"][:, 3:], x["beta"][:, 3:], 1.0)[0][0]
    np.testing.assert_allclose(both, alone, rtol=1e-12)
