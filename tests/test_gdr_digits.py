"""The delta rule's measure of digits (gdr_digits.py) on the CPU: a float32 evaluation passes it, and what is wrong does not."""

import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import gdr_digits as D  # noqa: E402
from oracle import mixer as M  # noqa: E402


def make(B, T, H, Hk, dk, dv, seed=0):
    r = np.random.default_rng(seed)
    unit = lambda *s: (lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True))(r.standard_normal(s))  # noqa: E731
    x = [unit(B, T, Hk, dk), unit(B, T, Hk, dk), r.standard_normal((B, T, H, dv)), -np.log1p(np.exp(-r.standard_normal((B, T, H)) - 3)),
         1 / (1 + np.exp(-r.standard_normal((B, T, H))))]
    return [a.astype(np.float32) for a in x], *((r.standard_normal((B, H, dk, dv)) * 0.3).astype(np.float32) for _ in range(2)), \
        r.standard_normal((B, T, H, dv)).astype(np.float32)


def outputs(x, state, d_last, d_o, scale):
    o, last, _, _ = M.gdr_forward(*x, scale, state)
    return dict(o=o, last=last, **M.gdr_backward(d_o, *x, scale, state, d_last)[0])


def in_float32(x, state, d_last, d_o, scale):
    """The rule and its gradients token by token, every step rounded to float32."""
    q, k, v, g, beta = x
    H = v.shape[2]
    q, k = (np.repeat(t, H // t.shape[2], 2) for t in (q, k))
    B, T, _, dk = q.shape
    f = np.float32
    S, R, scale = state.copy(), d_last.copy(), f(scale)
    zero = lambda t: np.zeros_like(t)  # noqa: E731
    r = dict(o=zero(v), dq=zero(q), dk=zero(q), dv=zero(v), dg=zero(g), dbeta=zero(g))
    seen = []
    for t in range(T):
        S1 = np.exp(g[:, t])[..., None, None] * S
        miss = v[:, t] - (k[:, t, :, :, None] * S1).sum(2)
        S = S1 + k[:, t, :, :, None] * (beta[:, t, :, None] * miss)[:, :, None]
        r["o"][:, t] = scale * (q[:, t, :, :, None] * S).sum(2)
        seen.append((S1, S, miss))
    for t in range(T - 1, -1, -1):
        S1, S2, miss = seen[t]
        e = scale * d_o[:, t]
        r["dq"][:, t] = (S2 * e[:, :, None]).sum(-1)
        R = R + q[:, t, :, :, None] * e[:, :, None]
        du = (k[:, t, :, :, None] * R).sum(2)
        d, u = beta[:, t, :, None] * du, beta[:, t, :, None] * miss
        r["dk"][:, t] = (R * u[:, :, None]).sum(-1) - (S1 * d[:, :, None]).sum(-1)
        r["dv"][:, t], r["dbeta"][:, t] = d, (du * miss).sum(-1)
        R = R - k[:, t, :, :, None] * d[:, :, None]
        r["dg"][:, t] = (R * S1).sum((2, 3))
        R = np.exp(g[:, t])[..., None, None] * R
    for n in ("dq", "dk"):
        r[n] = r[n].reshape(B, T, x[0].shape[2], -1, dk).sum(3)
    assert all(t.dtype == f for t in r.values())
    return dict(r, last=S, dstate=R)


@pytest.mark.parametrize("shape", D.SHAPES + D.SEGMENTED[:1])
def test_a_float32_evaluation_passes(shape):
    x, state, d_last, d_o = make(*shape)
    want, got = outputs(x, state, d_last, d_o, 0.3), in_float32(x, state, d_last, d_o, 0.3)
    for name in D.OUTPUTS:
        D.check(name, got[name], want[name], *shape[4:], False)


def test_what_is_wrong_does_not():
    shape = (1, 130, 4, 2, 32, 40)
    x, state, d_last, d_o = make(*shape)
    want = outputs(x, state, d_last, d_o, 0.3)

    def fails(name, got, bf):
        with pytest.raises(AssertionError):
            D.check(name, got, want[name], 32, 40, bf)
    for bf in (False, True):
        for name in D.OUTPUTS:
            fails(name, 0 * want[name], bf)
            D.check(name, want[name], want[name], 32, 40, bf)
            one = want[name].copy()
            one.reshape(one.shape[0], -1)[:, ::100] = 0    # one value in a hundred
            fails(name, one, bf)
        # Without the state before the first token or the last state's gradient; a gate's or a token's share of the other.
        for name in ("o", "last", "dq", "dk", "dg", "dbeta"):
            fails(name, outputs(x, 0 * state, d_last, d_o, 0.3)[name], bf)
        for name in ("dk", "dv", "dg", "dbeta", "dstate"):
            fails(name, outputs(x, state, 0 * d_last, d_o, 0.3)[name], bf)
        late = [t.copy() for t in x]
        late[3][:, 64:] = 0    # the second chunk's gates
        for name in D.OUTPUTS:
            fails(name, outputs(late, state, d_last, d_o, 0.3)[name], bf)
    # float32 results of factors of 16 bits, and bfloat16 results rounded twice as far as they may be.
    r = np.random.default_rng(1)
    for name in D.OUTPUTS:
        fails(name, want[name] * (1 + 2.0 ** -17 * r.choice([-1, 1], want[name].shape)), False)
        fails(name, want[name] * (1 + 2.0 ** -7 * r.choice([-1, 1], want[name].shape)), True)
