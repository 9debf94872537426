"""Pins of the mixer operators' oracle (oracle/mixer.py): gradients against central differences of its own forward
in float64, closed forms, and brute force over every pair of scores. CPU only."""

import numpy as np
import pytest

from oracle import mixer as M


def diff(f, x, d, eps=1e-6):
    """Central difference of f along d at x."""
    return (f(x + eps * d) - f(x - eps * d)) / (2 * eps)


@pytest.mark.parametrize("H,Hk,lens,with_state", [(2, 2, None, True), (4, 2, [5, 0, 3], True), (2, 1, None, False)])
def test_glr_gradients_are_the_differences(H, Hk, lens, with_state):
    r = np.random.default_rng(7)
    B, T, dk, dv, scale = 3, 5, 3, 4, 0.7
    x = dict(q=r.normal(size=(B, T, Hk, dk)), k=r.normal(size=(B, T, Hk, dk)), v=r.normal(size=(B, T, H, dv)),
             g=-np.abs(r.normal(size=(B, T, H))), state=r.normal(size=(B, H, dk, dv)) if with_state else None)
    d_o, d_last = r.normal(size=(B, T, H, dv)), r.normal(size=(B, H, dk, dv))

    def loss(**kw):
        y = dict(x, **kw)
        o, last, _, _ = M.glr_forward(y["q"], y["k"], y["v"], y["g"], scale, y["state"], lens)
        return (o * d_o).sum() + (last * d_last).sum()

    got, mag = M.glr_backward(d_o, x["q"], x["k"], x["v"], x["g"], scale, x["state"], d_last, lens)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("state", "dstate")):
        if x[name] is None:
            continue
        for _ in range(4):
            d = r.normal(size=x[name].shape)
            want = diff(lambda z: loss(**{name: z}), x[name], d)
            assert abs((got[grad] * d).sum() - want) < 1e-7 * max(1.0, abs(want)), name
        assert (np.abs(got[grad]) <= mag[grad] * (1 + 1e-12) + 1e-15).all()


def test_glr_closed_forms():
    r = np.random.default_rng(8)
    q, k, v = r.normal(size=(1, 6, 1, 2)), r.normal(size=(1, 6, 1, 2)), r.normal(size=(1, 6, 1, 3))
    g = np.zeros((1, 6, 1))
    o, last, _, _ = M.glr_forward(q, k, v, g, 1.0)       # no decay: causal linear attention
    s = np.tril(q[0, :, 0] @ k[0, :, 0].T) @ v[0, :, 0]
    assert np.allclose(o[0, :, 0], s) and np.allclose(last[0, 0], k[0, :, 0].T @ v[0, :, 0])
    g[0, 3] = -np.inf                                     # a reset: the rows from there on stand alone
    o, last, _, _ = M.glr_forward(q, k, v, g, 1.0, state=r.normal(size=(1, 1, 2, 3)))
    o2, last2, _, _ = M.glr_forward(q[:, 3:], k[:, 3:], v[:, 3:], np.zeros((1, 3, 1)), 1.0)
    assert np.allclose(o[:, 3:], o2) and np.allclose(last, last2)


@pytest.mark.parametrize("D,rot,inter", [(8, 8, False), (8, 4, True), (7, 2, False), (5, 0, False), (6, 6, True)])
def test_norm_rope(D, rot, inter):
    r = np.random.default_rng(9)
    x, w, pos = r.normal(size=(4, 3, D)), r.normal(size=D), np.array([0, 5, 2, 99])
    ang = np.arange(7)[:, None] * (0.3 ** np.arange(rot // 2))[None]
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    y = M.norm_rope(x, w, pos, table, rot, inter, 0.0)
    plain = M.norm_rope(x, w, pos, table, 0, inter, 0.0)
    assert np.allclose((plain / w) ** 2 @ np.ones(D), D)                      # unit root mean square
    assert np.allclose((y ** 2).sum(-1), (plain ** 2).sum(-1))                # a rotation keeps lengths
    if rot:
        i, j = M._pairs(D, rot, inter)
        z = (plain[..., i] + 1j * plain[..., j]) * np.exp(1j * ang[np.clip(pos, 0, 6)])[:, None]
        assert np.allclose(y[..., i], z.real) and np.allclose(y[..., j], z.imag)
    assert np.array_equal(y[..., rot:], plain[..., rot:])
    d = r.normal(size=x.shape)
    dx, dw, mx, mw = M.norm_rope_backward(d, x, w, pos, table, rot, inter, 1e-3)
    e = r.normal(size=x.shape)
    f = lambda z: (M.norm_rope(z, w, pos, table, rot, inter, 1e-3) * d).sum()  # noqa: E731
    assert np.isclose((dx * e).sum(), diff(f, x, e), rtol=1e-7)
    e = r.normal(size=D)
    f = lambda z: (M.norm_rope(x, z, pos, table, rot, inter, 1e-3) * d).sum()  # noqa: E731
    assert np.isclose((dw * e).sum(), diff(f, w, e), rtol=1e-7)
    assert (np.abs(dx) <= mx * (1 + 1e-12)).all() and (np.abs(dw) <= mw * (1 + 1e-12)).all()


@pytest.mark.parametrize("n1,n2,K", [(5, 7, 4), (3, 2, 6), (9, 9, 9), (1, 8, 8), (6, 6, 1)])
def test_slot_topk_is_the_best_of_all_pairs(n1, n2, K):
    r = np.random.default_rng(10)
    a, b = r.normal(size=(6, n1)).astype(np.float32), r.normal(size=(6, n2)).astype(np.float32)
    idx, val = M.slot_topk(a, b, K, 0.9)
    for t in range(6):
        s = (a[t][:, None] + b[t][None, :]).reshape(-1)
        best = np.sort(s)[::-1][:K]
        assert np.array_equal(s[idx[t]], best) and len(set(idx[t])) == K
        e = np.exp(0.9 * (best.astype(np.float64) - best[0]))
        assert np.allclose(val[t], e / e.sum(), rtol=1e-12)


def test_slot_topk_ties_and_empty_rows():
    z = np.zeros((1, 4), np.float32)
    idx, val = M.slot_topk(z, z, 3, 1.0)
    assert idx.tolist() == [[0, 1, 2]] and np.allclose(val, 1 / 3)
    m = np.full((1, 4), -np.inf, np.float32)
    idx, val = M.slot_topk(m, z, 3, 1.0)
    assert idx.tolist() == [[0, 1, 2]] and (val == 0).all()
    n = np.array([[np.nan, 1.0, np.nan, 0.5]], np.float32)
    idx, _ = M.slot_topk(n, z, 3, 1.0)
    assert idx.tolist() == [[4, 5, 6]]


def test_slot_gradients_are_the_differences():
    r = np.random.default_rng(11)
    a, b, K = r.normal(size=(3, 6)), r.normal(size=(3, 5)), 7
    idx, _ = M.slot_topk(a, b, K, 1.3)
    y = r.normal(size=(3, K))
    da, db, _, _ = M.slot_topk_backward(y, idx, a, b, 1.3)

    def loss(a, b):   # at the fixed selection
        s = np.take_along_axis(a, idx // 5, 1) + np.take_along_axis(b, idx % 5, 1)
        e = np.exp(1.3 * (s - s.max(1, keepdims=True)))
        return (e / e.sum(1, keepdims=True) * y).sum()

    d = r.normal(size=a.shape)
    assert np.isclose((da * d).sum(), diff(lambda x: loss(x, b), a, d), rtol=1e-7)
    d = r.normal(size=b.shape)
    assert np.isclose((db * d).sum(), diff(lambda x: loss(a, x), b, d), rtol=1e-7)
