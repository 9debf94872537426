"""GPU parity of the gated delta rule (gdr_forward, gdr_backward, gdr_step) with the float64 oracle.

Bounds, per element, from the oracle's magnitudes (mag, in units of one rounding of what is handled, added up in quadrature as
errors of independent sign are): the longest sum of a float32 evaluation has n = dk + dv + 64 terms, whose errors add up to
sqrt(n) roundings of 2^-24, and 8 times that is allowed for; a bfloat16 result is rounded once more, 2^-8 |value|.
"""

import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_delta_memory_amd as sdm  # noqa: E402
from oracle import mixer as M  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF, NAN = float("inf"), float("nan")


def say(*a):
    print(*a, flush=True)


def make(B, T, H, Hk, dk, dv, dtype, seed=3, gate=3.0, state=True, lens=None):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    unit = lambda *s: torch.nn.functional.normalize(rnd(*s), dim=-1)  # noqa: E731
    x = dict(q=unit(B, T, Hk, dk), k=unit(B, T, Hk, dk), v=rnd(B, T, H, dv), d_o=rnd(B, T, H, dv))
    x = {n: t.to(DT[dtype]) for n, t in x.items()}
    x["g"] = torch.nn.functional.logsigmoid(rnd(B, T, H) + gate)
    x["beta"] = rnd(B, T, H).sigmoid()
    x["state"] = rnd(B, H, dk, dv) * 0.3 if state else None
    x["d_last"] = rnd(B, H, dk, dv) * 0.3 if state else None
    x["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    return x


def host(x):
    return None if x is None else x.float().numpy() if x.is_floating_point() else x.numpy()


def cuda(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def near(name, got, want, mag, n, bf):
    got = got.float().cpu().numpy().astype(np.float64)
    tol = 8 * np.sqrt(n) * 2.0 ** -24 * mag + 1e-30
    if bf:
        tol = tol + 2.0 ** -8 * np.abs(want)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (name, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / tol))


def args(d):
    return [d[n] for n in ("q", "k", "v", "g", "beta")]


def forward(x, dtype, scale, dev=None):
    """The forward pass of the host inputs x (device tensors: dev) against the oracle."""
    d = cuda(x) if dev is None else dev
    dk, dv = x["q"].shape[3], x["v"].shape[3]
    h = {n: host(t) for n, t in x.items()}
    o, last = sdm.gdr_forward(*args(d), scale=scale, state=d["state"], lens=d["lens"])
    wo, wl, mo, ml = M.gdr_forward(*args(h), scale, h["state"], h["lens"])
    near("o", o, wo, mo, dk + dv + 64, dtype == "bf16")
    near("last", last, wl, ml, dk + dv + 64, False)
    return o, last


def backward(x, dtype, scale, dev=None):
    d = cuda(x) if dev is None else dev
    dk, dv = x["q"].shape[3], x["v"].shape[3]
    h = {n: host(t) for n, t in x.items()}
    r = sdm.gdr_backward(d["d_o"], *args(d), scale=scale, state=d["state"], d_last=d["d_last"], lens=d["lens"])
    w, m = M.gdr_backward(h["d_o"], *args(h), scale, h["state"], h["d_last"], h["lens"])
    for name in ("dq", "dk", "dv", "dbeta", "dg", "dstate"):
        near(name, r[name], w[name], m[name], dk + dv + 64, dtype == "bf16" and name in ("dq", "dk", "dv"))
    return r


SHAPES = [(1, 1, 1, 1, 64, 64), (2, 1, 2, 2, 128, 128), (1, 2, 1, 1, 1, 1), (1, 63, 1, 1, 64, 128), (1, 64, 2, 1, 128, 64), (2, 65, 1, 1, 120, 120),
          (1, 130, 3, 3, 9, 33), (1, 200, 4, 2, 64, 72), (2, 127, 2, 1, 65, 17), (1, 191, 1, 1, 128, 128), (1, 300, 1, 1, 16, 7)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,Hk,dk,dv", SHAPES)
def test_forward_matches_oracle(dtype, B, T, H, Hk, dk, dv):
    say("gdr forward", dtype, B, T, H, Hk, dk, dv)
    forward(make(B, T, H, Hk, dk, dv, dtype), dtype, dk ** -0.5)
    forward(make(B, T, H, Hk, dk, dv, dtype, state=False, seed=4), dtype, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,lens", [(150, [0, 150, 1, 64]), (300, [300, 0, 70, 129]), (100, [-3, 900, 100, 99])])
def test_forward_lengths(dtype, T, lens):
    """Tokens past a row's length may hold anything; a row of no tokens keeps its state."""
    say("gdr lens", dtype, T, lens)
    x = make(4, T, 2, 1, 24, 40, dtype, lens=lens)
    d = cuda(x)
    for b, n in enumerate(lens):
        for name in ("q", "k", "v", "g", "beta"):
            d[name][b, max(0, min(n, T)):] = NAN
    o, last = forward(x, dtype, 0.5, dev=d)
    for b, n in enumerate(lens):
        assert (o[b, max(0, min(n, T)):] == 0).all()
        if n <= 0:
            assert torch.equal(last[b], d["state"][b])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,dk,dv", [(1, 4, 4, 64, 64), (5, 2, 1, 128, 128), (3, 3, 3, 33, 50), (2, 1, 1, 1, 1), (300, 4, 2, 64, 72), (600, 4, 4, 128, 60)])
def test_step_matches_oracle(dtype, B, H, Hk, dk, dv):
    say("gdr step", dtype, B, H, Hk, dk, dv)
    x = make(B, 1, H, Hk, dk, dv, dtype)
    d, h = cuda(x), {n: host(t) for n, t in x.items()}
    wo, wl, mo, ml = M.gdr_forward(*args(h), 0.4, h["state"])
    new, n = torch.full_like(d["state"], NAN), dk + dv + 64
    one = [t[:, 0] for t in args(d)]
    o = sdm.gdr_step(*one, d["state"], scale=0.4, new_state=new)
    near("o", o, wo[:, 0], mo[:, 0], n, dtype == "bf16")
    near("state", new, wl, ml, n, False)
    # In place, in rows of a pool, and a request without one.
    pool = torch.full((2 * B + 1, H, dk, dv), 7.0, device="cuda")
    slots = torch.arange(B, device="cuda", dtype=torch.int32) * 2 + 1
    pool[slots.long()] = d["state"]
    slots[B // 2] = 2 * B + 1 if B > 1 else -1
    o2 = sdm.gdr_step(*one, pool, scale=0.4, slots=slots)
    keep = torch.arange(B, device="cuda") != B // 2
    assert torch.equal(o2[keep], o[keep]) and (o2[~keep] == 0).all()
    assert torch.equal(pool[slots[keep].long()], new[keep])
    assert (pool[0::2] == 7.0).all() and torch.equal(pool[2 * (B // 2) + 1], d["state"][B // 2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,Hk,dk,dv", SHAPES)
def test_backward_matches_oracle(dtype, B, T, H, Hk, dk, dv):
    say("gdr backward", dtype, B, T, H, Hk, dk, dv)
    backward(make(B, T, H, Hk, dk, dv, dtype), dtype, dk ** -0.5)
    backward(make(B, T, H, Hk, dk, dv, dtype, state=False, seed=4), dtype, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,lens", [(150, [0, 150, 1, 64]), (300, [300, 0, 70, 129]), (100, [-3, 900, 100, 99])])
def test_backward_lengths(dtype, T, lens):
    say("gdr backward lens", dtype, T, lens)
    x = make(4, T, 2, 1, 24, 40, dtype, lens=lens)
    d = cuda(x)
    for b, n in enumerate(lens):
        for name in ("q", "k", "v", "g", "beta", "d_o"):
            d[name][b, max(0, min(n, T)):] = NAN
    r = backward(x, dtype, 0.5, dev=d)
    for b, n in enumerate(lens):
        for name in ("dq", "dk", "dv", "dg", "dbeta"):
            assert (r[name][b, max(0, min(n, T)):] == 0).all(), name
        if n <= 0:
            assert torch.equal(r["dstate"][b], d["d_last"][b])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_resets_and_strong_gates(dtype):
    """Gates of -infinity (a new sequence starts), gates that leave almost nothing, gates of 0, and beta of 0 and of 1."""
    say("gdr resets", dtype)
    x = make(1, 333, 2, 2, 32, 64, dtype)
    x["g"][0, 0, 0] = x["g"][0, 70] = x["g"][0, 71, 1] = -INF
    x["g"][0, 127, 0] = -1e30
    x["g"][0, 128:140] = -90.0
    x["g"][0, 200:300] = 0.0
    x["beta"][0, 100:130] = 0.0
    x["beta"][0, 130:150, 1] = 1.0
    forward(x, dtype, 0.3)
    r = backward(x, dtype, 0.3)
    assert (r["dg"][0, 70] == 0).all() and r["dg"][0, 0, 0] == 0 and r["dg"][0, 127, 0] == 0 and (r["dstate"][0, 0] == 0).all()
    assert not (r["dg"][0, 1:70] == 0).any() and not (r["dbeta"][0, 100:130] == 0).any()
    x["state"] = x["d_last"] = None
    assert (backward(x, dtype, 0.3)["dg"][0, 0] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,dk,dv,lens", [(700, 1, 48, 40, None), (1090, 2, 128, 128, None), (1600, 1, 100, 33, None), (900, 1, 64, 128, [900, 130, 0, 515])])
def test_rows_cut_into_segments(dtype, T, H, dk, dv, lens):
    say("gdr segments", dtype, T, H, dk, dv, lens)
    B = 1 if lens is None else len(lens)
    few, many = (sdm.gdr_workspace_bytes(n, T, H, 1, dk, dv, DT[dtype]) for n in (1, 1000))
    assert few > many // 1000 + 4 * dk * dk   # the segments' transitions and states
    x = make(B, T, H, 1, dk, dv, dtype, gate=5.0, lens=lens)
    forward(x, dtype, 0.2)
    backward(x, dtype, 0.2)
    x = make(B, T, H, 1, dk, dv, dtype, gate=2.0, state=False, seed=5, lens=lens)
    x["g"][0, 300] = x["g"][0, 511] = -INF
    forward(x, dtype, 0.2)
    backward(x, dtype, 0.2)
