"""GPU: what the gated linear recurrence makes of values that are not finite. Where the float64 oracle's result is
finite the kernels' is within the bounds of finite inputs (a reset, or a later token, lets nothing through), and
where it is not, neither is the kernels' (infinity or NaN)."""

import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import sparse_delta_memory_amd as sdm  # noqa: E402
from oracle import mixer as M  # noqa: E402
from test_glr_gpu import DT, cuda, host, make, near, say  # noqa: E402

INF, NAN = float("inf"), float("nan")


def same(name, got, want, mag, n, bf):
    fin = np.isfinite(want)
    assert np.isfinite(mag[fin]).all()
    g = got.float().cpu()
    assert not np.isfinite(g.numpy()[~fin]).any(), "%s: finite where the definition is not" % name
    near(name, g[torch.from_numpy(fin)], want[fin], mag[fin], n, bf)


def check(x, dtype, scale, grads=("dq", "dk", "dv", "dstate")):
    bf = dtype == torch.bfloat16
    d, h = cuda(x), {k: host(t) for k, t in x.items()}
    B, T, Hk, dk = x["q"].shape
    H, dv = x["v"].shape[2:]
    n = dk + dv + 96 + T // 64
    args = [d[k] for k in ("q", "k", "v", "g")]
    o, last = sdm.glr_forward(*args, scale=scale, state=d["state"], lens=d["lens"])
    r = sdm.glr_backward(d["d_o"], *args, scale=scale, state=d["state"], d_last=d["d_last"], lens=d["lens"])
    with np.errstate(invalid="ignore", over="ignore"):
        wo, wl, mo, ml = M.glr_forward(h["q"], h["k"], h["v"], h["g"], scale, h["state"], h["lens"])
        w, m = M.glr_backward(h["d_o"], h["q"], h["k"], h["v"], h["g"], scale, h["state"], h["d_last"], h["lens"])
    same("o", o, wo, mo, n, bf)
    same("last", last, wl, ml, n, False)
    for name in grads:
        rounded = bf and name in ("dq", "dk", "dv")
        same(name, r[name], w[name], m[name], n + (2 * (H // Hk) if name != "dg" else 0), rounded)
    return wo, w


# (streams, tokens, heads): one chunk per segment, joined by each block or chained; rows of three chunks and no segments.
SHAPES = [(1, 60, 2), (1, 200, 1), (1, 700, 1), (128, 140, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H", SHAPES)
def test_a_reset_clears_what_is_not_finite(dtype, B, T, H):
    """States that hold NaN or infinity (rows of an uninitialised pool), cleared at the row's first token or later; and
    gradients of the last state that do, backwards."""
    say("glr reset of a state that is not finite", dtype, B, T, H)
    x = make(B, T, H, max(1, H // 2), 16, 24, DT[dtype])
    x["state"][:, 0] = NAN
    x["state"][:, -1, 3:5, ::2] = INF
    x["d_last"][0] = -INF
    x["d_last"][-1, -1, 2, 2] = NAN
    x["g"][0, 0] = -INF                      # a new sequence in every head
    x["g"][-1, min(T - 1, 70), 0] = -INF
    x["g"][-1, T // 2, -1] = -1e30
    wo, w = check(x, DT[dtype], 0.3)
    assert np.isfinite(wo[0]).all() and np.isfinite(w["dstate"][0]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dv", [24, 33])
def test_a_reset_in_a_step(dtype, dv):
    """Single tokens in rows of a pool that nobody has written: a gate of -infinity starts from nothing."""
    say("glr step reset", dtype, dv)
    B, H, dk, rows = 6, 2, 40, 9
    x = cuda(make(B, 1, H, 1, dk, dv, DT[dtype]))
    one = [x[n][:, 0] for n in ("q", "k", "v", "g")]
    one[3][:] = -INF
    one[3][5] = -0.5
    want_state = torch.zeros_like(x["state"])
    want_state[5] = x["state"][5]
    want = sdm.glr_step(*one, want_state)
    pool = torch.full((rows, H, dk, dv), NAN, device="cuda")
    pool[1::2] = INF
    slots = torch.tensor([8, 3, 0, 1, 4, 6], dtype=torch.int32, device="cuda")
    pool[6] = x["state"][5]
    out = sdm.glr_step(*one, pool, slots=slots)
    assert torch.isfinite(want).all() and torch.equal(out, want) and torch.equal(pool[slots.long()], want_state)
    assert not torch.isfinite(pool[2]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H", SHAPES)
@pytest.mark.parametrize("what", ["q", "k", "v", "d_o"])
@pytest.mark.parametrize("resets", [False, True])
def test_values_reach_only_what_they_are_part_of(dtype, B, T, H, what, resets):
    """NaN and infinities at single tokens and columns: no earlier token (no later one in the gradients that run backwards),
    no token on the other side of a reset, and no column or head of its own sees them."""
    say("glr values that are not finite", dtype, B, T, H, what, resets)
    # Gates near 0: no decay of a row's whole length falls below float32's smallest value.
    x = make(B, T, H, max(1, H // 2), 16, 24, DT[dtype], gate=6.0)
    heads = x[what].shape[2]
    for b, t, h, c, val in ((0, T // 2, 0, 3, NAN), (0, min(T - 1, 58), 0, 15, INF), (B - 1, min(T - 1, 20), heads - 1, 0, -INF),
                            (B // 2, min(T - 1, 177), heads // 2, 7, NAN), (B // 2, min(T - 1, 178), heads // 2, 8, INF)):
        x[what][b, t, h, c] = val
    if resets:
        for t in (T // 2 - 1, T // 2 + 1, 19, 22, 50, 178):
            if t < T:
                x["g"][:, t] = -INF
    wo, w = check(x, DT[dtype], 0.3)
    reached = wo if what in ("q", "k", "v") else w["dq"]
    assert 0 < np.isfinite(reached).sum() < reached.size


def test_every_token_of_a_chunk():
    """One infinity in v, at every place of two chunks in turn: outputs before it as without it, bit for bit."""
    T, dk, dv = 128, 32, 40
    x = cuda(make(1, T, 1, 1, dk, dv, torch.bfloat16, state=False))
    q, k, g = (x[n].expand(T, *x[n].shape[1:]) for n in ("q", "k", "g"))
    v = x["v"].repeat(T, 1, 1, 1)
    want, _ = sdm.glr_forward(q, k, v, g)
    at = torch.arange(T, device="cuda")
    v[at, at, 0, at % dv] = INF
    o, last = sdm.glr_forward(q, k, v, g)
    for t in range(T):
        c = t % dv
        assert torch.equal(o[t, :t], want[t, :t]) and not torch.isfinite(o[t, t:, 0, c]).any(), t
        rest = [n for n in range(dv) if n != c]
        assert torch.equal(o[t][..., rest], want[t][..., rest]) and not torch.isfinite(last[t, 0, :, c]).any(), t


def gate_gradients(x, dtype, scale=0.3):
    """dg of the kernels and the oracle's, and the magnitude of a row's whole sum, from finite values in place of the others."""
    d, h = cuda(x), {k: host(t) for k, t in x.items()}
    r = sdm.glr_backward(*(d[k] for k in ("d_o", "q", "k", "v", "g")), scale=scale, state=d["state"], d_last=d["d_last"], lens=d["lens"])
    args = lambda z: (*(z[k] for k in ("d_o", "q", "k", "v", "g")), scale, z["state"], z["d_last"], z["lens"])  # noqa: E731
    with np.errstate(invalid="ignore", over="ignore"):
        w, _ = M.glr_backward(*args(h))
        clean = {n: t if t is None or n in ("g", "lens") else np.where(np.isfinite(t), t, 1.0) for n, t in h.items()}
        _, m = M.glr_backward(*args(clean))
    return r["dg"], w["dg"], np.broadcast_to(m["dg"][:, :1], w["dg"].shape)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H", SHAPES)
@pytest.mark.parametrize("what", ["q", "k", "v", "d_o", "state", "d_last"])
@pytest.mark.parametrize("resets", [False, True])
def test_gate_gradients(dtype, B, T, H, what, resets):
    """A gate's gradient is made of the states before it and what comes from behind it: a key or value that is not finite
    leaves the gates up to it alone, a query or gradient those behind it, a reset both sides."""
    say("glr gate gradients, not finite", dtype, B, T, H, what, resets)
    x = make(B, T, H, max(1, H // 2), 16, 24, DT[dtype], gate=6.0, lens=[T - 3 * (b % 4) for b in range(B)])
    if what in ("state", "d_last"):
        x[what][0, 0, 2, 3] = NAN
        x[what][B - 1, H - 1, 0, 5] = INF
    else:
        x[what][0, T // 2, 0, 3] = NAN
        x[what][B - 1, min(T - 20, 70), -1, 1] = -INF
    if resets:
        for t in (T // 2 - 9, T // 2 - 8, T // 2 + 1, 3, 64, 150):
            if t < T:
                x["g"][:, t] = -INF
    got, want, mag = gate_gradients(x, DT[dtype])
    if resets:
        assert (got[torch.isneginf(x["g"]).cuda()] == 0).all()
    same("dg", got, want, mag, 16 + 24 + 96 + T // 64, False)
    if what not in ("state", "d_last"):
        assert np.isfinite(want).any(1).all()


@pytest.mark.parametrize("T", [60, 200, 1000])
def test_gate_gradients_of_packed_sequences(T):
    """Gates before a reset have the gradients that they have without the sequence behind it, however large that is."""
    x = make(2, T, 2, 1, 16, 24, torch.float32, gate=6.0)
    x["g"][:, T // 2] = -INF
    x["d_last"] = x["d_last"] * 0
    d = cuda(x)
    run = lambda n: sdm.glr_backward(*(d[k][:, :n] for k in ("d_o", "q", "k", "v", "g")), state=d["state"], d_last=d["d_last"])["dg"]  # noqa: E731
    alone = run(T // 2)
    for k in ("q", "v", "d_o"):
        d[k][:, T // 2:] *= 1e4
    both = run(T)
    assert (both[:, T // 2] == 0).all()
    assert torch.allclose(both[:, :T // 2], alone, rtol=0, atol=1e-5 * float(alone.abs().max()))


def test_gates_whose_factor_is_zero():
    """exp(g) below float32's range cuts like a reset: a gradient of 0, and nothing of the later tokens before it."""
    x = make(1, 300, 2, 1, 16, 24, torch.float32, gate=6.0)
    x["g"][:, 150] = -90.0
    x["g"][:, 151] = -200.0
    x["g"][:, 40] = -9999.0
    x["v"][0, 200, :, 3] = INF
    got, want, mag = gate_gradients(x, torch.float32)
    assert (got[:, [40, 150, 151]] == 0).all()
    assert torch.isfinite(got[:, :200]).all()
    n = 16 + 24 + 96 + 4
    near("dg", got[:, :150], want[:, :150], mag[:, :150], n, False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 64, 333])
def test_the_first_gate_without_a_state(dtype, T):
    """From no state the first gate scales nothing: its gradient is 0, not the rounding of the sums behind it."""
    x = make(3, T, 4, 2, 32, 40, DT[dtype], state=False, gate=6.0, lens=[T, 0, T])
    got, want, mag = gate_gradients(x, DT[dtype])
    assert (got[:, 0] == 0).all() and (want[:, 0] == 0).all()
    same("dg", got, want, mag, 32 + 40 + 96 + T // 64, False)
