"""GPU: what the gated delta rule makes of values that are not finite, where resets, gates, lengths and segments of the time axis
decide how far they get. Compared are where results are finite, and the finite ones with a run of finite inputs."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import sparse_delta_memory_amd as sdm  # noqa: E402
from test_gdr_gpu import INF, NAN, make, say  # noqa: E402
from test_gdr_more_gpu import close, run  # noqa: E402


# In a chunk, at its ends, and in rows cut into segments (800).
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,t0", [(90, 20), (90, 63), (90, 64), (100, 0), (800, 330)])
@pytest.mark.parametrize("name", ["k", "v", "q", "beta"])
@pytest.mark.parametrize("value", [INF, NAN])
def test_a_packed_sequence_of_one_token(dtype, T, t0, name, value):
    """A reset at a token and one behind it: nothing of the token reaches another one or the last state."""
    say("gdr one token between resets", dtype, T, t0, name, value)
    x = make(1, T, 2, 2, 32, 40, dtype)
    x["g"][0, t0] = x["g"][0, t0 + 1] = -INF
    clean = run(x)
    y = {n: None if t is None else t.clone() for n, t in x.items()}
    y[name][(0, t0, 1) if name == "beta" else (0, t0, 1, 3)] = value
    r = run(y)
    others = torch.arange(T) != t0
    for out in ("o", "dq", "dk", "dv", "dbeta", "dg"):
        assert torch.equal(r[out][:, :, 0], clean[out][:, :, 0]), out          # the other head
        close(name + " " + out, r[out][0, others, 1], clean[out][0, others, 1])
    assert not torch.isfinite(r["o"][0, t0, 1]).all()
    close("last", r["last"], clean["last"])
    close("dstate", r["dstate"], clean["dstate"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,t0,reset", [(90, 20, 45), (90, 63, 64), (130, 64, 129), (800, 200, 230), (800, 200, 700)])
@pytest.mark.parametrize("value", [INF, NAN])
def test_gradients_gates_and_betas_that_are_not_finite(dtype, T, t0, reset, value):
    say("gdr not finite: d_o, g, beta", dtype, T, t0, reset, value)
    x = make(1, T, 2, 2, 32, 40, dtype)
    x["g"][0, reset] = -INF
    clean = run(x)
    cols = torch.arange(40) != 3
    for name in ("d_o", "g", "beta"):
        if name == "g" and value == INF:
            continue   # gates are at most 0
        y = {n: None if t is None else t.clone() for n, t in x.items()}
        y[name][(0, t0, 1, 3) if name == "d_o" else (0, t0, 1)] = value
        r = run(y)
        for out in ("o", "dq", "dk", "dv", "dbeta", "dg"):
            assert torch.equal(r[out][:, :, 0], clean[out][:, :, 0]), (name, out)
        a, b = ({n: t[0, :, 1] for n, t in z.items() if n not in ("last", "dstate")} for z in (r, clean))
        close(name + " last", r["last"], clean["last"])
        for out in ("dq", "dk", "dv", "dbeta", "dg"):
            close(name + " " + out + " past the reset", a[out][reset:], b[out][reset:])
        if name == "d_o":
            assert torch.equal(r["o"], clean["o"])
            assert not torch.isfinite(a["dq"][t0]).any() and not torch.isfinite(a["dv"][:t0 + 1, 3]).any()
            others = torch.arange(T) != t0
            close("dq of other tokens", a["dq"][others], b["dq"][others])
            close("dv of other columns", a["dv"][:, cols], b["dv"][:, cols])
            for out in ("dk", "dv", "dbeta"):
                close(out + " of later tokens", a[out][t0 + 1:], b[out][t0 + 1:])
        else:
            assert not torch.isfinite(a["o"][t0:reset]).any() if name == "g" else not torch.isfinite(a["o"][t0:reset]).all(-1).any()
            close(name + " o before", a["o"][:t0], b["o"][:t0])
            close(name + " dq before", a["dq"][:t0], b["dq"][:t0])
            close(name + " o past the reset", a["o"][reset:], b["o"][reset:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [50, 64, 100, 900])
def test_a_last_gradient_that_is_not_finite_ends_at_a_reset(dtype, T):
    say("gdr not finite: d_last", dtype, T)
    x = make(1, T, 2, 1, 32, 40, dtype)
    for at in (T - 1, T // 2):
        x["g"][0, at] = -INF
        clean = run(x)
        r = run(dict(x, d_last=torch.full_like(x["d_last"], NAN)))
        assert torch.equal(r["o"], clean["o"]) and torch.equal(r["last"], clean["last"])
        for out in ("dq", "dk", "dv", "dbeta", "dg"):
            close(out, r[out][0, :at], clean[out][0, :at])
        close("dq", r["dq"], clean["dq"])
        close("dstate", r["dstate"], clean["dstate"])
        assert not torch.isfinite(r["dv"][0, at:]).any()
        x["g"][0, at] = -0.1
