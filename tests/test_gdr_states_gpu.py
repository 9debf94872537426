"""GPU: what gates and lengths do to states, the same for a whole row, for one whose time axis is cut into segments and for a token."""

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
from test_gdr_gpu import DT, INF, NAN, args, cuda, make, say  # noqa: E402
from test_gdr_more_gpu import close, run  # noqa: E402


def cut_into_segments(B, T, H, dk, dv, dtype):
    few, many = (sdm.gdr_workspace_bytes(n, T, H, H, dk, dv, DT[dtype]) for n in (B, 1000 * B))
    return few > many // 1000 + 4 * dk * dk


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [200, 900])
@pytest.mark.parametrize("value", [INF, NAN])
def test_only_a_reset_stops_a_value_that_is_not_finite(dtype, T, value):
    """Gates whose product is 0 in float32 (from 50 times e^-2 on) but none of which is by itself: every token's u takes what is not finite of its column
    into the state again, so the column stays that way, in a whole row and in segments; so does a gradient's, back in time."""
    say("gdr product of gates", dtype, T, value)
    x = make(1, T, 1, 1, 32, 40, dtype)
    assert cut_into_segments(1, T, 1, 32, 40, dtype) == (T == 900)
    x["g"].fill_(-2.0)
    clean = run(x)
    y = {n: None if t is None else t.clone() for n, t in x.items()}
    y["state"][0, 0, 3, 7] = value
    y["d_last"][0, 0, 5, 11] = value
    r = run(y)
    cols = torch.arange(40)
    for out in ("o", "last"):
        assert not torch.isfinite(r[out][..., 7]).any(), out
        close(out, r[out][..., cols != 7], clean[out][..., cols != 7])
    for out in ("dv", "dstate"):
        assert not torch.isfinite(r[out][..., 11]).any(), out
    close("dv", r["dv"][..., (cols != 7) & (cols != 11)], clean["dv"][..., (cols != 7) & (cols != 11)])
    assert not torch.isfinite(r["dk"]).any()
    # A reset ends it.
    for z in (y, x):
        z["g"][0, T // 2] = -INF
    r, clean = run(y), run(x)
    close("o", r["o"][:, T // 2:], clean["o"][:, T // 2:])
    close("last", r["last"], clean["last"])
    close("dv", r["dv"][:, :T // 2, :, cols != 7], clean["dv"][:, :T // 2, :, cols != 7])
    close("dstate", r["dstate"], clean["dstate"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,dk,dv", [(300, 24, 40), (1500, 32, 40), (1500, 128, 33)])
def test_no_tokens_leave_every_bit_of_a_state(dtype, T, dk, dv):
    """Infinities, subnormal values and zeros of either sign too: the state of a row without tokens, and its gradient."""
    say("gdr rows without tokens", dtype, T, dk, dv)
    lens = [0, T, -1]
    x = make(3, T, 1, 1, dk, dv, dtype, gate=4.0, lens=lens)
    assert cut_into_segments(3, T, 1, dk, dv, dtype) == (T == 1500)
    for name in ("state", "d_last"):
        for b in (0, 2):
            x[name][b, 0, 1, 2], x[name][b, 0, 2, 3], x[name][b, 0, 3, 4], x[name][b, 0, 4, 5], x[name][b, 0, 5, 6] = INF, -INF, 1e-40, -0.0, 3e-38
    r = run(x)
    bits = lambda t: t.cpu().view(torch.int32)  # noqa: E731
    for b in (0, 2):
        assert torch.equal(bits(r["last"][b]), bits(x["state"][b])), b
        assert torch.equal(bits(r["dstate"][b]), bits(x["d_last"][b])), b


@pytest.mark.parametrize("op", ["gdr", "glr"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_token_clears_what_a_prompt_clears(op, dtype):
    """Gates on both sides of where their factor is 0 (below 2^-126): a state that is not finite is gone after a prompt of one token if
    and only if it is gone after the token."""
    say("a token's gate", op, dtype)
    gates = [-0.5, -80.0, -87.0, -87.3, -87.33, -87.34, -87.5, -88.0, -90.0, -95.0, -100.0, -103.0, -103.9, -104.0, -150.0, -1e4, -1e30, -INF]
    border = torch.tensor(-126.0 / 1.4426950408889634)
    gates += [float(border + n * 2.0 ** -17) for n in range(-3, 4)]   # the float32 values next to it
    x = cuda(make(len(gates), 1, 2, 1, 16, 24, dtype))
    x["g"][:] = torch.tensor(gates, device="cuda")[:, None, None]
    ins = args(x) if op == "gdr" else args(x)[:4]
    forward, step = (sdm.gdr_forward, sdm.gdr_step) if op == "gdr" else (sdm.glr_forward, sdm.glr_step)
    for value in (INF, NAN, 1.0):
        state = torch.full_like(x["state"], value)
        o, last = forward(*ins, state=state)
        s = state.clone()
        p = step(*[t[:, 0] for t in ins], s)
        assert torch.equal(torch.isfinite(s), torch.isfinite(last)), value
        assert torch.equal(torch.isfinite(p), torch.isfinite(o[:, 0])), value
        gone = torch.isfinite(last).flatten(1).all(1)
        assert value == 1.0 or (not gone[:4].any() and gone[6:18].all())
    x["g"].fill_(NAN)   # which is no reset
    assert torch.isnan(step(*[t[:, 0] for t in ins], x["state"].clone())).all()
