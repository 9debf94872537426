"""GPU: the digits that every result of the delta rule keeps, by the measure of gdr_digits.py, in whole rows and in rows cut into segments."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import gdr_digits as D  # noqa: E402
import sparse_delta_memory_amd as sdm  # noqa: E402
from oracle import mixer as M  # noqa: E402
from test_gdr_gpu import DT, args, host, make, say  # noqa: E402
from test_gdr_more_gpu import run  # noqa: E402


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,Hk,dk,dv", D.SHAPES + D.SEGMENTED)
def test_digits(dtype, B, T, H, Hk, dk, dv):
    say("gdr digits", dtype, B, T, H, Hk, dk, dv)
    few, many = (sdm.gdr_workspace_bytes(n, T, H, Hk, dk, dv, DT[dtype]) for n in (B, 1000 * B))
    assert (few > many // 1000 + 4 * dk * dk) == ((B, T, H, Hk, dk, dv) in D.SEGMENTED)
    x = make(B, T, H, Hk, dk, dv, dtype)
    h = {n: host(t) for n, t in x.items()}
    got = run(x)
    o, last, _, _ = M.gdr_forward(*args(h), 0.3, h["state"])
    want = dict(o=o, last=last, **M.gdr_backward(h["d_o"], *args(h), 0.3, h["state"], h["d_last"])[0])
    for name in D.OUTPUTS:
        D.check(name, got[name].float().cpu().numpy(), want[name], dk, dv, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_token_keeps_them_too(dtype):
    x = make(40, 1, 4, 2, 128, 120, dtype)
    h = {n: host(t) for n, t in x.items()}
    o, last, _, _ = M.gdr_forward(*args(h), 0.3, h["state"])
    s = x["state"].cuda()
    got = sdm.gdr_step(*[t[:, 0].cuda() for t in args(x)], s, scale=0.3)
    D.check("o", got.float().cpu().numpy(), o[:, 0], 128, 120, dtype == "bf16")
    D.check("last", s.cpu().numpy(), last, 128, 120, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t0", [0, 40])
def test_chunks_taken_token_by_token_keep_them(dtype, t0):
    """A key that is not finite, alone between two resets: its chunk goes by the definition, and all other tokens' results are those
    of finite keys."""
    x = make(1, 64, 3, 3, 96, 72, dtype)
    x["g"][0, t0] = x["g"][0, t0 + 1] = -float("inf")
    h = {n: host(t) for n, t in x.items()}
    o, last, _, _ = M.gdr_forward(*args(h), 0.3, h["state"])
    want = dict(o=o, last=last, **M.gdr_backward(h["d_o"], *args(h), 0.3, h["state"], h["d_last"])[0])
    x["k"] = x["k"].clone()
    x["k"][0, t0, :, 5] = float("nan")
    got = run(x)
    others = [t for t in range(64) if t != t0]
    for name in D.OUTPUTS:
        if name == "dstate" and t0 == 0:
            assert (got[name] == 0).all()   # cut off by the first token
            continue
        a, b = got[name].float().cpu().numpy(), want[name]
        a, b = (a, b) if name in ("last", "dstate") else (a[:, others], b[:, others])
        D.check(name, a, b, 96, 72, dtype == "bf16")
