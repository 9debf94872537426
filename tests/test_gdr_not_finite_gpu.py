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
