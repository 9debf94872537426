"""GPU: calls of norm_rope and norm_rope_backward beside test_norm_rope_gpu.py's (whose bounds hold here too)."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_delta_memory_amd as sdm  # noqa: E402


def say(*a):
    print(*a, flush=True)


def test_weights_without_heads_are_not_read():
    """The weights of a tensor that is not given: of another length, type and alignment, they change nothing."""
    x, d = torch.randn(70, 3, 128, device="cuda"), torch.randn(70, 3, 128, device="cuda")
    w, other = torch.randn(128, device="cuda"), torch.randn(8, device="cuda").bfloat16()[1:4]
    say("norm_rope with weights of no heads")
    want = sdm.norm_rope(None, x, None, w)[1]
    assert torch.equal(sdm.norm_rope(None, x, other, w)[1], want)
    assert torch.equal(sdm.norm_rope(x, None, w, other)[0], want)
    back = sdm.norm_rope_backward(None, d, None, x, None, w)
    for r, n in ((sdm.norm_rope_backward(None, d, None, x, other, w), "k"), (sdm.norm_rope_backward(d, None, x, None, w, other), "q")):
        assert torch.equal(r["d" + n], back["dk"]) and torch.equal(r["dw" + n], back["dwk"])
    # No heads at all in a tensor that is given.
    none = x[:, :0]
    assert torch.equal(sdm.norm_rope(none, x, w, w)[1], want)
