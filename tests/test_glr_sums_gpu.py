"""GPU: bfloat16 rows of the gated linear recurrence whose sums cancel. What enters a product as a float32 value (a decayed
score, a state) keeps its 24 bits there. With few terms that shows: a result is the sum of dk products with a state (no values
in the row) or of two tokens' scores, each term with a handful of roundings of its factors, so it is within
(dk + 26) 2^-23 of the sum over absolute values, beside one rounding of the result, 2^-8 |value|, however small that is."""

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
from test_glr_gpu import cuda, host, make, say  # noqa: E402


@pytest.mark.parametrize("kind,B,T", [("state", 8, 40), ("scores", 64, 2)])
@pytest.mark.parametrize("dk,dv", [(2, 64), (8, 128), (16, 24)])
def test_cancelling_sums_keep_float32(kind, B, T, dk, dv):
    say("glr cancelling sums", kind, B, T, dk, dv)
    x = make(B, T, 2, 2, dk, dv, torch.bfloat16, state=kind == "state")
    x["g"][:] = -2.0 ** -10
    if kind == "state":       # rows of the states in pairs that all but cancel in the product with a row of equal pairs
        for n in ("q", "k"):
            x[n][..., 1::2] = x[n][..., ::2]
        for n in ("state", "d_last"):
            x[n][:, :, 1::2] = -x[n][:, :, ::2] * (1 + 2.0 ** -12)
        x["v"][:] = 0
        x["d_o"][:] = 0
    else:                     # two tokens that all but cancel
        for n in ("q", "k", "v", "d_o"):
            x[n][:, 1] = x[n][:, 0] * (1 if n in ("q", "k") else -1)
    d, h = cuda(x), {n: host(t) for n, t in x.items()}
    args = [d[n] for n in ("q", "k", "v", "g")]
    o, _ = sdm.glr_forward(*args, scale=1.0, state=d["state"])
    r = sdm.glr_backward(d["d_o"], *args, scale=1.0, state=d["state"], d_last=d["d_last"])
    wo, _, mo, _ = M.glr_forward(h["q"], h["k"], h["v"], h["g"], 1.0, h["state"])
    w, m = M.glr_backward(h["d_o"], h["q"], h["k"], h["v"], h["g"], 1.0, h["state"], h["d_last"])
    last = -1 if kind == "scores" else slice(None)      # the second token's o, the first one's dv
    for name, got, want, mag, at in (("o", o, wo, mo, last), ("dv", r["dv"], w["dv"], m["dv"], 0 if kind == "scores" else last)):
        got, want, mag = got.float().cpu().numpy().astype(np.float64)[:, at], want[:, at], mag[:, at]
        tol = (dk + 26) * 2.0 ** -23 * mag + 2.0 ** -8 * np.abs(want) + 1e-30
        off = np.abs(got - want) / tol
        assert np.median(np.abs(want) / (mag + 1e-30)) < 2.0 ** -8      # they do cancel
        assert (off <= 1).all(), "%s: %d of %d off, worst %.3g of its bound" % (name, (off > 1).sum(), off.size, off.max())
