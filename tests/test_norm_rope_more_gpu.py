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


@pytest.mark.parametrize("D", [8, 6])      # whole runs of four pairs; any other
def test_many_heads(D):
    """524288 tokens of 64 + 8 heads (more than 2^25): a plain evaluation in float64 of the first and last tokens and of those
    around 2^25 heads, and every token as in calls of fewer."""
    N, Hq, Hk = 1 << 19, 64, 8
    say("norm_rope of many heads", N * (Hq + Hk), D)
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k = (torch.randn((N, h, D), generator=gen, device="cuda").bfloat16() for h in (Hq, Hk))
    w = 1 + 0.1 * torch.randn((2, D), generator=gen, device="cuda")
    pos, table = torch.arange(N, device="cuda") % 500, sdm.rope_table(500, 4)
    yq, yk = sdm.norm_rope(q, k, w[0], w[1], pos, table)
    edge = (1 << 25) // (Hq + Hk)
    for at in (slice(0, 4), slice(edge - 3, edge + 3), slice(N - 4, N)):
        for x, y, u in ((q, yq, w[0]), (k, yk, w[1])):
            z = x[at].double()
            z = z / (z.square().mean(-1, keepdim=True) + 1e-6).sqrt() * u.double()
            c, s = table[pos[at]].double()[:, None].split(2, -1)
            z[..., :4] = torch.cat([z[..., :2] * c - z[..., 2:4] * s, z[..., 2:4] * c + z[..., :2] * s], -1)
            assert ((y[at].double() - z).abs() <= 2.0 ** -8 * z.abs() + (D + 16) * 2.0 ** -23 * 8).all()
    for t in range(0, N, 1 << 17):
        at = slice(t, t + (1 << 17))
        a, b = sdm.norm_rope(q[at], k[at], w[0], w[1], pos[at], table)
        assert torch.equal(yq[at], a) and torch.equal(yk[at], b)
    r = sdm.norm_rope_backward(yq, yk, q, k, w[0], w[1], pos, table)
    for t in range(0, N, 1 << 17):
        at = slice(t, t + (1 << 17))
        p = sdm.norm_rope_backward(yq[at], yk[at], q[at], k[at], w[0], w[1], pos[at], table)
        assert torch.equal(r["dq"][at], p["dq"]) and torch.equal(r["dk"][at], p["dk"])
