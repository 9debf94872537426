"""GPU: a prompt run through the delta-rule block in parts, and its backward pass through the states carried between them."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sparse_delta_memory_amd.mixer import DeltaBlock  # noqa: E402


@pytest.mark.parametrize("norm_y", [True, False])
def test_parts_have_the_gradients_of_the_whole(norm_y):
    """float32: both ways are the same sums in another order, a few hundred roundings of 2^-24 of sums of both signs; 1e-4 of the
    largest element, as for the block's own gradients. The parts are views of the whole rows."""
    b = DeltaBlock(model=72, heads=4, key_heads=2, d=32, rot=16, norm_y=norm_y, dtype=torch.float32, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    P, T, cut = 2, 190, 70
    x, n, d_x, d_n = (torch.randn((P, T, 72), generator=gen, device="cuda") for _ in range(4))
    state, d_state = (torch.randn((P, 4, 32, 32), generator=gen, device="cuda") * 0.3 for _ in range(2))
    h, m, last, saved = b.prompt(x, n, state)
    want = b.backward(d_x, d_n, saved, d_state=d_state)
    h1, m1, mid, saved1 = b.prompt(x[:, :cut], n[:, :cut], state)
    h2, m2, end, saved2 = b.prompt(x[:, cut:], n[:, cut:], mid, start=cut)
    g2 = b.backward(d_x[:, cut:], d_n[:, cut:], saved2, d_state=d_state)
    g1 = b.backward(d_x[:, :cut], d_n[:, :cut], saved1, d_state=g2["state"])

    def near(name, got, want):
        assert float((got - want).abs().max()) <= 1e-4 * float(want.abs().max()), name
    near("h", torch.cat([h1, h2], 1), h)
    near("n", torch.cat([m1, m2], 1), m)
    near("last", end, last)
    for name in ("x", "n"):
        near(name, torch.cat([g1[name], g2[name]], 1), want[name])
    near("state", g1["state"], want["state"])
    for name in ("w", "w_out", "o_norm", "scale", "next_norm") + (("y_norm",) if norm_y else ()):
        near(name, g1[name] + g2[name], want[name])
    assert norm_y or g1["y_norm"] is None
    # Without it the last state's gradient is 0.
    none, zero = b.backward(d_x, d_n, saved), b.backward(d_x, d_n, saved, d_state=torch.zeros_like(d_state))
    assert torch.equal(none["state"], zero["state"]) and torch.equal(none["w"], zero["w"])
    assert not torch.equal(none["w"], want["w"])
    # So is x's.
    none, zero = b.backward(None, d_n, saved), b.backward(torch.zeros_like(d_x), d_n, saved)
    assert all(none[k] is zero[k] is None or torch.equal(none[k], zero[k]) for k in zero)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_as_views_of_their_rows(dtype):
    b = DeltaBlock(dtype=dtype, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, n = (torch.randn((3, 7, 256), generator=gen, device="cuda").to(dtype) for _ in range(2))
    one, two = (b.prompt(x[:, :5], n[:, :5])[2] for _ in range(2))
    for t in (5, 6):
        h, m = b.token(x[:, t], n[:, t], one, t)
        k, p = b.token(x[:, t].contiguous(), n[:, t].contiguous(), two, t)
        assert torch.equal(h, k) and torch.equal(m, p)
    assert torch.equal(one, two)
