"""GPU: the gate's norm where its gates are so far out that exp(z) is near the smallest normal number."""

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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [60, 64, 520, 2056, 4104])
def test_gates_down_to_the_smallest_normal_silu(dtype, D):
    """silu(z) and its slope keep their digits while they are normal numbers, down to z = -91.8. Bounds as in test_block_norms_gpu.py;
    for float32 also |z| log2(e) / 2^24 / 4 for the exponent's two parts, less than one rounding more. Weights and gradients of 2^20
    keep results and factors away from subnormal numbers, where a rounding has no relative bound."""
    gen = torch.Generator(device="cuda").manual_seed(D)
    x, d = (torch.randn((4, 2, D), generator=gen, device="cuda").to(DT[dtype]) for _ in range(2))
    d = d * 2.0 ** 20
    z = torch.linspace(-91.5, -84, 8 * D, device="cuda")[torch.randperm(8 * D, generator=gen, device="cuda")].view(4, 2, D).to(DT[dtype])
    z[0, 0, 0], z[1, 1, 1] = 91.0, 300.0    # next to gates of the other side
    w = torch.full((D,), 2.0 ** 20, device="cuda")
    host = lambda t: t.float().cpu().numpy()  # noqa: E731
    want = M.gate_norm(host(x), host(z), host(w), 1e-6)
    g, m = M.gate_norm_backward(host(d), host(x), host(z), host(w), 1e-6)
    y, r = sdm.gate_norm(x, z, w), sdm.gate_norm_backward(d, x, z, w)

    def near(name, got, want, mag):
        got = got.float().cpu().numpy().astype(np.float64)
        tol = (21 + np.sqrt(D)) * 2.0 ** -23 * np.abs(mag) + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0.0)
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (name, bad.sum(), bad.size, (np.abs(got - want) / tol).max())
    near("y", y, want, want)
    near("dx", r["dx"], g["dx"], m["dx"])
    near("dz", r["dz"], g["dz"], m["dz"])
    # Far past it, and the other way.
    far = torch.tensor([-92.5, -104.0, -126.0, -200.0, -3e38, 200.0, 1e30, 3e38], device="cuda").to(DT[dtype]).view(1, 1, 8)
    one = torch.ones_like(far)
    y = sdm.gate_norm(one, far, eps=0.0)
    assert (y[0, 0, 3:5] == 0).all() and (y[0, 0, :3].abs() <= 1e-38).all() and torch.equal(y[0, 0, 5:], far[0, 0, 5:])
    r = sdm.gate_norm_backward(one, one, far, eps=0.0)
    assert (r["dz"][0, 0, 3:5] == 0).all() and (r["dz"][0, 0, :3].abs() <= 1e-38).all() and (r["dz"][0, 0, 5:] == 1).all()
