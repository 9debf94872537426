"""GPU: the block's norms past the first trip of their loops: rows that a team has loaded ahead, the other slots of its sums, its walk
from head to head. Bounds as in test_block_norms_gpu.py, a weight's gradient being a sum over all rows."""

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
from oracle import mixer as M  # noqa: E402
from test_block_norms_gpu import DT, EPS, heads, host, near, say  # noqa: E402

# More rows than 2048 blocks take at once: 32, 16, 8 and 4 of a block's teams of 8 to 64 lanes, one of longer rows; teams of 64 lanes
# with narrow accesses (D = 129, `odd`).
GATE = [(23400, 3, 64, "whole"), (11000, 3, 128, "part"), (5500, 3, 200, "whole"), (2800, 3, 264, "whole"), (2800, 3, 129, "odd"), (1500, 3, 600, "whole"),
        (1100, 2, 2056, "whole"), (700, 3, 4104, "whole")]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H,D,layout", GATE)
def test_gate_norm(dtype, N, H, D, layout):
    say("gate_norm loops", dtype, N, H, D, layout)
    x, z, d = heads(N, H, D, dtype, layout, seed=D)
    w, bf = 1 + 0.1 * torch.randn(D, device="cuda"), dtype == "bf16"
    want = M.gate_norm(host(x), host(z), host(w), EPS)
    near("y", sdm.gate_norm(x, z, w, eps=EPS), want, want, D, bf)
    r = sdm.gate_norm_backward(d, x, z, w, eps=EPS)
    g, m = M.gate_norm_backward(host(d), host(x), host(z), host(w), EPS)
    near("dx", r["dx"], g["dx"], m["dx"], D, bf)
    near("dz", r["dz"], g["dz"], m["dz"], D, bf)
    near("dw", r["dw"], g["dw"], m["dw"], D + N * H, False)
    inplace = sdm.gate_norm(x, z, w, eps=EPS)
    assert torch.equal(sdm.gate_norm(x, z, w, eps=EPS, out=x), inplace)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norm_y", [True, False])
@pytest.mark.parametrize("N,D,pad", [(67000, 64, 0), (9000, 260, 0), (8500, 130, 1), (4500, 600, 0), (2300, 2056, 8), (2100, 4104, 0)])
def test_residual_norm(dtype, norm_y, N, D, pad):
    say("residual_norm loops", dtype, norm_y, N, D, pad)
    gen = torch.Generator(device="cuda").manual_seed(N + D)
    x, y, dh, dn = (torch.randn((N, D + pad), generator=gen, device="cuda").to(DT[dtype])[:, pad:] for _ in range(4))
    w, a, wy = (c + 0.1 * torch.randn(D, generator=gen, device="cuda") for c in (1.0, 0.3, 1.0))
    wy = wy if norm_y else None
    more, bf = dict(weight=w, scale=a, norm_y=norm_y, y_weight=wy, eps=EPS), dtype == "bf16"
    h, n = sdm.residual_norm(x, y, **more)
    wh, wn, mh = M.residual_norm(host(x), host(y), host(w), host(a), norm_y, host(wy), EPS, host(h))
    near("h", h, wh, mh, D, bf)
    near("n", n, wn, wn, D, bf)
    r = sdm.residual_norm_backward(dh, dn, h, y, **more)
    g, m = M.residual_norm_backward(host(dh), host(dn), host(h), host(y), host(w), host(a), norm_y, host(wy), EPS)
    near("dx", r["dx"], g["dx"], m["dx"], D, bf)
    near("dy", r["dy"], g["dy"], m["dy"], 2 * D, bf)
    for name in ("dw", "dscale") + (("dwy",) if norm_y else ()):
        near(name, r[name], g[name], m[name], 2 * D + N, False)
    sdm.residual_norm(x, y, out=x, norm=y, **more)
    assert torch.equal(x, h) and torch.equal(y, n)
