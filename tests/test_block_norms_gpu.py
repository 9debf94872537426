"""GPU parity of gate_norm and residual_norm, forward and backward, with the float64 oracle.

Bounds: a float32 result is off by the roundings on its way, (16 + sqrt of the terms of its longest sum) 2^-23 times the
magnitude of what is added up (a row's mean of squares errs by its terms' roundings in quadrature, and its root by half
of that); gates' sigmoids by 4 more. A bfloat16 result is rounded once more, 2^-8 |value|.
"""

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
EPS = 1e-5


def say(*a):
    print(*a, flush=True)


def host(x):
    return None if x is None else x.float().cpu().numpy()


def near(name, got, want, mag, terms, bf):
    got = got.float().cpu().numpy().astype(np.float64)
    tol = (20 + np.sqrt(terms)) * 2.0 ** -23 * np.abs(mag) + 1e-37 + (2.0 ** -8 * np.abs(want) if bf else 0.0)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (name, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / tol))


def heads(N, H, D, dtype, layout, seed=0):
    """x, z, d: whole, or parts of wider rows; `odd`: rows that start on no 16 bytes."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i in range(3):
        if layout == "whole":
            t = torch.randn((N, H, D), generator=gen, device="cuda").to(DT[dtype])
        else:
            pad = 8 * (i + 1) if layout == "part" else 1 + i
            t = torch.randn((N, H * D + pad), generator=gen, device="cuda").to(DT[dtype])[:, pad:].view(N, H, D) if layout == "part" else \
                torch.randn((N, H, D + pad), generator=gen, device="cuda").to(DT[dtype])[..., pad:]
        out.append(t * (3.0 if i == 1 else 1.0) if layout == "whole" else t)
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H,D,layout,weight", [
    (1, 1, 1, "whole", True), (3, 2, 8, "whole", True), (5, 3, 64, "part", True), (700, 5, 128, "part", True), (9, 4, 120, "whole", False),
    (37, 3, 72, "odd", True), (11, 1, 200, "whole", True), (6, 2, 512, "whole", True), (3, 1, 513, "whole", True), (4, 2, 1000, "part", True),
    (2, 1, 2049, "whole", True), (3, 1, 4096, "whole", True), (3, 2, 8192, "whole", True), (2, 1, 8191, "odd", False), (5000, 4, 16, "whole", True)])
def test_gate_norm(dtype, N, H, D, layout, weight):
    say("gate_norm", dtype, N, H, D, layout, weight)
    x, z, d = heads(N, H, D, dtype, layout)
    w = 1 + 0.1 * torch.randn(D, device="cuda") if weight else None
    if weight and N % 2:
        w = w.bfloat16()
    bf = dtype == "bf16"
    want = M.gate_norm(host(x), host(z), host(w), EPS)
    y = sdm.gate_norm(x, z, w, eps=EPS)
    near("y", y, want, want, D, bf)
    r = sdm.gate_norm_backward(d, x, z, w, eps=EPS)
    g, m = M.gate_norm_backward(host(d), host(x), host(z), host(w), EPS)
    near("dx", r["dx"], g["dx"], m["dx"], D, bf)
    near("dz", r["dz"], g["dz"], m["dz"], D, bf)
    if weight:
        near("dw", r["dw"], g["dw"], m["dw"], D + N * H, False)
    else:
        assert r["dw"] is None
    # The same bits again, and in place of either input.
    again = sdm.gate_norm_backward(d, x, z, w, eps=EPS)
    assert all(r[k] is None or torch.equal(r[k], again[k]) for k in r)
    x2, z2 = x.clone(), z.clone()
    assert torch.equal(sdm.gate_norm(x2, z, w, eps=EPS, out=x2), y) and torch.equal(sdm.gate_norm(x, z2, w, eps=EPS, out=z2), y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gate_norm_extremes(dtype):
    """Gates far out on either side, rows of zeros, rows of large and of tiny values, values that are not finite."""
    D = 64
    x = torch.randn((8, 1, D), device="cuda")
    z = torch.linspace(-300, 300, 8 * D, device="cuda").view(8, 1, D)
    x[1] = 0
    x[2] *= 1e15
    x[3] *= 1e-20
    x, z = x.to(DT[dtype]), z.to(DT[dtype])
    want = M.gate_norm(host(x), host(z), None, EPS)
    # |z| exp(z) below the smallest normal number comes out as 0
    near("y", sdm.gate_norm(x, z, eps=EPS), want, np.maximum(np.abs(want), 1e-30), D, dtype == "bf16")
    clean = sdm.gate_norm(x, z, eps=EPS)
    x[4, 0, 3], z[5, 0, 7] = float("inf"), float("nan")
    y = sdm.gate_norm(x, z, eps=EPS)
    keep = [0, 1, 2, 3, 6, 7]
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[5, 0, 7]) and torch.equal(y[5, 0, :7], clean[5, 0, :7])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norm_y,scaled,weights", [(False, False, True), (True, True, True), (True, False, False), (False, True, True)])
@pytest.mark.parametrize("N,D,layout", [(1, 1, "whole"), (5, 8, "whole"), (7, 100, "odd"), (33, 256, "part"), (3000, 64, "whole"), (9, 520, "part"),
                                        (1500, 768, "whole"), (4, 2048, "whole"), (3, 2056, "part"), (2, 4097, "whole"), (5, 8192, "whole")])
def test_residual_norm(dtype, norm_y, scaled, weights, N, D, layout):
    say("residual_norm", dtype, norm_y, scaled, weights, N, D, layout)
    gen = torch.Generator(device="cuda").manual_seed(N + D)
    pad = dict(whole=0, part=8, odd=3)[layout]
    x, y, dh, dn = (torch.randn((N, D + pad), generator=gen, device="cuda").to(DT[dtype])[:, pad:] for _ in range(4))
    vec = lambda on, c: c + 0.1 * torch.randn(D, generator=gen, device="cuda") if on else None  # noqa: E731
    w, a, wy = vec(weights, 1.0), vec(scaled, 0.3), vec(norm_y and weights, 1.0)
    more = dict(weight=w, scale=a, norm_y=norm_y, y_weight=wy, eps=EPS)
    bf = dtype == "bf16"
    h, n = sdm.residual_norm(x, y, **more)
    wh, wn, mh = M.residual_norm(host(x), host(y), host(w), host(a), norm_y, host(wy), EPS, host(h))
    near("h", h, wh, mh, D, bf)
    near("n", n, wn, wn, D, bf)
    for given in (dh, None):
        r = sdm.residual_norm_backward(given, dn, h, y, **more)
        g, m = M.residual_norm_backward(host(given), host(dn), host(h), host(y), host(w), host(a), norm_y, host(wy), EPS)
        near("dx", r["dx"], g["dx"], m["dx"], D, bf)
        near("dy", r["dy"], g["dy"], m["dy"], 2 * D, bf)
        for name, on in (("dw", weights), ("dscale", scaled), ("dwy", norm_y and weights)):
            if on:
                near(name, r[name], g[name], m[name], 2 * D + N, False)
            else:
                assert r[name] is None
    # In place: h over x, n over y.
    x2, y2 = x.clone(), y.clone()
    sdm.residual_norm(x2, y2, out=x2, norm=y2, **more)
    assert torch.equal(x2, h) and torch.equal(y2, n)
    y2, x2 = y.clone(), x.clone()
    sdm.residual_norm(x2, y2, out=y2, norm=x2, **more)
    assert torch.equal(y2, h) and torch.equal(x2, n)


def test_no_rows_and_leading_dimensions():
    x = torch.randn((2, 3, 40), device="cuda")
    y, w = torch.randn((2, 3, 40), device="cuda"), torch.randn(40, device="cuda")
    h, n = sdm.residual_norm(x, y, w)
    h2, n2 = sdm.residual_norm(x.view(6, 40), y.view(6, 40), w)
    assert h.shape == x.shape and torch.equal(h.view(6, 40), h2) and torch.equal(n.view(6, 40), n2)
    e = torch.empty((0, 40), device="cuda")
    h, n = sdm.residual_norm(e, e, w)
    assert h.shape == e.shape
    r = sdm.residual_norm_backward(None, e, e, e, w, scale=w)
    assert (r["dw"] == 0).all() and (r["dscale"] == 0).all()
    e = torch.empty((0, 2, 40), device="cuda")
    assert sdm.gate_norm(e, e, w).shape == e.shape
    assert (sdm.gate_norm_backward(e, e, e, w)["dw"] == 0).all()
