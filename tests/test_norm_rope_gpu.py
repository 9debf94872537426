"""GPU parity of the head norms with rotation (norm_rope, norm_rope_backward) with the float64 oracle.

Bounds: a head's sum of squares and dot are chains of at most D terms, and a result a handful of products
beside them: (D + 16) 2^-23 of the magnitude added up (for a turned column: of the pair's two columns),
then one rounding of a bfloat16 result, 2^-8 |value|. A weight's gradient sums N * H rows in partial sums of
at most N * H terms: (N H + D + 16) 2^-23 of its magnitude."""

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


def say(*a):
    print(*a, flush=True)


def host(t):
    return None if t is None else t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def near(name, got, want, mag, n, bf):
    got = host(got).astype(np.float64)
    tol = n * 2.0 ** -23 * mag + 1e-30 + (2.0 ** -8 * np.abs(want) if bf else 0.0)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (name, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / tol))


def pair_mag(y, plain, rot, inter):
    m = np.abs(plain)
    if rot:
        i, j = M._pairs(y.shape[-1], rot, inter)
        s = m[..., i] + m[..., j]
        m[..., i] = s
        m[..., j] = s
    return m


def run(N, Hq, Hk, D, rot, inter, dtype, weights="f32", pos64=False, kind="packed", eps=1e-6):
    gen = torch.Generator().manual_seed(5)
    bf, dt = dtype == "bf16", DT[dtype]
    rows = torch.randn((N, (Hq + Hk + 1) * D), generator=gen).to(dt).cuda()
    if N > 1:
        rows[1] = 0       # a head of zeros
        if N > 2:
            rows[2] *= 1e-4
    q, k = rows[:, :Hq * D].view(N, Hq, D), rows[:, Hq * D:(Hq + Hk) * D].view(N, Hk, D)
    if kind == "odd":     # one element off, and no multiple of 16 bytes between rows
        t = torch.zeros(N * ((Hq + Hk) * D + 3) + 1, dtype=dt, device="cuda")[1:].view(N, (Hq + Hk) * D + 3)
        t[:, :(Hq + Hk) * D] = rows[:, :(Hq + Hk) * D]
        q, k = t[:, :Hq * D].view(N, Hq, D), t[:, Hq * D:(Hq + Hk) * D].view(N, Hk, D)
    w = [None, None] if weights is None else [(1 + 0.3 * torch.randn(D, generator=gen)).to(DT[weights]).cuda() for _ in range(2)]
    table = sdm.rope_table(50, rot, scaling=2.0)
    pos = torch.randint(-3, 60, (N,), generator=gen).to(torch.int64 if pos64 else torch.int32).cuda()   # some outside the table
    a = dict(positions=pos, table=table, interleaved=inter, eps=eps)
    yq, yk = sdm.norm_rope(q, k, *w, **a)
    d = [torch.randn(t.shape, generator=gen).to(dt).cuda() for t in (q, k)]
    r = sdm.norm_rope_backward(*d, q, k, *w, **a)
    for n, x, ww, y, e in (("q", q, w[0], yq, d[0]), ("k", k, w[1], yk, d[1])):
        ha = (host(x), host(ww), host(pos), host(table))
        want = M.norm_rope(*ha, rot, inter, eps)
        plain = M.norm_rope(*ha, 0, inter, eps)
        near(n, y, want, pair_mag(want, plain, rot, inter), D + 16, bf)
        dx, dw, mx, mw = M.norm_rope_backward(host(e), *ha, rot, inter, eps)
        near("d" + n, r["d" + n], dx, mx, D + 16, bf)
        near("dw" + n, r["dw" + n], dw, mw, N * x.shape[1] + D + 16, False)
    return q, k, w, a, yq, yk, d, r


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("N,Hq,Hk,D,rot", [
    (1, 1, 1, 128, 128), (5, 4, 2, 64, 64), (3, 2, 1, 128, 64), (7, 3, 1, 120, 120), (4, 16, 4, 256, 64), (2, 1, 1, 512, 512),
    (9, 2, 2, 8, 8), (3, 2, 2, 128, 0), (600, 16, 4, 128, 128), (700, 3, 2, 72, 24),      # whole runs of four pairs
    (3, 2, 2, 6, 4), (4, 3, 1, 7, 2), (2, 1, 1, 1, 0), (5, 2, 1, 127, 62), (3, 1, 2, 511, 100), (650, 5, 1, 44, 36),  # any other
])
def test_matches_oracle(dtype, inter, N, Hq, Hk, D, rot):
    say("norm_rope", dtype, inter, N, Hq, Hk, D, rot)
    run(N, Hq, Hk, D, rot, inter, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(weights=None), dict(weights="bf16"), dict(pos64=True), dict(kind="odd"), dict(eps=0.5)])
def test_variants(dtype, kw):
    say("norm_rope variant", dtype, kw)
    run(37, 4, 2, 128, 64, False, dtype, **kw)


@pytest.mark.parametrize("kind", ["packed", "odd"])
def test_in_place_one_tensor_and_many_tokens(kind):
    q, k, w, a, yq, yk, d, r = run(2100, 16, 4, 64, 32, True, "bf16", kind=kind)
    only, none = sdm.norm_rope(q, None, w[0], None, **a)
    assert none is None and torch.equal(only, yq)
    only = sdm.norm_rope_backward(None, d[1], None, k, None, w[1], **a)
    # Fewer heads in the call, other partial sums: the rows' gradients are the same bits.
    assert only["dq"] is None and only["dwq"] is None and torch.equal(only["dk"], r["dk"])
    again = sdm.norm_rope_backward(*d, q, k, *w, **a)
    assert all(torch.equal(again[n], r[n]) for n in r)
    sdm.norm_rope(q, k, *w, q_out=q, k_out=k, **a)
    assert torch.equal(q, yq) and torch.equal(k, yk)


def test_empty_and_other_stream():
    e = torch.empty((0, 4, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    pos, table = torch.empty(0, dtype=torch.int32, device="cuda"), sdm.rope_table(8, 64)
    q, k = sdm.norm_rope(e, e, w, w, pos, table)
    assert q.shape == e.shape
    r = sdm.norm_rope_backward(e, e, e, e, w, w, pos, table)
    assert (r["dwq"] == 0).all() and (r["dwk"] == 0).all()
    x = torch.randn(300, 4, 64, device="cuda")
    want, _ = sdm.norm_rope(x, None, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = sdm.norm_rope(x, None, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


def test_graph_replays():
    x, d = torch.randn(4000, 6, 128, device="cuda").bfloat16(), torch.randn(4000, 6, 128, device="cuda").bfloat16()
    w, pos, table = torch.ones(128, device="cuda"), torch.arange(4000, device="cuda"), sdm.rope_table(4000, 128)
    f = lambda: (*sdm.norm_rope(x, None, w, None, pos, table)[:1], *[t for t in sdm.norm_rope_backward(d, None, x, None, w, None, pos, table).values() if t is not None])  # noqa: E731
    want = f()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = f()
    for rep in range(3):
        say("norm_rope graph replay", rep)
        for t in got:
            t.fill_(3.0)
        f()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_rope_table():
    t = sdm.rope_table(5, 6, base=100.0).cpu().double()
    ang = torch.arange(5, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(3, dtype=torch.float64) / 3)
    assert torch.allclose(t, torch.cat([ang.cos(), ang.sin()], 1), atol=1e-7)
    s = sdm.rope_table(9, 6, base=100.0, scaling=2.0).cpu()
    assert torch.allclose(s[::2], sdm.rope_table(5, 6, base=100.0).cpu(), atol=1e-6)
    b = sdm.rope_table(9, 6, base=100.0, base_growth=4.0).cpu().double()   # fastest as it was, slowest 4 times slower
    p = torch.arange(9, dtype=torch.float64)
    assert torch.allclose(b[:, 0], p.cos(), atol=1e-6) and torch.allclose(b[:, 2], (p * 100.0 ** (-2 / 3) / 4).cos(), atol=1e-6)
    assert sdm.rope_table(3, 0).shape == (3, 0)


def test_refusals():
    x, w = torch.randn(4, 2, 64, device="cuda"), torch.ones(64, device="cuda")
    pos, table = torch.zeros(4, dtype=torch.int32, device="cuda"), sdm.rope_table(8, 64)
    for bad in (lambda: sdm.norm_rope(None, None), lambda: sdm.norm_rope(x.half(), None), lambda: sdm.norm_rope(x, x.bfloat16()),
                lambda: sdm.norm_rope(x, None, w.half()), lambda: sdm.norm_rope(x, None, w, None, pos.float(), table),
                lambda: sdm.norm_rope(x, None, w, None, None, table), lambda: sdm.norm_rope(x.cpu(), None),
                lambda: sdm.norm_rope(x, None, w, None, pos, table.double()), lambda: sdm.norm_rope(x, x, w, w.bfloat16())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: sdm.norm_rope(x, x[:3]), lambda: sdm.norm_rope(x, None, w[:32]), lambda: sdm.norm_rope(x.transpose(1, 2), None),
                lambda: sdm.norm_rope(x, None, w, None, pos[:2], table), lambda: sdm.rope_table(4, 5), lambda: sdm.rope_table(4, 4, base=0.5)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sdm.norm_rope(x, None, eps=-1.0), lambda: sdm.norm_rope(x, None, eps=float("nan")),
                lambda: sdm.norm_rope(x[:, :, :32], None, None, None, pos, table),
                lambda: sdm.norm_rope(torch.randn(2, 1, 513, device="cuda"), None)):
        with pytest.raises(sdm.SdmError):
            bad()
