"""GPU parity of slot selection (slot_topk, slot_topk_backward) with the oracle: the ids exactly, the weights and
gradients within float32 bounds. A weight's exponent is a float32 difference times scale (|x| up to x_max here),
so the weight is within (x_max + K + 16) 2^-23 of itself; a gradient within as much of its magnitude, with the
float32 rounding of the sums beside it."""

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
    return t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy().astype(np.int64)


def check(a, b, K, scale=1.0, **kw):
    idx, val = sdm.slot_topk(a, b, K, scale=scale, **kw)
    ha, hb = host(a).reshape(-1, a.shape[-1]), host(b).reshape(-1, b.shape[-1])
    wi, wv = M.slot_topk(ha, hb, K, scale)
    got = host(idx).reshape(-1, K)
    bad = np.argwhere((got != wi).any(1))
    assert not len(bad), "row %d: %s, expected %s" % (bad[0, 0], got[bad[0, 0]], wi[bad[0, 0]])
    gv = host(val).reshape(-1, K).astype(np.float64)
    tol = (64 + K) * 2.0 ** -23 * wv + 1e-37 + (2.0 ** -8 * wv if val.dtype == torch.bfloat16 else 0)
    assert (np.abs(gv - wv) <= tol).all(), np.max(np.abs(gv - wv) / tol)
    dval = torch.randn(idx.shape, generator=torch.Generator().manual_seed(2)).cuda()
    da, db = sdm.slot_topk_backward(dval, idx, a, b, scale=scale)
    wa, wb, ma, mb = M.slot_topk_backward(host(dval).reshape(-1, K), wi, ha, hb, scale)
    for n, g, w, m in (("da", da, wa, ma), ("db", db, wb, mb)):
        g = host(g).reshape(w.shape).astype(np.float64)
        t = (96 + 2 * K) * 2.0 ** -23 * m + 1e-37 + (2.0 ** -8 * np.abs(w) if a.dtype == torch.bfloat16 else 0)
        assert (np.abs(g - w) <= t).all(), (n, np.max(np.abs(g - w) / t))
        assert (g[m == 0] == 0).all()
    return idx, val, da, db


def scores(N, n, dtype, seed, mul=1.0):
    return (torch.randn((N, n), generator=torch.Generator().manual_seed(seed)) * mul).to(DT[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,n1,n2,K", [
    (1, 1, 1, 1), (3, 1, 70, 64), (5, 64, 64, 4), (4, 65, 63, 8), (9, 128, 128, 16), (7, 130, 40, 33), (5, 256, 256, 64),
    (6, 512, 512, 32), (3, 1000, 1024, 17), (4, 2048, 2048, 32), (2, 4096, 4096, 64), (2, 4095, 300, 5), (3, 2, 3, 6), (66, 37, 41, 64),
    (5, 192, 136, 1),
])
def test_matches_oracle(dtype, N, n1, n2, K):
    say("slot_topk", dtype, N, n1, n2, K)
    check(scores(N, n1, dtype, 1), scores(N, n2, dtype, 2), K)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [40, 64, 200, 2048])
def test_ties_and_rows_without_order(dtype, n):
    """Equal scores everywhere, few distinct ones, rising and falling rows, both zeros."""
    say("slot_topk ties", dtype, n)
    a = scores(8, n, dtype, 3)
    a[0] = 0.25
    a[1] = torch.arange(n, device="cuda") % 3
    a[2] = torch.arange(n, device="cuda") / n
    a[3] = -torch.arange(n, device="cuda") / n
    a[4] = 0.0
    a[4, ::2] = -0.0
    a[5] = (torch.arange(n, device="cuda") // 7 % 5).to(a.dtype)
    b = a.flip(0).contiguous()
    for K in (1, 5, 32, 40):
        check(a, b, K)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [48, 300])
def test_masked_scores(dtype, n):
    """Rows with few, one or no scores left, by -infinity, NaN or the type's lowest value."""
    say("slot_topk masks", dtype, n)
    low = torch.finfo(DT[dtype]).min
    a, b = scores(7, n, dtype, 4), scores(7, n, dtype, 5)
    a[0] = float("-inf")
    b[1] = float("nan")
    a[2] = float("-inf")
    a[2, n // 2] = 1.0
    b[2] = float("-inf")
    b[2, 3] = 0.5
    a[3, 5:] = float("nan")
    a[4] = low
    a[4, 7] = 2.0
    a[5] = low
    b[5] = low           # sums overflow to -infinity
    a[6, ::2] = float("-inf")
    idx, val, da, db = check(a, b, 8)
    assert (val[0] == 0).all() and (val[1] == 0).all() and val[2, 0] == 1 and (val[2, 1:] == 0).all() and (val[5] == 0).all()
    assert (idx >= 0).all() and (idx < n * n).all() and torch.isfinite(da).all() and torch.isfinite(db).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_types_strides_and_scale(dtype):
    a, b = scores(20, 256, dtype, 6), scores(20, 192, dtype, 7)
    idx, val, _, _ = check(a, b, 12, scale=0.125)
    i64, v16, _, _ = check(a, b, 12, scale=0.125, idx_dtype=torch.int64, val_dtype=torch.bfloat16)
    assert torch.equal(i64, idx.long()) and torch.equal(v16, val.bfloat16())
    both = torch.cat([a, b], 1)          # halves of one projection's rows
    i2, v2 = sdm.slot_topk(both[:, :256], both[:, 256:], 12, scale=0.125)
    assert torch.equal(i2, idx) and torch.equal(v2, val)
    odd = torch.zeros((20, 451), dtype=a.dtype, device="cuda")[:, 1:]
    odd[:, :256] = a
    odd[:, 256:448] = b
    i2, v2 = sdm.slot_topk(odd[:, :256], odd[:, 256:448], 12, scale=0.125)
    assert torch.equal(i2, idx) and torch.equal(v2, val)


def test_feeds_phase1():
    """Absolute ids of a Phase-1 shape's chunks, in its layouts."""
    N, C, P, n, K = 6, 8, 3, 16, 4
    shape = sdm.make_shape(N, C, K, K, P=P, key_bits=8, stream_offset=n * n)
    a, b = scores(N * C, n, "f32", 8).view(N, C, n), scores(N * C, n, "f32", 9).view(N, C, n)
    loc, val = sdm.slot_topk(a, b, K)
    idx, val2 = sdm.slot_topk(a, b, K, shape=shape)
    off = (torch.arange(N, device="cuda") % P * n * n).view(N, 1, 1)
    assert torch.equal(idx, (loc + off).int()) and torch.equal(val, val2)
    dval = torch.randn(N, C, K, device="cuda")
    for x, y in zip(sdm.slot_topk_backward(dval, loc, a, b), sdm.slot_topk_backward(dval, idx, a, b, shape=shape)):
        assert x.shape == (N, C, n) and torch.equal(x, y)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sdm.phase1(shape, idx, idx, val, val, torch.zeros(N, C, device="cuda"), status=status)
    assert int(status) == 0


def test_bits_empty_and_graph():
    a, b = scores(5000, 512, "bf16", 10), scores(5000, 512, "bf16", 11)
    dval = torch.randn(5000, 32, device="cuda")

    def f():
        i, v = sdm.slot_topk(a, b, 32)
        return (i, v) + sdm.slot_topk_backward(dval, i, a, b)

    want = f()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = f()
    for rep in range(3):
        say("slot_topk graph replay", rep)
        for t in got:
            t.fill_(1)
        f()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))
    i, v = sdm.slot_topk(a[:0], b[:0], 4)
    assert i.shape == (0, 4)
    da, db = sdm.slot_topk_backward(dval[:0, :4].contiguous(), i, a[:0], b[:0])
    assert da.shape == (0, 512)


def test_refusals():
    a, b = scores(4, 32, "f32", 1), scores(4, 32, "f32", 2)
    for bad in (lambda: sdm.slot_topk(a.half(), b.half(), 4), lambda: sdm.slot_topk(a.cpu(), b, 4), lambda: sdm.slot_topk(a, b, 4, val_dtype=torch.half),
                lambda: sdm.slot_topk(a, b, 4, idx_dtype=torch.int16)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: sdm.slot_topk(a, b[:3], 4), lambda: sdm.slot_topk(a, b.bfloat16(), 4), lambda: sdm.slot_topk(a.t(), b.t(), 4),
                lambda: sdm.slot_topk(a, b, 4, idx=torch.empty(4, 5, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sdm.slot_topk(a, b, 65), lambda: sdm.slot_topk(a, b, 0), lambda: sdm.slot_topk(a[:, :1], b[:, :2], 3),
                lambda: sdm.slot_topk(a, b, 4, scale=0.0), lambda: sdm.slot_topk(a, b, 4, scale=float("nan")),
                lambda: sdm.slot_topk(scores(1, 4097, "f32", 1), scores(1, 8, "f32", 1), 4)):
        with pytest.raises(sdm.SdmError):
            bad()
