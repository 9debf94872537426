"""GPU: the mixer kernels past the first trip of their loops, against plain evaluations in float64 on the GPU: segments
of several chunks in the recurrence (tiles loaded again, the other gate and tile buffers, states carried over chunks), a
norm team's walk over many heads and tokens, a slot-backward wave's next token.

Bounds as in test_glr_gpu.py, test_norm_rope_gpu.py and test_slot_topk_gpu.py; a norm weight's gradient is added up in chains
of at most 42 rows per team, 16 teams, 16 partial rows and 6 steps of a tree at the sizes here."""

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
from test_glr_gpu import DT, cuda, host, make, say  # noqa: E402


def plain(x, scale):
    """glr's results and magnitudes from the definition, token by token in float64: dicts of o, last, dq, dk, dv, dg, dstate."""
    q, k, v, d, g = (x[n].double() for n in ("q", "k", "v", "d_o", "g"))
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    per = H // Hk
    q, k = (t.repeat_interleave(per, 2) for t in (q, k))
    live = torch.ones(B, T, dtype=torch.bool, device="cuda") if x["lens"] is None else torch.arange(T, device="cuda") < x["lens"][:, None]
    z = (lambda *s: torch.zeros(s, dtype=torch.float64, device="cuda"))
    r, m = ({n: z(*s) for n, s in (("o", (B, T, H, dv)), ("dq", (B, T, H, dk)), ("dk", (B, T, H, dk)), ("dv", (B, T, H, dv)), ("dg", (B, T, H)))}
            for _ in range(2))
    S = z(B, H, dk, dv) if x["state"] is None else x["state"].double()
    A = S.abs()
    row = lambda t, s: (t[..., :, None] * s).sum(-2)  # noqa: E731
    col = lambda t, s: (t[..., None, :] * s).sum(-1)  # noqa: E731
    outer = lambda a, b: a[..., :, None] * b[..., None, :]  # noqa: E731
    before, part = [], z(B, T, H)
    for t in range(T):
        on = live[:, t, None, None, None]
        a = g[:, t].exp()[..., None, None]
        before.append(S)
        kv = outer(k[:, t], v[:, t])
        S, A = torch.where(on, a * S + kv, S), torch.where(on, a * A + kv.abs(), A)
        o = on[..., 0]
        r["o"][:, t], m["o"][:, t] = scale * row(q[:, t], S) * o, scale * row(q[:, t].abs(), A) * o
        r["dq"][:, t], m["dq"][:, t] = scale * col(d[:, t], S) * o, scale * col(d[:, t].abs(), A) * o
        part[:, t] = (q[:, t].abs() * m["dq"][:, t]).sum(-1)
    r["last"], m["last"] = S, A
    R = z(B, H, dk, dv) if x["d_last"] is None else x["d_last"].double()
    N = R.abs()
    rest = (A * N).sum((-1, -2))
    for t in range(T - 1, -1, -1):
        on = live[:, t, None, None, None]
        o = on[..., 0]
        a = g[:, t].exp()[..., None, None]
        qd = scale * outer(q[:, t], d[:, t])
        P, Q = R + qd, N + qd.abs()
        r["dk"][:, t], m["dk"][:, t] = col(v[:, t], P) * o, col(v[:, t].abs(), Q) * o
        r["dv"][:, t], m["dv"][:, t] = row(k[:, t], P) * o, row(k[:, t].abs(), Q) * o
        r["dg"][:, t] = (a * before[t] * P).sum((-1, -2)) * o[..., 0]
        rest = rest + (part[:, t] + (k[:, t].abs() * m["dk"][:, t]).sum(-1)) * o[..., 0]
        m["dg"][:, t] = rest
        R, N = torch.where(on, a * P, R), torch.where(on, a * Q, N)
    r["dstate"], m["dstate"] = R, N
    for n in ("dq", "dk"):
        for u in (r, m):
            u[n] = u[n].unflatten(2, (Hk, per)).sum(3)
    return r, m


def near(name, got, want, mag, n, bf):
    tol = n * 2.0 ** -23 * mag + 1e-30
    if bf:
        tol = tol + 4 * 2.0 ** -16 * mag + 2.0 ** -8 * want.abs()
    off = (got.double() - want).abs() / tol
    assert (off <= 1).all(), "%s: %d of %d off, worst %.3g of its bound" % (name, int((~(off <= 1)).sum()), off.numel(), float(off.max()))


def segments(B, T, H, Hk, dk, dv):
    """Segments of a row, from the workspace that holds their states and decays (none for one segment)."""
    size, up = sdm.glr_workspace_bytes(B, T, H, Hk, dk, dv), lambda n: -(-n // 256) * 256
    return 1 if size == 0 else next(n for n in range(2, T) if up(B * H * n * dk * dv * 4) + up(B * H * n * 4) == size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,Hk,dk,dv,ragged,chunks,nseg", [
    (64, 200, 4, 2, 24, 40, True, 4, 1),        # whole rows of four chunks
    (43, 600, 6, 3, 64, 120, False, 10, 1),
    (16, 330, 8, 8, 128, 128, True, 3, 2),      # segments of several chunks, joined by each block
    (4, 2500, 32, 8, 40, 72, False, 20, 2),
    (1, 16421, 8, 8, 64, 64, False, 9, 29),     # and chained
    (1, 2200, 2, 1, 16, 24, False, 1, 35),      # chained, more than are in flight at once
])
def test_segments_of_several_chunks(dtype, B, T, H, Hk, dk, dv, ragged, chunks, nseg):
    say("glr loops", dtype, B, T, H, Hk, dk, dv)
    got = segments(B, T, H, Hk, dk, dv)
    assert (got, -(-(-(-T // 64)) // got)) == (nseg, chunks), "other segments than these sizes are here for"
    lens = [max(0, T - 37 * b % (T + 5)) for b in range(B)] if ragged else None
    x = cuda(make(B, T, H, Hk, dk, dv, DT[dtype], lens=lens, gate=3.0))
    if lens is not None:
        for b, n in enumerate(lens):
            for name in ("q", "k", "v", "g", "d_o"):
                x[name][b, n:] = 0.25
    bf, n = dtype == "bf16", dk + dv + 96 + T // 64
    want, mag = plain(x, 0.3)
    args = [x[k] for k in ("q", "k", "v", "g")]
    o, last = sdm.glr_forward(*args, scale=0.3, state=x["state"], lens=x["lens"])
    near("o", o, want["o"], mag["o"], n, bf)
    near("last", last, want["last"], mag["last"], n, False)
    r = sdm.glr_backward(x["d_o"], *args, scale=0.3, state=x["state"], d_last=x["d_last"], lens=x["lens"])
    for name in ("dq", "dk", "dv"):
        near(name, r[name], want[name], mag[name], n + 2 * (H // Hk), bf)
    near("dg", r["dg"], want["dg"], mag["dg"], n, False)
    near("dstate", r["dstate"], want["dstate"], mag["dstate"], n, False)


def test_plain_is_the_oracle():
    x = make(3, 20, 4, 2, 7, 9, torch.float32, lens=[20, 0, 11])
    r, m = plain(cuda(x), 0.7)
    h = {n: host(t) for n, t in x.items()}
    o, last, mo, ml = M.glr_forward(h["q"], h["k"], h["v"], h["g"], 0.7, h["state"], h["lens"])
    w, wm = M.glr_backward(h["d_o"], h["q"], h["k"], h["v"], h["g"], 0.7, h["state"], h["d_last"], h["lens"])
    wm["dg"][h["lens"] == 0] = m["dg"].cpu().numpy()[h["lens"] == 0]
    for b, n in enumerate(h["lens"]):
        wm["dg"][b, n:] = m["dg"][b, n:].cpu().numpy()
    for got, want in ((r, dict(w, o=o, last=last)), (m, dict(wm, o=mo, last=ml))):
        for name in got:
            assert np.allclose(got[name].cpu().numpy(), want[name], rtol=1e-10, atol=1e-12), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_walks(dtype, inter):
    """21 heads per team and more tokens than 1024 blocks hold: the walks' further trips, queries and keys in one."""
    N, Hq, Hk, D, rot = 20011, 16, 5, 128, 64
    say("norm_rope walks", dtype, inter)
    gen = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, k, dq, dk = (rnd(N, h, D).to(DT[dtype]) for h in (Hq, Hk, Hq, Hk))
    w = 1 + 0.3 * rnd(2, D)
    pos, table = torch.arange(N, device="cuda"), sdm.rope_table(N, rot)
    a = dict(positions=pos, table=table, interleaved=inter)
    y = sdm.norm_rope(q, k, w[0], w[1], **a)
    r = sdm.norm_rope_backward(dq, dk, q, k, w[0], w[1], **a)
    c, s = table.double()[:, None].split(rot // 2, -1)
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    ulp, bf = 2.0 ** -23, 2.0 ** -8 if dtype == "bf16" else 0.0

    def turn(t, sin):
        u = t.clone()
        u[..., i], u[..., j] = t[..., i] * c - t[..., j] * sin, t[..., j] * c + t[..., i] * sin
        return u

    def size(t):   # the magnitudes of a pair's two columns, in both
        u = t.abs()
        both = u[..., i] + u[..., j]
        u[..., i], u[..., j] = both, both
        return u

    for n, x, d, u, out in (("q", q, dq, w[0], y[0]), ("k", k, dk, w[1], y[1])):
        x, d, u = x.double(), d.double(), u.double()
        rms = (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        nx = x * rms
        want = turn(nx * u, s)
        assert ((out.double() - want).abs() <= (D + 16) * ulp * size(nx * u) + bf * want.abs() + 1e-30).all(), n
        e, me = turn(d, -s), size(d)
        dx = rms * (e * u - nx * (e * u * nx).mean(-1, keepdim=True))
        mx = rms * (me * u.abs() + nx.abs() * (me * u.abs() * nx.abs()).mean(-1, keepdim=True))
        assert ((r["d" + n].double() - dx).abs() <= (D + 16) * ulp * mx + bf * dx.abs() + 1e-30).all(), n
        dw, mw = (e * nx).sum((0, 1)), (me * nx.abs()).sum((0, 1))
        assert ((r["dw" + n].double() - dw).abs() <= (42 + 16 + 16 + 6 + D + 16) * ulp * mw).all(), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n1,n2,K", [(40, 56, 8), (24, 17, 40)])
def test_slot_backward_walks(dtype, n1, n2, K):
    """More tokens than the launch has waves: a wave's row of sums is clean for its next token."""
    N, scale = 40001, 0.7
    say("slot backward walks", dtype, n1, n2, K)
    gen = torch.Generator(device="cuda").manual_seed(8)
    a, b = (torch.randn((N, n), generator=gen, device="cuda").to(DT[dtype]) for n in (n1, n2))
    y = torch.randn((N, K), generator=gen, device="cuda")
    idx, val = sdm.slot_topk(a, b, K, scale=scale)
    da, db = sdm.slot_topk_backward(y, idx, a, b, scale=scale)
    i, j = idx.long() // n2, idx.long() % n2
    p = ((a.double().gather(1, i) + b.double().gather(1, j)) * scale).softmax(1)
    assert ((val.double() - p).abs() <= (64 + K) * 2.0 ** -23 * p + 1e-37).all()
    y = y.double()
    d = scale * p * (y - (p * y).sum(1, keepdim=True))
    m = scale * p * (y.abs() + (p * y.abs()).sum(1, keepdim=True))
    for g, at, n in ((da, i, n1), (db, j, n2)):
        want, mag = (torch.zeros((N, n), dtype=torch.float64, device="cuda").scatter_add_(1, at, t) for t in (d, m))
        tol = (96 + 2 * K) * 2.0 ** -23 * mag + 1e-37 + (2.0 ** -8 * want.abs() if dtype == "bf16" else 0)
        assert ((g.double() - want).abs() <= tol).all()
