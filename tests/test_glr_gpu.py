"""GPU parity of the gated linear recurrence (glr_forward, glr_backward, glr_step) with the float64 oracle.

Bounds, per element, from the oracle's magnitude of the same sums over absolute values (mag):
- a float32 evaluation adds at most n = dk + dv + 64 + T/64 terms in a chain, and each term carries a few
  roundings of its gate factors: (n + 32) 2^-23 mag;
- bfloat16 inputs are exact, and what a rounded result uses of a score or a state is kept to 16 bits in
  each: 4 2^-16 mag beside it, then one rounding of the result, 2^-8 |value|.
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


def say(*a):
    print(*a, flush=True)


def make(B, T, H, Hk, dk, dv, dtype, seed=3, gate=2.0, state=True, lens=None, packed=False):
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x = dict(q=rnd(B, T, Hk, dk), k=rnd(B, T, Hk, dk) * dk ** -0.5, v=rnd(B, T, H, dv), d_o=rnd(B, T, H, dv))
    x = {n: t.to(dtype) for n, t in x.items()}
    x["g"] = torch.nn.functional.logsigmoid(rnd(B, T, H) + gate)
    x["state"] = rnd(B, H, dk, dv) * 0.3 if state else None
    x["d_last"] = rnd(B, H, dk, dv) * 0.3 if state else None
    x["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    return x


def host(x):
    return None if x is None else x.float().numpy() if x.is_floating_point() else x.numpy()


def cuda(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def near(name, got, want, mag, n, bf):
    got = got.float().cpu().numpy().astype(np.float64)
    tol = n * 2.0 ** -23 * mag + 1e-30
    if bf:
        tol = tol + 4 * 2.0 ** -16 * mag + 2.0 ** -8 * np.abs(want)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (
        name, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / tol))


def check(x, dtype, scale, dev=None):
    """Forward and backward of the host inputs x (device tensors: dev) against the oracle."""
    bf = dtype == torch.bfloat16
    d = cuda(x) if dev is None else dev
    B, T, Hk, dk = x["q"].shape
    H, dv = x["v"].shape[2:]
    n = dk + dv + 96 + T // 64
    h = {k: host(t) for k, t in x.items()}
    o, last = sdm.glr_forward(d["q"], d["k"], d["v"], d["g"], scale=scale, state=d["state"], lens=d["lens"])
    wo, wl, mo, ml = M.glr_forward(h["q"], h["k"], h["v"], h["g"], scale, h["state"], h["lens"])
    near("o", o, wo, mo, n, bf)
    near("last", last, wl, ml, n, False)
    r = sdm.glr_backward(d["d_o"], d["q"], d["k"], d["v"], d["g"], scale=scale, state=d["state"], d_last=d["d_last"], lens=d["lens"])
    w, m = M.glr_backward(h["d_o"], h["q"], h["k"], h["v"], h["g"], scale, h["state"], h["d_last"], h["lens"])
    for name in ("dq", "dk", "dv"):
        near(name, r[name], w[name], m[name], n + 2 * (H // Hk), bf)
    near("dg", r["dg"], w["dg"], m["dg"], n, False)
    near("dstate", r["dstate"], w["dstate"], m["dstate"], n, False)
    return o, last, r


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,Hk,dk,dv", [
    (1, 1, 1, 1, 64, 64), (2, 1, 2, 2, 128, 128), (1, 2, 1, 1, 1, 1), (1, 63, 1, 1, 64, 128), (1, 64, 2, 1, 128, 64),
    (2, 65, 1, 1, 120, 120), (1, 130, 3, 3, 9, 33), (1, 200, 4, 2, 64, 72), (2, 127, 2, 1, 65, 17), (1, 191, 1, 1, 128, 128),
])
def test_matches_oracle(dtype, B, T, H, Hk, dk, dv):
    say("glr", dtype, B, T, H, Hk, dk, dv)
    check(make(B, T, H, Hk, dk, dv, DT[dtype]), DT[dtype], dk ** -0.5)
    check(make(B, T, H, Hk, dk, dv, DT[dtype], state=False, seed=4), DT[dtype], 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,gate", [(700, 1, 2.0), (1090, 2, 6.0), (1024, 1, -2.0)])
def test_rows_cut_into_segments(dtype, T, H, gate):
    say("glr segments", dtype, T, H, gate)
    assert sdm.glr_workspace_bytes(1, T, H, 1, 48, 40) > 0
    check(make(1, T, H, 1, 48, 40, DT[dtype], gate=gate), DT[dtype], 0.2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,lens", [(150, [0, 150, 1, 64]), (600, [600, 0, 70, 300]), (100, [-3, 900, 100, 99])])
def test_lengths(dtype, T, lens):
    """Tokens past a row's length may hold anything; a row of no tokens keeps its state."""
    say("glr lens", dtype, T, lens)
    x = make(4, T, 2, 1, 24, 40, DT[dtype], lens=lens)
    d = cuda(x)
    for b, n in enumerate(lens):
        for name in ("q", "k", "v", "g", "d_o"):
            d[name][b, max(0, min(n, T)):] = float("nan")
    o, last, r = check(x, DT[dtype], 0.5, dev=d)
    for b, n in enumerate(lens):
        n = max(0, min(n, T))
        assert (o[b, n:] == 0).all() and (r["dq"][b, n:] == 0).all() and (r["dg"][b, n:] == 0).all()
        if n == 0:
            assert torch.equal(last[b], d["state"][b]) and torch.equal(r["dstate"][b], d["d_last"][b])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_resets_and_strong_gates(dtype):
    """Gates of -infinity (a new sequence starts), gates that leave almost nothing, and gates of 0."""
    x = make(1, 333, 2, 2, 32, 64, DT[dtype])
    x["g"][0, 0, 0] = float("-inf")
    x["g"][0, 70, :] = float("-inf")
    x["g"][0, 71, 1] = float("-inf")
    x["g"][0, 127, 0] = -1e30
    x["g"][0, 128:140] = -90.0
    x["g"][0, 200:300] = 0.0
    say("glr resets", dtype)
    check(x, DT[dtype], 0.3)


def views(x, kind):
    """The inputs as views a caller may have."""
    d = cuda(x)
    B, T, Hk, dk = x["q"].shape
    H, dv = x["v"].shape[2:]
    if kind == "packed":            # one projection's rows
        rows = torch.cat([d[n].flatten(2) for n in ("q", "k", "v")], 2)
        q, k, v = rows.split([Hk * dk, Hk * dk, H * dv], 2)
        d["q"], d["k"], d["v"] = q.view(B, T, Hk, dk), k.view(B, T, Hk, dk), v.view(B, T, H, dv)
    elif kind == "heads_first":     # [B, H, T, d] seen as [B, T, H, d]
        for n in ("q", "k", "v", "d_o"):
            d[n] = d[n].transpose(1, 2).contiguous().transpose(1, 2)
        d["g"] = d["g"].transpose(1, 2).contiguous().transpose(1, 2)
    elif kind == "odd":             # rows that start one element off 16 bytes
        for n in ("q", "k", "v", "d_o"):
            t = torch.zeros(d[n].numel() + 1, dtype=d[n].dtype, device="cuda")
            t[1:] = d[n].flatten()
            d[n] = t[1:].view(d[n].shape)
    elif kind == "same":            # every stream the same rows (stride 0)
        for n in ("q", "k", "v", "d_o", "g"):
            x[n] = x[n][:1].expand(x[n].shape)
            d[n] = d[n][:1].expand(d[n].shape)
    return d


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["packed", "heads_first", "odd", "same"])
def test_strides_and_alignment(dtype, kind):
    say("glr views", dtype, kind)
    x = make(2, 100, 4, 2, 40, 24, DT[dtype])
    check(x, DT[dtype], 0.4, dev=views(x, kind))


def test_empty():
    x = cuda(make(2, 0, 2, 1, 16, 24, torch.float32))
    o, last = sdm.glr_forward(x["q"], x["k"], x["v"], x["g"], state=x["state"])
    assert o.shape == (2, 0, 2, 24) and torch.equal(last, x["state"])
    r = sdm.glr_backward(x["d_o"], x["q"], x["k"], x["v"], x["g"], state=x["state"], d_last=x["d_last"])
    assert torch.equal(r["dstate"], x["d_last"]) and r["dq"].shape == (2, 0, 1, 16)
    x = cuda(make(0, 5, 2, 1, 16, 24, torch.float32, state=False))
    o, last = sdm.glr_forward(x["q"], x["k"], x["v"], x["g"])
    assert o.shape == (0, 5, 2, 24) and last.shape == (0, 2, 16, 24)


def test_continues_a_state():
    """Two halves, the second from the first one's state, give what the whole row gives (within the bound)."""
    x = make(1, 300, 2, 1, 64, 64, torch.float32)
    d = cuda(x)
    o, last = sdm.glr_forward(d["q"], d["k"], d["v"], d["g"], state=d["state"])
    a, mid = sdm.glr_forward(*(d[n][:, :130] for n in "qkvg"), state=d["state"])
    b, end = sdm.glr_forward(*(d[n][:, 130:] for n in "qkvg"), state=mid)
    _, _, mo, ml = M.glr_forward(*(host(x[n]) for n in "qkvg"), 64 ** -0.5, host(x["state"]))
    near("halves", torch.cat([a, b], 1), o.cpu().numpy().astype(np.float64), mo, 2 * 230, False)
    near("state", end, last.cpu().numpy().astype(np.float64), ml, 2 * 230, False)


def test_bits_stream_and_graph():
    """The same bits on every run, on another stream, with a workspace of the caller's, and in graph replays."""
    x = cuda(make(2, 600, 2, 1, 128, 128, torch.bfloat16))
    args, kw = [x[n] for n in ("q", "k", "v", "g")], dict(scale=0.1, state=x["state"])
    f = lambda **k: sdm.glr_forward(*args, **kw, **k)  # noqa: E731
    b = lambda **k: sdm.glr_backward(x["d_o"], *args, d_last=x["d_last"], **kw, **k)  # noqa: E731
    o, last = f()
    r = b()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2, last2 = f(workspace=torch.empty(sdm.glr_workspace_bytes(2, 600, 2, 1, 128, 128), dtype=torch.uint8, device="cuda"))
        r2 = b(workspace=torch.empty(sdm.glr_workspace_bytes(2, 600, 2, 1, 128, 128, backward=True), dtype=torch.uint8, device="cuda"))
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, o2) and torch.equal(last, last2) and all(torch.equal(r[n], r2[n]) for n in r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, last3 = f()
        r3 = b()
    for rep in range(3):
        say("glr graph replay", rep)
        for t in (o3, last3, *r3.values()):
            t.fill_(7.0)
        f()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o3) and torch.equal(last, last3) and all(torch.equal(r[n], r3[n]) for n in r)


def test_workspace_on_another_stream():
    """A call on a stream of its own, whose workspace the call allocates: what the current stream allocates and fills
    meanwhile does not reach it."""
    x = cuda(make(1, 4096, 4, 4, 128, 128, torch.bfloat16))
    args = [x[n] for n in ("q", "k", "v", "g")]
    o, last = sdm.glr_forward(*args, state=x["state"])
    r = sdm.glr_backward(x["d_o"], *args, state=x["state"], d_last=x["d_last"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    o2, last2 = sdm.glr_forward(*args, state=x["state"], stream=s)
    size = max(sdm.glr_workspace_bytes(1, 4096, 4, 4, 128, 128, backward=b) for b in (False, True))
    for _ in range(4):
        torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255)
    r2 = sdm.glr_backward(x["d_o"], *args, state=x["state"], d_last=x["d_last"], stream=s)
    for _ in range(4):
        torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(last, last2) and all(torch.equal(r[n], r2[n]) for n in r)


# ---------------------------------------------------------------------------------------- one token

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,dk,dv", [(1, 1, 1, 1, 1), (1, 4, 4, 64, 64), (3, 4, 2, 120, 120), (5, 2, 1, 9, 33), (2, 3, 3, 128, 128),
                                          (40, 32, 8, 40, 24), (7, 2, 2, 128, 7)])
def test_step_matches_oracle(dtype, B, H, Hk, dk, dv):
    say("glr step", dtype, B, H, Hk, dk, dv)
    bf = dtype == "bf16"
    x = make(B, 1, H, Hk, dk, dv, DT[dtype])
    h = {k: host(t) for k, t in x.items()}
    wo, wl, mo, ml = M.glr_forward(h["q"], h["k"], h["v"], h["g"], 0.7, h["state"])
    d = cuda(x)
    one = [d[n][:, 0] for n in ("q", "k", "v", "g")]
    new = torch.full_like(d["state"], 9.0)
    state = d["state"].clone()
    o = sdm.glr_step(*one, state, scale=0.7, new_state=new)
    assert torch.equal(state, d["state"])
    near("o", o, wo[:, 0], mo[:, 0], dk + 32, bf)
    near("new state", new, wl, ml, 8, False)
    o2 = sdm.glr_step(*one, state, scale=0.7)          # in place
    assert torch.equal(o, o2) and torch.equal(state, new)
    # Requests in rows of a larger pool, some left out.
    pool = torch.full((2 * B + 3, H, dk, dv), 5.0, device="cuda")
    slots = torch.randperm(2 * B + 3, generator=torch.Generator().manual_seed(1))[:B].int()
    pool[slots.long().cuda()] = d["state"]
    out = torch.full((B, H, dv), 3.0, dtype=DT[dtype], device="cuda")
    left = [b for b in range(B) if b % 3 == 2]
    before = pool.clone()
    for n, b in enumerate(left):
        slots[b] = -1 if n % 2 else 2 * B + 3 + n
    sdm.glr_step(*one, pool, scale=0.7, slots=slots.cuda(), out=out)
    touched = set()
    for b in range(B):
        if b in left:
            assert (out[b] == 0).all()
        else:
            assert torch.equal(out[b], o[b]) and torch.equal(pool[slots[b]], new[b])
            touched.add(int(slots[b]))
    for row in range(2 * B + 3):
        if row not in touched:
            assert torch.equal(pool[row], before[row])


def test_steps_follow_the_forward():
    """A prompt, then token by token: what the forward gives on the whole row."""
    x = make(2, 80, 2, 2, 64, 40, torch.float32)
    d = cuda(x)
    o, last = sdm.glr_forward(d["q"], d["k"], d["v"], d["g"], state=d["state"])
    _, s = sdm.glr_forward(*(d[n][:, :70] for n in "qkvg"), state=d["state"])
    _, _, mo, ml = M.glr_forward(*(host(x[n]) for n in "qkvg"), 64 ** -0.5, host(x["state"]))
    for t in range(70, 80):
        y = sdm.glr_step(*(d[n][:, t] for n in "qkvg"), s)
        near("token %d" % t, y, o[:, t].cpu().numpy().astype(np.float64), mo[:, t], 2 * 200, False)
    near("state", s, last.cpu().numpy().astype(np.float64), ml, 2 * 200, False)


def test_step_state_offsets_past_32_bits():
    """A pool of more than 2^31 elements: the last rows are as good as the first."""
    H, dk, dv = 16, 128, 128
    rows = (1 << 31) // (H * dk * dv) + 3
    pool = torch.empty((rows, H, dk, dv), device="cuda")
    x = cuda(make(2, 1, H, H, dk, dv, torch.bfloat16))
    one = [x[n][:, 0] for n in ("q", "k", "v", "g")]
    pool[rows - 1] = x["state"][0]
    pool[0] = x["state"][1]
    slots = torch.tensor([rows - 1, 0], dtype=torch.int32, device="cuda")
    say("glr step over a pool of", pool.numel(), "elements")
    o = sdm.glr_step(*one, pool, slots=slots)
    new = torch.empty_like(x["state"])
    want = sdm.glr_step(*one, x["state"], new_state=new)
    assert torch.equal(o, want) and torch.equal(pool[rows - 1], new[0]) and torch.equal(pool[0], new[1])


def test_refusals():
    x = cuda(make(2, 8, 4, 2, 16, 24, torch.bfloat16))
    q, k, v, g = (x[n] for n in ("q", "k", "v", "g"))
    with pytest.raises(TypeError):
        sdm.glr_forward(q.half(), k.half(), v.half(), g)
    with pytest.raises(TypeError):
        sdm.glr_forward(q, k, v.float(), g)
    with pytest.raises(TypeError):
        sdm.glr_forward(q, k, v, g.bfloat16())
    with pytest.raises(ValueError):
        sdm.glr_forward(q, k[:, :7], v, g)
    with pytest.raises(ValueError):
        sdm.glr_forward(q.transpose(2, 3), k.transpose(2, 3), v, g)
    with pytest.raises(ValueError):
        sdm.glr_forward(q, k, v, g, state=x["state"][:1])
    with pytest.raises(TypeError):
        sdm.glr_forward(q, k, v, g, state=x["state"].transpose(2, 3).contiguous().transpose(2, 3))
    with pytest.raises(TypeError):
        sdm.glr_forward(q.cpu(), k, v, g)
    with pytest.raises(TypeError):
        sdm.glr_forward(q, k.cpu(), v, g)
    with pytest.raises(sdm.SdmError):   # 4 value heads on 3 key heads
        sdm.glr_forward(q[:, :, :1].expand(-1, -1, 3, -1), k[:, :, :1].expand(-1, -1, 3, -1), v, g)
    with pytest.raises(sdm.SdmError):
        sdm.glr_forward(q, k, v, g, state=x["state"], last=x["state"])
    with pytest.raises(sdm.SdmError):
        sdm.glr_backward(x["d_o"], q, k, v, g, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        sdm.glr_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], x["state"][:, :2].contiguous())
    with pytest.raises(sdm.SdmError):   # fewer states than requests
        sdm.glr_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], x["state"][:1])
    with pytest.raises(TypeError):
        sdm.glr_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], x["state"], slots=torch.zeros(2, dtype=torch.int64, device="cuda"))
