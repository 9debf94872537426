"""GPU: the gated delta rule where it can go wrong beyond the sizes: values that are not finite, strides, packed sequences, other
streams, captured graphs, the same bits again; and the digits that its results keep."""

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
from test_gdr_gpu import DT, INF, NAN, args, backward, cuda, forward, host, make, near, say  # noqa: E402


def run(x, scale=0.3):
    d = cuda(x)
    o, last = sdm.gdr_forward(*args(d), scale=scale, state=d["state"], lens=d["lens"])
    return dict(o=o, last=last, **sdm.gdr_backward(d["d_o"], *args(d), scale=scale, state=d["state"], d_last=d["d_last"], lens=d["lens"]))


def close(name, got, want):
    """Of the same inputs by another path (token by token): float32 roundings, and a bfloat16 rounding either way."""
    got, want = got.float(), want.float()
    assert torch.isfinite(got).all(), "%s: %d values not finite" % (name, int((~torch.isfinite(got)).sum()))
    top = float(want.abs().max())
    tol = 2.0 ** -7 * want.abs() + 1e-4 * top
    assert ((got - want).abs() <= tol).all(), "%s: off by %.3g of %.3g" % (name, float((got - want).abs().max()), top)


# one chunk and a bit, and rows cut into segments
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,t0,reset", [(90, 20, 45), (90, 63, 64), (800, 200, 230), (800, 200, 700)])
@pytest.mark.parametrize("value", [INF, NAN])
def test_what_is_not_finite_reaches_what_it_is_part_of(dtype, T, t0, reset, value):
    say("gdr not finite", dtype, T, t0, reset, value)
    x = make(1, T, 2, 2, 32, 40, dtype)
    x["g"][0, reset] = -INF
    clean = run(x)
    for name in ("v", "k", "q"):
        y = {n: None if t is None else t.clone() for n, t in x.items()}
        y[name][0, t0, 1, 3] = value
        r = run(y)
        for out in ("o", "dq", "dk", "dv", "dbeta"):      # the other head is not touched at all
            assert torch.equal(r[out][:, :, 0], clean[out][:, :, 0]), (name, out)
        o = r["o"][0, :, 1]
        close(name + " o before", o[:t0], clean["o"][0, :t0, 1])
        close(name + " o past the reset", o[reset:], clean["o"][0, reset:, 1])
        close(name + " last", r["last"][0, 1], clean["last"][0, 1])
        if name == "q":
            close("o after", o[t0 + 1:], clean["o"][0, t0 + 1:, 1])
            assert not torch.isfinite(o[t0]).any()
            close("dq", r["dq"][0, :, 1], clean["dq"][0, :, 1])
            at = slice(t0 + 1, None)
        else:
            assert not torch.isfinite(o[t0:reset]).all(-1).any() if name == "k" else not torch.isfinite(o[t0:reset, 3]).any()
            at = slice(reset, None)
            close(name + " dq before", r["dq"][0, :t0, 1], clean["dq"][0, :t0, 1])
        if name == "v":
            close("dv", r["dv"][0, :, 1], clean["dv"][0, :, 1])
            close("dk before", r["dk"][0, :t0, 1], clean["dk"][0, :t0, 1])
        for out in ("dq", "dk", "dv", "dbeta", "dg"):
            close(name + " " + out + " past it", r[out][0, at, 1], clean[out][0, at, 1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [50, 700])
def test_a_reset_clears_a_state_that_is_not_finite(dtype, T):
    say("gdr reset", dtype, T)
    x = make(1, T, 2, 1, 32, 40, dtype)
    for at in (0, 20):
        x["g"][0, at] = -INF
        clean = run(x)
        y = dict(x, state=torch.full_like(x["state"], NAN))
        r = run(y)
        for name in ("o", "dq", "dk", "dv", "dbeta", "dg"):
            close(name, r[name][0, at:], clean[name][0, at:])
        close("last", r["last"], clean["last"])
        x["g"][0, at] = -0.1
    step = {n: t[:, 0] if n in ("q", "k", "v", "g", "beta") else t for n, t in cuda(x).items()}
    step["g"] = torch.full_like(step["g"], -INF)
    bad = torch.full_like(step["state"], NAN)
    o = sdm.gdr_step(*args(step), bad)
    assert torch.isfinite(o).all() and torch.isfinite(bad).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 8, 1])
def test_views_of_a_projection(dtype, pad):
    """q, k, v as parts of one row, outputs into a wider buffer, gates and beta with strides; pad 1: nothing starts on 16 bytes."""
    say("gdr views", dtype, pad)
    B, T, H, Hk, dk, dv = 2, 130, 4, 2, 32, 48
    x = make(B, T, H, Hk, dk, dv, dtype)
    d = cuda(x)
    plain = run(x)
    width = pad + 2 * Hk * dk + H * dv
    rows = torch.full((B, T, width), NAN, device="cuda").to(DT[dtype])
    rows[..., pad:] = torch.cat([d["q"].flatten(2), d["k"].flatten(2), d["v"].flatten(2)], -1)
    q, k, v = rows[..., pad:].split([Hk * dk, Hk * dk, H * dv], -1)
    q, k, v = q.unflatten(-1, (Hk, dk)), k.unflatten(-1, (Hk, dk)), v.unflatten(-1, (H, dv))
    gb = torch.stack([d["g"], d["beta"]], -1)
    g, beta = gb[..., 0], gb[..., 1]
    out = torch.full((B, T, H, dv + 3), 7.0, device="cuda").to(DT[dtype])
    o, last = sdm.gdr_forward(q, k, v, g, beta, scale=0.3, state=d["state"], out=out[..., :dv])
    assert torch.equal(o, plain["o"]) and torch.equal(last, plain["last"]) and (out[..., dv:] == 7.0).all()
    r = sdm.gdr_backward(out[..., :dv].copy_(d["d_o"]), q, k, v, g, beta, scale=0.3, state=d["state"], d_last=d["d_last"])
    for name, t in r.items():
        assert torch.equal(t, plain[name]), name
    wide = torch.full((B, H, dv + 5), 7.0, device="cuda").to(DT[dtype])
    a = sdm.gdr_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], d["state"].clone(), out=wide[..., :dv])
    b = sdm.gdr_step(*[t[:, 0].contiguous() for t in (q, k, v, g, beta)], d["state"].clone())
    assert torch.equal(a, b) and (wide[..., dv:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_sequences(dtype):
    """Sequences behind each other in one row, each started by a reset: as each by itself."""
    say("gdr packed", dtype)
    lens = [1, 63, 64, 65, 2, 200, 105]
    x = make(1, sum(lens), 2, 1, 48, 64, dtype, state=False)
    at = np.cumsum([0] + lens)
    for a in at[:-1]:
        x["g"][0, a] = -INF
    r = run(x)
    for a, b in zip(at[:-1], at[1:]):
        y = {n: None if t is None else t[:, a:b].contiguous() for n, t in x.items()}
        one = run(y)
        for name in ("o", "dq", "dk", "dv", "dbeta", "dg"):
            close("%s %d" % (name, a), r[name][:, a:b], one[name])


def test_the_same_bits_and_a_given_workspace():
    x = make(2, 900, 3, 3, 64, 96, "bf16")
    a, b = run(x), run(x)
    assert all(torch.equal(a[n], b[n]) for n in a)
    d = cuda(x)
    ws = torch.full((sdm.gdr_workspace_bytes(2, 900, 3, 3, 64, 96, torch.bfloat16, backward=True),), 255, dtype=torch.uint8, device="cuda")
    r = sdm.gdr_backward(d["d_o"], *args(d), scale=0.3, state=d["state"], d_last=d["d_last"], workspace=ws)
    assert all(torch.equal(r[n], a[n]) for n in r)
    o, last = sdm.gdr_forward(*args(d), scale=0.3, state=d["state"], workspace=ws)
    assert torch.equal(o, a["o"]) and torch.equal(last, a["last"])
    with pytest.raises(sdm.SdmError):
        sdm.gdr_backward(d["d_o"], *args(d), state=d["state"], workspace=ws[:256])


def test_results_keep_24_bits():
    """float32 results of bfloat16 inputs: the last state and the gates' and betas' gradients. An evaluation in float32 token by
    token is off by some 2^-24 of a state's norm in quadrature; products of 16-bit parts would be off by 2^-17 and more."""
    x = make(1, 256, 2, 2, 128, 128, "bf16", gate=4.0)
    h = {n: host(t) for n, t in x.items()}
    r = run(x)
    _, wl, _, _ = M.gdr_forward(*args(h), 0.3, h["state"])
    w, _ = M.gdr_backward(h["d_o"], *args(h), 0.3, h["state"], h["d_last"])
    for name, got, want in (("last", r["last"], wl), ("dstate", r["dstate"], w["dstate"]), ("dbeta", r["dbeta"], w["dbeta"]), ("dg", r["dg"], w["dg"])):
        e = np.sqrt(((got.cpu().numpy() - want) ** 2).mean() / (want ** 2).mean())
        assert e < 2.0 ** -19, (name, e)


def test_on_another_stream():
    x = make(2, 700, 2, 2, 64, 64, "bf16")
    d, want = cuda(x), run(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, last = sdm.gdr_forward(*args(d), scale=0.3, state=d["state"], stream=side)
    r = sdm.gdr_backward(d["d_o"], *args(d), scale=0.3, state=d["state"], d_last=d["d_last"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want["o"]) and torch.equal(last, want["last"]) and all(torch.equal(r[n], want[n]) for n in r)


def test_captured_and_replayed():
    """Forward, backward, a token and both norms in one graph, replayed on new inputs with eager work in between."""
    say("gdr graph")
    x = cuda(make(1, 700, 2, 1, 64, 64, "bf16"))
    z, w = torch.randn((700, 2, 64), device="cuda").bfloat16(), torch.randn(64, device="cuda")

    def all_of(x):
        o, last = sdm.gdr_forward(*args(x), state=x["state"])
        r = sdm.gdr_backward(x["d_o"], *args(x), state=x["state"], d_last=x["d_last"])
        y = sdm.gate_norm(o[0], z, w)
        e = sdm.gate_norm_backward(x["d_o"][0], o[0], z, w)
        h, n = sdm.residual_norm(y.flatten(1), z.flatten(1), scale=torch.cat([w, w]))
        f = sdm.residual_norm_backward(h, n, h, z.flatten(1), scale=torch.cat([w, w]))
        s = last.clone()
        t = sdm.gdr_step(*[a[:, 0] for a in args(x)], s)
        return [o, last, *r.values(), y, e["dx"], e["dz"], e["dw"], h, n, f["dx"], f["dy"], f["dscale"], s, t]

    for _ in range(2):
        all_of(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_of(x)
    for seed in range(4):
        new = cuda(make(1, 700, 2, 1, 64, 64, "bf16", seed=10 + seed))
        for n, t in x.items():
            if t is not None:
                t.copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, all_of(new))):
            assert torch.equal(a, b), (seed, i)
