"""The example mixer layer: its operators used together as a layer uses them."""

import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
from oracle import mixer as M  # noqa: E402
from sparse_delta_memory_amd.mixer import Mixer  # noqa: E402


def say(*a):
    print(*a, flush=True)


def layer(dtype):
    m = Mixer(model=96, heads=4, key_heads=2, d=32, hd=48, n=16, W=3, R=2, C=16, rot=16, dtype=dtype, seed=3)
    x = torch.randn((2, 64, 96), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(dtype)
    return m, x


def delta_reads(m, P, T, k_idx, k_val, q_idx, q_val, gate, beta, u):
    """The bank token by token in float64: decay each written slot once, predict, write the delta, read."""
    h = lambda t: t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()  # noqa: E731
    k_idx, k_val, q_idx, q_val, gate, beta, u = (h(t) for t in (k_idx, k_val, q_idx, q_val, gate, beta, u))
    bank, reads = np.zeros((P, m.n * m.n, m.hd)), np.zeros((P, T, m.hd))
    for p in range(P):
        for t in range(T):
            r = p * T + t
            for s in set(k_idx[r]):
                bank[p, s] *= np.exp(gate[r])
            pred = k_val[r] @ bank[p, k_idx[r]]
            dv = beta[r] * (u[r] - pred)
            for s, w in zip(k_idx[r], k_val[r]):
                bank[p, s] += w * dv
            reads[p, t] = q_val[r] @ bank[p, q_idx[r]]
    return reads, bank


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_matches_the_definitions(dtype):
    say("mixer prompt", dtype)
    m, x = layer(dtype)
    P, T = x.shape[:2]
    bank = m.bank(P)
    y, state = m.prompt(x, bank)
    q, k, v, gates, *sparse = m.project(x, torch.arange(T, dtype=torch.int32, device="cuda").repeat(P))
    seq = lambda t: t.unflatten(0, (P, T)).float().cpu().numpy()  # noqa: E731
    o, last, mo, ml = M.glr_forward(seq(q), seq(k), seq(v), seq(gates), m.d ** -0.5)
    got = y[..., :m.heads * m.d].reshape(P, T, m.heads, m.d).cpu().numpy()
    n = (2 * m.d + 96 + 1) * 2.0 ** -23
    bf = (4 * 2.0 ** -16 * mo + 2.0 ** -8 * np.abs(o)) if dtype == torch.bfloat16 else 0.0
    assert (np.abs(got - o) <= n * mo + bf + 1e-30).all()
    assert (np.abs(state.cpu().numpy() - last) <= n * ml + 1e-30).all()
    reads, full = delta_reads(m, P, T, *sparse)
    got = y[..., m.heads * m.d:].cpu().numpy()
    # Softmax weights are at most 1 and sum to 1, beta below 1: reads and rows stay of u's size, with the float32
    # fields' 1e-5 relative error in every step of the substitution.
    top = np.abs(sparse[-1].cpu().numpy()).max()
    assert np.abs(got - reads).max() <= 1e-3 * top and np.abs(bank.view(P, -1, m.hd).cpu().numpy() - full).max() <= 1e-3 * top


def test_tokens_follow_a_prompt():
    """A prompt of three chunks and then single tokens: the fourth chunk's outputs, within rounding."""
    m, x = layer(torch.float32)
    bank, part = m.bank(2), m.bank(2)
    y, state = m.prompt(x, bank)
    _, s = m.prompt(x[:, :48], part)
    for t in range(48, 64):
        z = m.token(x[:, t], part, s, t)
        assert torch.allclose(z, y[:, t], rtol=0, atol=2e-3 * float(y.abs().max())), t
    assert torch.allclose(part, bank, rtol=0, atol=2e-3 * float(bank.abs().max()))
    assert torch.allclose(s, state, rtol=0, atol=2e-3 * float(state.abs().max()))
    with pytest.raises(ValueError):
        m.prompt(x[:, :50], bank)


def test_command():
    r = subprocess.run([sys.executable, "-m", "sparse_delta_memory_amd.mixer"], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "slots written" in r.stdout, r.stderr[-2000:]
