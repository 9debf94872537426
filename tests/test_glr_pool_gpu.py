"""GPU: states of the recurrence as rows of a pool, in odd widths: any row may be where a state begins."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_delta_memory_amd as sdm  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(5, 7), (9, 33), (1, 1), (66, 127)])
def test_rows_of_a_pool(dtype, dk, dv):
    print("glr pool rows", dtype, dk, dv, flush=True)
    H, T = 1, 90
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen).cuda()  # noqa: E731
    q, k, v, d = r(1, T, H, dk).to(dtype), r(1, T, H, dk).to(dtype), r(1, T, H, dv).to(dtype), r(1, T, H, dv).to(dtype)
    g, pool = -r(1, T, H).abs(), r(7, H, dk, dv)
    for row in (1, 2, 3):
        s, e = pool[row:row + 1], r(7, H, dk, dv)[row:row + 1]
        last = torch.empty_like(pool)[row:row + 1]
        o, _ = sdm.glr_forward(q, k, v, g, state=s, last=last)
        want, wlast = sdm.glr_forward(q, k, v, g, state=s.clone())
        assert torch.equal(o, want) and torch.equal(last, wlast)
        a, b = sdm.glr_backward(d, q, k, v, g, state=s, d_last=e), sdm.glr_backward(d, q, k, v, g, state=s.clone(), d_last=e.clone())
        assert all(torch.equal(a[n], b[n]) for n in a)
        one = [t[:, 0] for t in (q, k, v, g)]
        keep, before = s.clone(), pool.clone()
        y, z = sdm.glr_step(*one, s), sdm.glr_step(*one, keep)
        assert torch.equal(y, z) and torch.equal(s, keep)
        rest = [n for n in range(7) if n != row]
        assert torch.equal(pool[rest], before[rest])
