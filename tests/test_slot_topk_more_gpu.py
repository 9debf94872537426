"""GPU: layouts of slot_topk's scores beside test_slot_topk_gpu.py's."""

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
@pytest.mark.parametrize("lead", [(3, 20), (1, 7), (7, 1), (2, 3, 5), (1, 1), (0, 4)])
def test_views_of_a_packed_projection(dtype, lead):
    """Parts of rows with any number of leading dimensions: what copies of them give."""
    print("slot views", dtype, lead, flush=True)
    rows = torch.randn((*lead, 200), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    a, b = rows[..., 8:72], rows[..., 73:150]
    idx, val = sdm.slot_topk(a, b, 6)
    want = sdm.slot_topk(a.contiguous(), b.contiguous(), 6)
    assert idx.shape == (*lead, 6) and torch.equal(idx, want[0]) and torch.equal(val, want[1])
    dval = torch.randn((*lead, 6), generator=torch.Generator().manual_seed(2)).cuda()
    for x, y, like in zip(sdm.slot_topk_backward(dval, idx, a, b), sdm.slot_topk_backward(dval, idx, a.contiguous(), b.contiguous()), (a, b)):
        assert x.shape == like.shape and torch.equal(x, y)


def test_rows_without_one_spacing():
    x = torch.randn(4, 6, 64, device="cuda")
    flat = torch.randn(24, 64, device="cuda")
    one = torch.randn(1, 64, device="cuda").expand(24, 64)      # every token the same row
    idx, val = sdm.slot_topk(one, flat, 4)
    want = sdm.slot_topk(one.contiguous(), flat, 4)
    assert torch.equal(idx, want[0]) and torch.equal(val, want[1])
    even = x[:, ::2]                                            # (384, 128): every second row
    assert torch.equal(sdm.slot_topk(even, even, 4)[0], sdm.slot_topk(even.contiguous(), even.contiguous(), 4)[0])
    for bad in (x.transpose(0, 1), x[:, :5], x[:, ::4]):
        with pytest.raises(ValueError):
            sdm.slot_topk(bad, bad, 4)
