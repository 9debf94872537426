"""GPU: the example mixer layer gives its operators rows on which their wide loads work."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from sparse_delta_memory_amd import mixer  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kw", [dict(), dict(heads=3, key_heads=1, n=20, hd=33)])
def test_every_part_of_the_projection_is_aligned(monkeypatch, dtype, kw):
    m = mixer.Mixer(dtype=dtype, C=8, **kw)
    seen = []

    def spy(f):
        def g(*args, **kwargs):
            # The gates are read one by one: the recurrence's fourth argument.
            rows = args[:3] if f.__name__.startswith("glr") else args
            seen.extend(t for t in rows if isinstance(t, torch.Tensor) and t.dtype == dtype and t.dim() > 1)
            return f(*args, **kwargs)
        return g

    for name in ("norm_rope", "slot_topk", "glr_forward", "glr_step"):
        monkeypatch.setattr(mixer, name, spy(getattr(mixer, name)))
    x = torch.randn(2, 17, m.w.shape[0], device="cuda").to(dtype)
    bank = m.bank(2)
    y, state = m.prompt(x[:, :16], bank)
    m.token(x[:, 16], bank, state, 16)
    unit = 16 // dtype.itemsize
    assert len(seen) >= 2 * (2 + 4 + 3)      # heads, scores of the writes and reads, q k v (and a float32 table)
    for t in seen:
        assert t.data_ptr() % 16 == 0 and all(s % unit == 0 for s, n in zip(t.stride()[:-1], t.shape) if n > 1), (t.shape, t.stride())


def test_rows_of_another_count_than_the_shape():
    """slot_topk with a Phase-1 shape takes that shape's tokens."""
    import sparse_delta_memory_amd as sdm
    shape = sdm.make_shape(6, 8, 4, 4, P=3, key_bits=8, stream_offset=256)
    a = torch.randn(48, 16, device="cuda")
    idx, _ = sdm.slot_topk(a, a, 4, shape=shape)
    for rows in (a[:40], a[:40].view(5, 8, 16)):
        with pytest.raises(ValueError):
            sdm.slot_topk(rows, rows, 4, shape=shape)
    with pytest.raises(ValueError):
        sdm.slot_topk_backward(torch.zeros(40, 4, device="cuda"), idx[:40].contiguous(), a[:40], a[:40], shape=shape)


def test_positions_past_the_table():
    m = mixer.Mixer(C=8, positions=32)
    x = torch.randn(1, 40, m.w.shape[0], device="cuda").bfloat16()
    bank = m.bank(1)
    _, state = m.prompt(x[:, :32], bank)
    for bad in (lambda: m.prompt(x, bank), lambda: m.prompt(x[:, :8], bank, start=25), lambda: m.token(x[:, 0], bank, state, 32),
                lambda: m.token(x[:, 0], bank, state, -1)):
        with pytest.raises(ValueError):
            bad()
