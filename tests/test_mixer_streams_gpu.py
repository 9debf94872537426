"""GPU: calls of the mixer operators on a stream of their own (stream=...): what they allocate is not memory that work still
queued on the current stream uses."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_delta_memory_amd as sdm  # noqa: E402


def say(*a):
    print(*a, flush=True)


def calls():
    """Per operator: a call that takes the stream, and the bytes of its workspace."""
    r = lambda *s: torch.randn(s, generator=torch.Generator().manual_seed(len(s)))  # noqa: E731
    h, w = r(3000, 6, 128).cuda(), r(128).cuda()
    pos, table = torch.arange(3000, device="cuda"), sdm.rope_table(3000, 128)
    a, b, dval = r(9000, 160).cuda(), r(9000, 96).cuda(), r(9000, 8).cuda()
    idx, _ = sdm.slot_topk(a, b, 8)
    q, k, v, d, g = r(2, 900, 4, 64).cuda(), r(2, 900, 4, 64).cuda() / 8, r(2, 900, 4, 96).cuda(), r(2, 900, 4, 96).cuda(), -r(2, 900, 4).abs().cuda()
    pool = r(9, 4, 64, 96).cuda()
    return dict(
        norm_rope=(lambda s: sdm.norm_rope(h, h, w, w, pos, table, stream=s), 0),
        norm_rope_backward=(lambda s: sdm.norm_rope_backward(h, h, h, h, w, w, pos, table, stream=s), 1024 * 2 * 128 * 4),
        slot_topk=(lambda s: sdm.slot_topk(a, b, 8, stream=s), 0),
        slot_topk_backward=(lambda s: sdm.slot_topk_backward(dval, idx, a, b, stream=s), 0),
        glr_forward=(lambda s: sdm.glr_forward(q, k, v, g, stream=s), sdm.glr_workspace_bytes(2, 900, 4, 4, 64, 96)),
        glr_backward=(lambda s: sdm.glr_backward(d, q, k, v, g, stream=s), sdm.glr_workspace_bytes(2, 900, 4, 4, 64, 96, backward=True)),
        glr_step=(lambda s: sdm.glr_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], pool, stream=s), 0))


def tensors(x):
    return [t for t in (x.values() if isinstance(x, dict) else x if isinstance(x, tuple) else [x]) if t is not None]


@pytest.mark.parametrize("name", ["norm_rope", "norm_rope_backward", "slot_topk", "slot_topk_backward", "glr_forward", "glr_backward", "glr_step"])
def test_memory_still_in_use_on_the_current_stream(name):
    """Blocks of the sizes that the call allocates are freed while copies of them wait behind long products on the current
    stream; the call's stream has nothing to wait for."""
    say("mixer streams", name)
    call, workspace = calls()[name]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in tensors(call(side))] + ([workspace] if workspace else [])
    big = torch.randn(8192, 8192, device="cuda").bfloat16()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.full((n,), 123, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.synchronize()
    for _ in range(24):
        big @ big
    copies = [t.clone() for t in blocks]
    del blocks
    call(side)
    torch.cuda.synchronize()
    assert all((t == 123).all() for t in copies)


def test_outputs_and_refusal():
    """Outputs of a call on another stream, used and dropped on the current one, are not given out again before that."""
    x = torch.randn(4096, 8, 128, device="cuda")
    big = torch.randn(8192, 8192, device="cuda").bfloat16()
    want, _ = sdm.norm_rope(x, None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y, _ = sdm.norm_rope(x, None, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(24):
        big @ big
    z = y.clone()
    del y
    for _ in range(4):
        sdm.norm_rope(-x, None, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(z, want)
