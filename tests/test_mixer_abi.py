"""The mixer operators' C ABI on the CPU: struct layouts, host refusals with their status codes (nothing is
launched), workspace sizes and calls that have nothing to do."""

import ctypes
import os
import shutil
import subprocess
import tempfile

import pytest

from sparse_delta_memory_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIP_INCLUDE = "/opt/rocm/include"
STRUCTS = [("sdm_norm_rope_io", _lib.NormRopeIO), ("sdm_norm_rope_grad", _lib.NormRopeGrad), ("sdm_slot_topk_io", _lib.SlotTopkIO),
           ("sdm_slot_topk_grad", _lib.SlotTopkGrad), ("sdm_glr_io", _lib.GlrIO), ("sdm_glr_grad", _lib.GlrGrad),
           ("sdm_glr_step_io", _lib.GlrStepIO)]
FAKE = 0x10000   # never dereferenced: every check below fails before a launch
built = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libsdm_amd.so not built")


@pytest.mark.skipif(shutil.which("gcc") is None or not os.path.exists(os.path.join(HIP_INCLUDE, "hip", "hip_runtime_api.h")),
                    reason="gcc or the HIP headers are missing")
def test_ctypes_mirrors_match_c_layout():
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "sdm.h"', "int main(void) {"]
    for cname, cls in STRUCTS:
        lines.append('    printf("%s sizeof %%zu\\n", sizeof(%s));' % (cname, cname))
        for fname, _ in cls._fields_:
            lines.append('    printf("%s %s %%zu\\n", offsetof(%s, %s));' % (cname, fname, cname, fname))
    lines += ["    return 0;", "}"]
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "layout.c"), os.path.join(d, "layout")
        with open(src, "w") as f:
            f.write("\n".join(lines) + "\n")
        subprocess.run(["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", HIP_INCLUDE, src, "-o", exe],
                       check=True, capture_output=True)
        out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")
    c = {tuple(line.split()[:2]): int(line.split()[2]) for line in out if line}
    for cname, cls in STRUCTS:
        assert c[(cname, "sizeof")] == ctypes.sizeof(cls), cname
        for fname, _ in cls._fields_:
            assert c[(cname, fname)] == getattr(cls, fname).offset, (cname, fname)


def fill(cls, base, kw):
    s = cls()
    for k, v in {**base, **kw}.items():
        setattr(s, k, v)
    return s


NR = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, wq=FAKE, wk=FAKE, pos=FAKE, table=FAKE, table_rows=4, N=8, Hq=2, Hk=1, D=64, rot=64,
          pos_bytes=4, eps=1e-6)


@built
@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), _lib.SDM_ESHAPE), (dict(Hq=0, Hk=0), _lib.SDM_ESHAPE), (dict(Hq=-1), _lib.SDM_ESHAPE), (dict(D=0), _lib.SDM_ESHAPE),
    (dict(D=513), _lib.SDM_ESHAPE), (dict(rot=3), _lib.SDM_ESHAPE), (dict(rot=66), _lib.SDM_ESHAPE), (dict(N=1 << 25), _lib.SDM_ESHAPE),
    (dict(rot=-2), _lib.SDM_ESHAPE), (dict(interleaved=2), _lib.SDM_EINVAL), (dict(dtype=2), _lib.SDM_EINVAL), (dict(w_dtype=-1), _lib.SDM_EINVAL),
    (dict(eps=-1.0), _lib.SDM_EINVAL), (dict(eps=float("nan")), _lib.SDM_EINVAL), (dict(eps=float("inf")), _lib.SDM_EINVAL),
    (dict(pos_bytes=2), _lib.SDM_EINVAL), (dict(table_rows=0), _lib.SDM_EINVAL), (dict(q=None), _lib.SDM_EINVAL), (dict(k_out=None), _lib.SDM_EINVAL),
    (dict(pos=None), _lib.SDM_EINVAL), (dict(table=None), _lib.SDM_EINVAL), (dict(q=FAKE + 2), _lib.SDM_EALIGN), (dict(wq=FAKE + 1), _lib.SDM_EALIGN),
    (dict(table=FAKE + 2), _lib.SDM_EALIGN), (dict(pos=FAKE + 4, pos_bytes=8), _lib.SDM_EALIGN),
])
def test_norm_rope_refusals(kw, status):
    lib = _lib.load()
    io = fill(_lib.NormRopeIO, NR, kw)
    g = fill(_lib.NormRopeGrad, dict(dq=FAKE, dk=FAKE, workspace=FAKE, workspace_bytes=1 << 40), {})
    assert lib.sdm_norm_rope(ctypes.byref(io), None) == status and len(lib.sdm_last_error()) > 0
    assert lib.sdm_norm_rope_backward(ctypes.byref(io), ctypes.byref(g), None) == status


@built
def test_norm_rope_backward_refusals_and_workspace():
    lib = _lib.load()
    io = fill(_lib.NormRopeIO, NR, {})
    assert lib.sdm_norm_rope_workspace(ctypes.byref(io)) == 8 * 3 * 2 * 64 * 4          # a row per head at most
    big = fill(_lib.NormRopeIO, NR, dict(N=100000))
    assert lib.sdm_norm_rope_workspace(ctypes.byref(big)) == 1024 * 2 * 64 * 4
    assert lib.sdm_norm_rope_workspace(None) == 0
    ok = dict(dq=FAKE, dk=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    for kw, status in ((dict(dq=None), _lib.SDM_EINVAL), (dict(dk=None), _lib.SDM_EINVAL), (dict(dq=FAKE + 2), _lib.SDM_EALIGN),
                       (dict(workspace=None), _lib.SDM_EWORKSPACE), (dict(workspace_bytes=16), _lib.SDM_EWORKSPACE),
                       (dict(workspace=FAKE + 8), _lib.SDM_EALIGN), (dict(dwq=FAKE + 2), _lib.SDM_EALIGN)):
        g = fill(_lib.NormRopeGrad, ok, kw)
        assert lib.sdm_norm_rope_backward(ctypes.byref(io), ctypes.byref(g), None) == status, kw
    assert lib.sdm_norm_rope_backward(ctypes.byref(io), None, None) == _lib.SDM_EINVAL
    assert lib.sdm_norm_rope(None, None) == _lib.SDM_EINVAL
    assert lib.sdm_norm_rope(ctypes.byref(fill(_lib.NormRopeIO, NR, dict(N=0))), None) == _lib.SDM_OK


ST = dict(a=FAKE, b=FAKE, a_row=64, b_row=64, idx=FAKE, val=FAKE, N=4, n1=64, n2=64, K=8, idx_bytes=4, scale=1.0, P=1)


@built
@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), _lib.SDM_ESHAPE), (dict(n1=0), _lib.SDM_ESHAPE), (dict(n2=4097), _lib.SDM_ESHAPE), (dict(K=0), _lib.SDM_ESHAPE),
    (dict(K=65), _lib.SDM_ESHAPE), (dict(n1=2, n2=3, K=7), _lib.SDM_ESHAPE), (dict(dtype=7), _lib.SDM_EINVAL), (dict(idx_bytes=2), _lib.SDM_EINVAL),
    (dict(scale=0.0), _lib.SDM_EINVAL), (dict(scale=float("inf")), _lib.SDM_EINVAL), (dict(scale=float("nan")), _lib.SDM_EINVAL),
    (dict(chunk_rows=-1), _lib.SDM_EINVAL), (dict(chunk_rows=8, P=0), _lib.SDM_EINVAL), (dict(chunk_rows=8, stream_offset=-1), _lib.SDM_EINVAL),
    (dict(chunk_rows=8, P=1 << 20, stream_offset=4096), _lib.SDM_EINVAL), (dict(a=None), _lib.SDM_EINVAL), (dict(idx=None), _lib.SDM_EINVAL),
    (dict(a=FAKE + 2), _lib.SDM_EALIGN), (dict(idx=FAKE + 4, idx_bytes=8), _lib.SDM_EALIGN),
])
def test_slot_refusals(kw, status):
    lib = _lib.load()
    io = fill(_lib.SlotTopkIO, ST, kw)
    g = fill(_lib.SlotTopkGrad, dict(dval=FAKE, da=FAKE, db=FAKE, da_row=64, db_row=64), {})
    assert lib.sdm_slot_topk(ctypes.byref(io), None) == status and len(lib.sdm_last_error()) > 0
    assert lib.sdm_slot_topk_backward(ctypes.byref(io), ctypes.byref(g), None) == status


@built
def test_slot_more_refusals():
    lib = _lib.load()
    for kw, status in ((dict(val=None), _lib.SDM_EINVAL), (dict(val_dtype=3), _lib.SDM_EINVAL), (dict(val=FAKE + 2), _lib.SDM_EALIGN)):
        assert lib.sdm_slot_topk(ctypes.byref(fill(_lib.SlotTopkIO, ST, kw)), None) == status
    io = fill(_lib.SlotTopkIO, ST, {})
    for kw, status in ((dict(dval=None), _lib.SDM_EINVAL), (dict(da=FAKE + 1), _lib.SDM_EALIGN), (dict(da=None, db=None), _lib.SDM_OK)):
        g = fill(_lib.SlotTopkGrad, dict(dval=FAKE, da=FAKE, db=FAKE, da_row=64, db_row=64), kw)
        assert lib.sdm_slot_topk_backward(ctypes.byref(io), ctypes.byref(g), None) == status
    assert lib.sdm_slot_topk_backward(ctypes.byref(io), None, None) == _lib.SDM_EINVAL
    assert lib.sdm_slot_topk(None, None) == _lib.SDM_EINVAL
    assert lib.sdm_slot_topk(ctypes.byref(fill(_lib.SlotTopkIO, ST, dict(N=0))), None) == _lib.SDM_OK


GL = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, o=FAKE, B=2, T=8, H=4, Hk=2, dk=16, dv=24, scale=1.0, workspace=FAKE, workspace_bytes=1 << 40)
GG = dict(d_o=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE)


@built
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), _lib.SDM_ESHAPE), (dict(T=-1), _lib.SDM_ESHAPE), (dict(H=0), _lib.SDM_ESHAPE), (dict(H=3), _lib.SDM_ESHAPE), (dict(Hk=0), _lib.SDM_ESHAPE),
    (dict(dk=0), _lib.SDM_ESHAPE), (dict(dk=129), _lib.SDM_ESHAPE), (dict(dv=129), _lib.SDM_ESHAPE), (dict(B=1 << 19, H=4), _lib.SDM_ESHAPE),
    (dict(B=1 << 16, T=1 << 16), _lib.SDM_ESHAPE), (dict(B=1, H=1, Hk=1, T=(1 << 30) + 1), _lib.SDM_ESHAPE), (dict(dtype=5), _lib.SDM_EINVAL), (dict(scale=float("nan")), _lib.SDM_EINVAL),
    (dict(q=None), _lib.SDM_EINVAL), (dict(g=None), _lib.SDM_EINVAL), (dict(v=FAKE + 2), _lib.SDM_EALIGN), (dict(state=FAKE + 4), _lib.SDM_EALIGN),
    (dict(lens=FAKE + 2), _lib.SDM_EALIGN), (dict(workspace=FAKE + 16), _lib.SDM_EALIGN),
    (dict(B=1, T=4096, workspace=None), _lib.SDM_EWORKSPACE), (dict(B=1, T=4096, workspace_bytes=256), _lib.SDM_EWORKSPACE),
])
def test_glr_refusals(kw, status):
    lib = _lib.load()
    io, g = fill(_lib.GlrIO, GL, kw), fill(_lib.GlrGrad, GG, {})
    assert lib.sdm_glr_forward(ctypes.byref(io), None) == status and len(lib.sdm_last_error()) > 0
    assert lib.sdm_glr_backward(ctypes.byref(io), ctypes.byref(g), None) == status


@built
def test_glr_more_refusals():
    lib = _lib.load()
    for kw, status in ((dict(o=None), _lib.SDM_EINVAL), (dict(o=FAKE + 1), _lib.SDM_EALIGN), (dict(last=FAKE + 4), _lib.SDM_EALIGN),
                       (dict(last=FAKE, state=FAKE), _lib.SDM_EINVAL)):
        assert lib.sdm_glr_forward(ctypes.byref(fill(_lib.GlrIO, GL, kw)), None) == status
    io = fill(_lib.GlrIO, GL, {})
    for kw, status in ((dict(d_o=None), _lib.SDM_EINVAL), (dict(dq=None), _lib.SDM_EINVAL), (dict(dg=None), _lib.SDM_EINVAL),
                       (dict(d_last=FAKE, d_state=FAKE), _lib.SDM_EINVAL), (dict(dv=FAKE + 4), _lib.SDM_EALIGN), (dict(d_last=FAKE + 4), _lib.SDM_EALIGN), (dict(d_o=FAKE + 1), _lib.SDM_EALIGN)):
        assert lib.sdm_glr_backward(ctypes.byref(io), ctypes.byref(fill(_lib.GlrGrad, GG, kw)), None) == status
    assert lib.sdm_glr_backward(ctypes.byref(io), None, None) == _lib.SDM_EINVAL
    assert lib.sdm_glr_forward(None, None) == _lib.SDM_EINVAL
    empty = fill(_lib.GlrIO, GL, dict(B=0))
    assert lib.sdm_glr_forward(ctypes.byref(empty), None) == _lib.SDM_OK
    assert lib.sdm_glr_backward(ctypes.byref(empty), ctypes.byref(fill(_lib.GlrGrad, GG, {})), None) == _lib.SDM_OK
    assert lib.sdm_glr_workspace(None, 0) == 0
    short = fill(_lib.GlrIO, GL, {})
    assert lib.sdm_glr_workspace(ctypes.byref(short), 0) == 0 and lib.sdm_glr_workspace(ctypes.byref(short), 1) > 0


GS = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, o=FAKE, state=FAKE, new_state=FAKE, rows=2, B=2, H=4, Hk=2, dk=16, dv=24, scale=1.0)


@built
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), _lib.SDM_ESHAPE), (dict(H=3), _lib.SDM_ESHAPE), (dict(dk=129), _lib.SDM_ESHAPE), (dict(dtype=2), _lib.SDM_EINVAL),
    (dict(rows=1), _lib.SDM_EINVAL), (dict(rows=-1, slots=FAKE), _lib.SDM_EINVAL), (dict(state=None), _lib.SDM_EINVAL), (dict(o=None), _lib.SDM_EINVAL),
    (dict(g=FAKE + 2), _lib.SDM_EALIGN), (dict(new_state=FAKE + 8), _lib.SDM_EALIGN), (dict(slots=FAKE + 2), _lib.SDM_EALIGN),
    (dict(B=1 << 23, rows=1 << 23), _lib.SDM_ESHAPE), (dict(scale=float("inf")), _lib.SDM_EINVAL), (dict(B=0), _lib.SDM_OK),
])
def test_glr_step_refusals(kw, status):
    assert _lib.load().sdm_glr_step(ctypes.byref(fill(_lib.GlrStepIO, GS, kw)), None) == status


@built
def test_norm_rope_heads_of_one_grid():
    """524288 tokens of 72 heads are taken; what no grid of a wave per head holds is refused."""
    lib = _lib.load()
    ok = fill(_lib.NormRopeIO, NR, dict(N=1 << 19, Hq=64, Hk=8))
    assert lib.sdm_norm_rope_workspace(ctypes.byref(ok)) == 1024 * 2 * 64 * 4
    most = fill(_lib.NormRopeIO, NR, dict(N=(1 << 26) - 4, Hq=1, Hk=0))
    assert lib.sdm_norm_rope_workspace(ctypes.byref(most)) == 1024 * 2 * 64 * 4
    for kw in (dict(N=(1 << 26) - 3, Hq=1, Hk=0), dict(N=1 << 20, Hq=64)):
        io = fill(_lib.NormRopeIO, NR, kw)
        assert lib.sdm_norm_rope_workspace(ctypes.byref(io)) == 0
        assert lib.sdm_norm_rope(ctypes.byref(io), None) == _lib.SDM_ESHAPE


@built
@pytest.mark.parametrize("kw", [
    dict(P=(1 << 24) + 1, stream_offset=1 << 40), dict(P=(1 << 24) + 1, stream_offset=1 << 40, idx_bytes=8),   # products of 2^64, 2^63
    dict(P=(1 << 23) + 1, stream_offset=1 << 40, idx_bytes=8), dict(P=(1 << 31) - 1, stream_offset=1 << 40), dict(P=2, stream_offset=(1 << 31) - 4095),
])
def test_slot_ids_past_their_type(kw):
    lib = _lib.load()
    io = fill(_lib.SlotTopkIO, {**ST, "chunk_rows": 8}, kw)
    g = fill(_lib.SlotTopkGrad, dict(dval=FAKE, da=FAKE, db=FAKE, da_row=64, db_row=64), {})
    assert lib.sdm_slot_topk(ctypes.byref(io), None) == _lib.SDM_EINVAL
    assert lib.sdm_slot_topk_backward(ctypes.byref(io), ctypes.byref(g), None) == _lib.SDM_EINVAL


@built
def test_slot_ids_that_fit():
    lib = _lib.load()
    for kw in (dict(P=2, stream_offset=(1 << 31) - 4096), dict(P=(1 << 23) - 1, stream_offset=1 << 40, idx_bytes=8), dict(P=1 << 30, stream_offset=0)):
        io = fill(_lib.SlotTopkIO, {**ST, "chunk_rows": 8, "N": 0}, kw)
        assert lib.sdm_slot_topk(ctypes.byref(io), None) == _lib.SDM_OK


@built
def test_states_of_odd_widths_are_aligned_by_element():
    """Rows of a pool whose states are no whole 16-byte pieces; B = 0 and missing outputs keep everything on the host."""
    lib = _lib.load()
    for dv, status in ((24, _lib.SDM_EALIGN), (25, _lib.SDM_EINVAL)):      # EINVAL: o is missing, found after the alignment
        io = fill(_lib.GlrIO, GL, dict(dk=15, dv=dv, state=FAKE + 4, o=None))
        assert lib.sdm_glr_forward(ctypes.byref(io), None) == status
    odd = fill(_lib.GlrIO, GL, dict(dk=15, dv=25, state=FAKE + 2))
    assert lib.sdm_glr_forward(ctypes.byref(odd), None) == _lib.SDM_EALIGN
    for kw, status in ((dict(dk=15, dv=25, state=FAKE + 2), _lib.SDM_EALIGN), (dict(dk=16, dv=25, new_state=FAKE + 4), _lib.SDM_EALIGN)):
        assert lib.sdm_glr_step(ctypes.byref(fill(_lib.GlrStepIO, GS, kw)), None) == status
