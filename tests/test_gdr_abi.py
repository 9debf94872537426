"""The C ABI of the gated delta rule and the block's norms on the CPU: struct layouts, host refusals with their status codes (nothing
is launched), workspace sizes and calls that have nothing to do."""

import ctypes
import os

import pytest

import test_mixer_abi as A
from sparse_delta_memory_amd import _lib

FAKE = 0x10000   # never dereferenced: every check below fails before a launch
built = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libsdm_amd.so not built")
E = {n: getattr(_lib, "SDM_E" + n) for n in ("INVAL", "SHAPE", "ALIGN", "WORKSPACE")}
fill, by = A.fill, ctypes.byref


def test_ctypes_mirrors_match_c_layout(monkeypatch):
    monkeypatch.setattr(A, "STRUCTS", [
        ("sdm_gdr_io", _lib.GdrIO), ("sdm_gdr_grad", _lib.GdrGrad), ("sdm_gdr_step_io", _lib.GdrStepIO), ("sdm_gate_norm_io", _lib.GateNormIO),
        ("sdm_gate_norm_grad", _lib.GateNormGrad), ("sdm_residual_norm_io", _lib.ResidualNormIO), ("sdm_residual_norm_grad", _lib.ResidualNormGrad)])
    A.test_ctypes_mirrors_match_c_layout()


GD = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, o=FAKE, B=2, T=8, H=4, Hk=2, dk=16, dv=24, scale=1.0, workspace=FAKE, workspace_bytes=1 << 40)
GG = dict(d_o=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE, dbeta=FAKE)


@built
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(H=0), "SHAPE"), (dict(H=3), "SHAPE"), (dict(Hk=0), "SHAPE"), (dict(dk=0), "SHAPE"),
    (dict(dk=129), "SHAPE"), (dict(dv=129), "SHAPE"), (dict(B=1 << 19, H=4), "SHAPE"), (dict(B=1 << 16, T=1 << 16), "SHAPE"),
    (dict(B=1, H=1, Hk=1, T=(1 << 30) + 1), "SHAPE"), (dict(dtype=5), "INVAL"), (dict(scale=float("nan")), "INVAL"), (dict(q=None), "INVAL"),
    (dict(g=None), "INVAL"), (dict(beta=None), "INVAL"), (dict(v=FAKE + 2), "ALIGN"), (dict(state=FAKE + 4), "ALIGN"), (dict(beta=FAKE + 2), "ALIGN"),
    (dict(lens=FAKE + 2), "ALIGN"), (dict(workspace=FAKE + 16), "ALIGN"), (dict(workspace=None), "WORKSPACE"), (dict(workspace_bytes=256), "WORKSPACE"),
])
def test_gdr_refusals(kw, status):
    lib = _lib.load()
    io, g = fill(_lib.GdrIO, GD, kw), fill(_lib.GdrGrad, GG, {})
    assert lib.sdm_gdr_forward(by(io), None) == E[status] and len(lib.sdm_last_error()) > 0
    assert lib.sdm_gdr_backward(by(io), by(g), None) == E[status]


@built
def test_gdr_more_refusals_and_workspace():
    lib = _lib.load()
    for kw, status in ((dict(o=None), "INVAL"), (dict(o=FAKE + 1), "ALIGN"), (dict(last=FAKE + 4), "ALIGN"), (dict(last=FAKE, state=FAKE), "INVAL")):
        assert lib.sdm_gdr_forward(by(fill(_lib.GdrIO, GD, kw)), None) == E[status], kw
    io = fill(_lib.GdrIO, GD, {})
    for kw, status in ((dict(d_o=None), "INVAL"), (dict(dq=None), "INVAL"), (dict(dg=None), "INVAL"), (dict(dbeta=None), "INVAL"),
                       (dict(d_last=FAKE, d_state=FAKE), "INVAL"), (dict(dv=FAKE + 4), "ALIGN"), (dict(dbeta=FAKE + 2), "ALIGN"),
                       (dict(d_last=FAKE + 4), "ALIGN"), (dict(d_o=FAKE + 1), "ALIGN")):
        assert lib.sdm_gdr_backward(by(io), by(fill(_lib.GdrGrad, GG, kw)), None) == E[status], kw
    assert lib.sdm_gdr_backward(by(io), None, None) == E["INVAL"] and lib.sdm_gdr_forward(None, None) == E["INVAL"]
    empty = fill(_lib.GdrIO, GD, dict(B=0))
    assert lib.sdm_gdr_forward(by(empty), None) == 0 and lib.sdm_gdr_backward(by(empty), by(fill(_lib.GdrGrad, GG, {})), None) == 0
    assert lib.sdm_gdr_workspace(None, 0) == 0 and lib.sdm_gdr_workspace(by(fill(_lib.GdrIO, GD, dict(T=0))), 1) == 0
    assert lib.sdm_gdr_workspace(by(fill(_lib.GdrIO, GD, dict(dtype=9))), 0) == 0
    fwd, back = lib.sdm_gdr_workspace(by(io), 0), lib.sdm_gdr_workspace(by(io), 1)
    assert fwd == 8 * 21 * 1024                                             # a record of two triangles and the factors per chunk
    states, rows = 8 * 16 * 24 * 4, 8 * 8 * 24 * 4
    assert back == 8 * 31 * 1024 + 2 * states + 2 * rows + 2 * 8 * 8 * 16 * 4


GS = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, o=FAKE, state=FAKE, new_state=FAKE, rows=2, B=2, H=4, Hk=2, dk=16, dv=24, scale=1.0)


@built
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), "SHAPE"), (dict(H=3), "SHAPE"), (dict(dk=129), "SHAPE"), (dict(dtype=2), "INVAL"), (dict(rows=1), "INVAL"),
    (dict(rows=-1, slots=FAKE), "INVAL"), (dict(state=None), "INVAL"), (dict(o=None), "INVAL"), (dict(beta=None), "INVAL"), (dict(g=FAKE + 2), "ALIGN"),
    (dict(new_state=FAKE + 8), "ALIGN"), (dict(slots=FAKE + 2), "ALIGN"), (dict(B=1 << 20, rows=1 << 20), "SHAPE"), (dict(scale=float("inf")), "INVAL"),
])
def test_gdr_step_refusals(kw, status):
    assert _lib.load().sdm_gdr_step(by(fill(_lib.GdrStepIO, GS, kw)), None) == E[status]
    assert _lib.load().sdm_gdr_step(by(fill(_lib.GdrStepIO, GS, dict(B=0))), None) == 0


GN = dict(x=FAKE, z=FAKE, out=FAKE, w=FAKE, N=8, H=2, D=64, eps=1e-6)
GNG = dict(d=FAKE, dx=FAKE, dz=FAKE, dw=FAKE, workspace=FAKE, workspace_bytes=1 << 40)


@built
@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), "SHAPE"), (dict(H=0), "SHAPE"), (dict(N=1 << 30), "SHAPE"), (dict(D=0), "SHAPE"), (dict(D=8193), "SHAPE"), (dict(dtype=3), "INVAL"),
    (dict(w_dtype=-1), "INVAL"), (dict(eps=-1.0), "INVAL"), (dict(eps=float("nan")), "INVAL"), (dict(eps=float("inf")), "INVAL"), (dict(x=None), "INVAL"),
    (dict(z=None), "INVAL"), (dict(x=FAKE + 2), "ALIGN"), (dict(z=FAKE + 1), "ALIGN"), (dict(w=FAKE + 2), "ALIGN"),
])
def test_gate_norm_refusals(kw, status):
    lib = _lib.load()
    io = fill(_lib.GateNormIO, GN, kw)
    assert lib.sdm_gate_norm(by(io), None) == E[status] and len(lib.sdm_last_error()) > 0
    assert lib.sdm_gate_norm_backward(by(io), by(fill(_lib.GateNormGrad, GNG, {})), None) == E[status]


RN = dict(x=FAKE, y=FAKE, h=FAKE + 64, n=FAKE, w=FAKE, wy=FAKE, a=FAKE, N=8, D=64, norm_y=1, eps=1e-6)
RNG = dict(dh=FAKE, dn=FAKE, dx=FAKE, dy=FAKE, dw=FAKE, dwy=FAKE, da=FAKE, workspace=FAKE, workspace_bytes=1 << 40)


@built
@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), "SHAPE"), (dict(N=1 << 31), "SHAPE"), (dict(D=0), "SHAPE"), (dict(D=8193), "SHAPE"), (dict(dtype=3), "INVAL"), (dict(w_dtype=2), "INVAL"),
    (dict(eps=-1.0), "INVAL"), (dict(norm_y=2), "INVAL"), (dict(norm_y=0), "INVAL"), (dict(y=None), "INVAL"), (dict(h=None), "INVAL"),
    (dict(y=FAKE + 2), "ALIGN"), (dict(h=FAKE + 1), "ALIGN"), (dict(w=FAKE + 2), "ALIGN"), (dict(wy=FAKE + 2), "ALIGN"), (dict(a=FAKE + 1), "ALIGN"),
])
def test_residual_norm_refusals(kw, status):
    lib = _lib.load()
    io = fill(_lib.ResidualNormIO, RN, kw)
    assert lib.sdm_residual_norm(by(io), None) == E[status] and len(lib.sdm_last_error()) > 0
    assert lib.sdm_residual_norm_backward(by(io), by(fill(_lib.ResidualNormGrad, RNG, {})), None) == E[status]


@built
def test_norms_more_refusals_and_workspaces():
    lib = _lib.load()
    assert lib.sdm_gate_norm(by(fill(_lib.GateNormIO, GN, dict(out=None))), None) == E["INVAL"]
    assert lib.sdm_gate_norm(by(fill(_lib.GateNormIO, GN, dict(out=FAKE + 2))), None) == E["ALIGN"]
    assert lib.sdm_gate_norm(by(fill(_lib.GateNormIO, GN, dict(N=0, x=None))), None) == 0 and lib.sdm_gate_norm(None, None) == E["INVAL"]
    io = fill(_lib.GateNormIO, GN, {})
    for kw, status in ((dict(d=None), "INVAL"), (dict(dx=None), "INVAL"), (dict(dz=None), "INVAL"), (dict(dw=FAKE + 2), "ALIGN"), (dict(d=FAKE + 2), "ALIGN"),
                       (dict(workspace=None), "WORKSPACE"), (dict(workspace_bytes=16), "WORKSPACE"), (dict(workspace=FAKE + 8), "ALIGN")):
        assert lib.sdm_gate_norm_backward(by(io), by(fill(_lib.GateNormGrad, GNG, kw)), None) == E[status], kw
    assert lib.sdm_gate_norm_backward(by(io), None, None) == E["INVAL"]
    assert lib.sdm_gate_norm_workspace(by(io)) == 16 * 64 * 4 and lib.sdm_gate_norm_workspace(None) == 0
    assert lib.sdm_gate_norm_workspace(by(fill(_lib.GateNormIO, GN, dict(N=100000)))) == 1024 * 64 * 4
    for kw, status in ((dict(x=None), "INVAL"), (dict(n=None), "INVAL"), (dict(n=FAKE + 64), "INVAL"), (dict(x=FAKE + 2), "ALIGN"), (dict(n=FAKE + 2), "ALIGN")):
        assert lib.sdm_residual_norm(by(fill(_lib.ResidualNormIO, RN, kw)), None) == E[status], kw
    io = fill(_lib.ResidualNormIO, RN, {})
    for kw, status in ((dict(dn=None), "INVAL"), (dict(dy=None), "INVAL"), (dict(da=FAKE + 2), "ALIGN"), (dict(dh=FAKE + 2), "ALIGN"),
                       (dict(workspace=None), "WORKSPACE"), (dict(workspace_bytes=16), "WORKSPACE")):
        assert lib.sdm_residual_norm_backward(by(io), by(fill(_lib.ResidualNormGrad, RNG, kw)), None) == E[status], kw
    plain = fill(_lib.ResidualNormIO, RN, dict(norm_y=0, wy=None))
    assert lib.sdm_residual_norm_backward(by(plain), by(fill(_lib.ResidualNormGrad, RNG, {})), None) == E["INVAL"]   # dwy without norm_y
    assert lib.sdm_residual_norm_backward(by(io), None, None) == E["INVAL"] and lib.sdm_residual_norm(None, None) == E["INVAL"]
    assert lib.sdm_residual_norm_workspace(by(io)) == 8 * 3 * 64 * 4
    assert lib.sdm_residual_norm_workspace(by(fill(_lib.ResidualNormIO, RN, dict(N=100000, D=8192)))) == 256 * 3 * 8192 * 4
