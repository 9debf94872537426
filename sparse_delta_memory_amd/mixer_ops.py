"""The mixer operators beside the bank: head norms with rotation, slot selection and the gated linear
recurrence. Argument marshalling only, as in the rest of the binding: torch provides device memory and
the current stream, the HIP kernels of libsdm_amd.so do every step, and there is no CPU fallback.

Heads are [.., heads, columns] device tensors with contiguous columns and any strides before them (views
of a packed projection, say), float32 or bfloat16. Outputs are allocated unless given. Every call takes
the current stream of the inputs' device, or `stream`; tensors that come from another stream are the
caller's to order, as everywhere in torch.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib

_CODE = {torch.float32: _lib.SDM_F32, torch.bfloat16: _lib.SDM_BF16}


def _code(name, t):
    c = _CODE.get(t.dtype)
    if c is None:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    return c


def _same(fn, first, **others):
    """Every tensor on the first one's device (any that are None are left out)."""
    if not first.is_cuda:
        raise TypeError("%s: the tensors must be on a GPU" % fn)
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise TypeError("%s: %s is on %s, not on %s" % (fn, name, t.device, first.device))


def _shape(fn, name, t, want):
    if tuple(t.shape) != tuple(want):
        raise ValueError("%s: %s is %s, expected %s" % (fn, name, tuple(t.shape), tuple(want)))


def _columns(fn, **tensors):
    """Contiguous columns (a last dimension of one element has no stride to speak of)."""
    for name, t in tensors.items():
        if t is not None and t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError("%s: %s must have contiguous columns" % (fn, name))


def _dense(fn, dtype, **tensors):
    for name, t in tensors.items():
        if t is not None and (t.dtype != dtype or not t.is_contiguous()):
            raise TypeError("%s: %s must be a contiguous %s tensor" % (fn, name, dtype))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(fn, device, stream, *structs):
    st = torch.cuda.current_stream(device) if stream is None else stream
    if device.index is not None and device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            _lib.check(fn(*[ctypes.byref(s) for s in structs], st.cuda_stream))
    else:
        _lib.check(fn(*[ctypes.byref(s) for s in structs], st.cuda_stream))


# --------------------------------------------------------------------------- head norms with rotation

def rope_table(rows, rot, base=10000.0, scaling=1.0, base_growth=1.0, device="cuda"):
    """Cosines and sines of every position's angles, [rows, rot] float32 (the cosines of the rot/2 angles,
    then the sines): angle i of position p is p / scaling * b^(-2 i / rot). Made once per model.

    For contexts longer than the trained one by a factor f: scaling = f spreads the trained angles over
    the longer range; base_growth = f instead raises the base, b = base * f^(rot / (rot - 2)), so that the
    slowest angle is spread by f and the fastest one stays."""
    rot = int(rot)
    if rot < 0 or rot % 2 or rows < 1 or not base > 1.0 or not scaling > 0.0 or not base_growth > 0.0:
        raise ValueError("rope_table: rows >= 1, rot even and >= 0, base > 1, scaling and base_growth > 0")
    if rot == 0:
        return torch.zeros((rows, 0), dtype=torch.float32, device=device)
    b = base * base_growth ** (rot / (rot - 2)) if rot > 2 else base
    freq = b ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot) / scaling
    ang = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _norm_rope_io(fn, q, k, q_weight, k_weight, positions, table, interleaved, eps, q_out, k_out):
    if q is None and k is None:
        raise TypeError("%s: q or k is required" % fn)
    one = q if q is not None else k
    _same(fn, one, q=q, k=k, q_weight=q_weight, k_weight=k_weight, positions=positions, table=table, q_out=q_out, k_out=k_out)
    N, D = one.shape[0], one.shape[-1]
    dt = _code("%s: q and k" % fn, one)
    for name, t, o, w in (("q", q, q_out, q_weight), ("k", k, k_out, k_weight)):
        if t is None:
            continue
        if t.dim() != 3 or t.shape[0] != N or t.shape[2] != D:
            raise ValueError("%s: %s is %s, expected [%d, heads, %d]" % (fn, name, tuple(t.shape), N, D))
        if t.dtype != one.dtype or o.dtype != one.dtype:
            raise TypeError("%s: q, k and the outputs must have one dtype" % fn)
        _shape(fn, "%s's output" % name, o, t.shape)
        if w is not None:
            _shape(fn, "%s_weight" % name, w, (D,))
    _columns(fn, q=q, k=k, q_out=q_out, k_out=k_out, q_weight=q_weight, k_weight=k_weight)
    wd = _lib.SDM_F32
    for w in (q_weight, k_weight):
        if w is not None:
            wd = _code("%s: the norm weights" % fn, w)
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise TypeError("%s: q_weight and k_weight must have one dtype" % fn)
    rot = 0
    if table is not None and table.shape[-1] > 0:
        _dense(fn, torch.float32, table=table)
        if table.dim() != 2:
            raise ValueError("%s: table must be [positions, rot]" % fn)
        rot = table.shape[1]
        if positions is None or positions.dtype not in (torch.int32, torch.int64) or not positions.is_contiguous():
            raise TypeError("%s: positions must be a contiguous int32 or int64 tensor" % fn)
        _shape(fn, "positions", positions, (N,))
    st = lambda t: (0, 0) if t is None else (t.stride(0), t.stride(1))  # noqa: E731
    return _lib.NormRopeIO(
        _ptr(q), _ptr(k), *st(q), *st(k), _ptr(q_out), _ptr(k_out), *st(q_out), *st(k_out), _ptr(q_weight), _ptr(k_weight),
        _ptr(positions) if rot else None, _ptr(table) if rot else None, table.shape[0] if rot else 0, N,
        0 if q is None else q.shape[1], 0 if k is None else k.shape[1], D, rot, int(bool(interleaved)), dt, wd,
        positions.element_size() if rot else 4, float(eps))


def norm_rope(q, k, q_weight=None, k_weight=None, positions=None, table=None, interleaved=False, eps=1e-6, q_out=None, k_out=None,
              stream=None):
    """(q_out, k_out): every head of q [N, Hq, D] and k [N, Hk, D] divided by its root mean square (eps added
    to the mean), times the weights [D] (float32 or bfloat16; None: ones), and its first rot columns turned by
    the token's angles: row positions[t] of `table` [rows, rot] (rope_table; None: no rotation). Pairs are
    (i, i + rot/2), or (2i, 2i + 1) when interleaved. A position outside the table takes its nearest row. q or k may
    be None; an output may be its input."""
    if q_out is None and q is not None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if k_out is None and k is not None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    io = _norm_rope_io("norm_rope", q, k, q_weight, k_weight, positions, table, interleaved, eps, q_out, k_out)
    _call(_lib.load().sdm_norm_rope, (q if q is not None else k).device, stream, io)
    return q_out, k_out


def norm_rope_backward(d_q, d_k, q, k, q_weight=None, k_weight=None, positions=None, table=None, interleaved=False, eps=1e-6,
                       stream=None):
    """The backward of norm_rope at its inputs, from the gradients d_q and d_k of its outputs: a dict of dq, dk (like
    q and k, contiguous) and dwq, dwk ([D] float32; None without that tensor)."""
    fn = "norm_rope_backward"
    dq = None if q is None else torch.empty(q.shape, dtype=q.dtype, device=q.device)
    dk = None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device)
    io = _norm_rope_io(fn, q, k, q_weight, k_weight, positions, table, interleaved, eps, dq, dk)
    one = q if q is not None else k
    for name, t, d in (("d_q", q, d_q), ("d_k", k, d_k)):
        if t is None:
            continue
        if d is None or d.dtype != t.dtype or d.device != t.device:
            raise TypeError("%s: %s must have the dtype and device of its head tensor" % (fn, name))
        _shape(fn, name, d, t.shape)
    _columns(fn, d_q=d_q if q is not None else None, d_k=d_k if k is not None else None)
    lib = _lib.load()
    ws = torch.empty(max(int(lib.sdm_norm_rope_workspace(ctypes.byref(io))), 16), dtype=torch.uint8, device=one.device)
    dw = torch.empty((2, one.shape[-1]), dtype=torch.float32, device=one.device)
    st = lambda t: (0, 0) if t is None else (t.stride(0), t.stride(1))  # noqa: E731
    g = _lib.NormRopeGrad(_ptr(d_q) if q is not None else None, _ptr(d_k) if k is not None else None,
                          *st(d_q if q is not None else None), *st(d_k if k is not None else None),
                          dw[0].data_ptr() if q is not None else None, dw[1].data_ptr() if k is not None else None,
                          ws.data_ptr(), ws.numel())
    _call(lib.sdm_norm_rope_backward, one.device, stream, io, g)
    return dict(dq=dq, dk=dk, dwq=None if q is None else dw[0], dwk=None if k is None else dw[1])


# ------------------------------------------------------------------------------------- slot selection

def _slot_io(fn, a, b, K, idx, val, scale, shape):
    _same(fn, a, b=b, idx=idx, val=val)
    if a.dim() < 2 or a.shape[:-1] != b.shape[:-1] or a.dtype != b.dtype:
        raise ValueError("%s: a %s and b %s must be [.., n1] and [.., n2] of one dtype" % (fn, tuple(a.shape), tuple(b.shape)))
    _columns(fn, a=a, b=b)
    rows = []
    for name, t in (("a", a), ("b", b)):   # leading dimensions that fold into one row stride
        v = t if t.dim() == 2 else t.flatten(0, -2) if t.is_contiguous() else None
        if v is None:
            raise ValueError("%s: %s must be 2-D or contiguous" % (fn, name))
        rows.append(v)
    C, P, off = 0, 1, 0
    if shape is not None:
        C, P, off = shape.C, shape.P, shape.stream_offset
    return _lib.SlotTopkIO(
        a.data_ptr(), b.data_ptr(), rows[0].stride(0), rows[1].stride(0), _ptr(idx), _ptr(val), rows[0].shape[0], a.shape[-1], b.shape[-1],
        int(K), _code("%s: the scores" % fn, a), _lib.SDM_F32 if val is None else _code("%s: val" % fn, val), idx.element_size(),
        float(scale), C, P, off)


def slot_topk(a, b, K, scale=1.0, shape=None, idx=None, val=None, idx_dtype=torch.int32, val_dtype=torch.float32, stream=None):
    """(idx, val) [.., K]: ids and weights of each token's K best slots of a bank of n1 x n2, from its scores
    a [.., n1] and b [.., n2]; a slot's score is a[i] + b[j], its id i * n2 + j. The K best of each row, then the K
    best sums of those, the best first (of equal ones the lower column; of equal sums the better a, then the better
    b), and the softmax of the K sums times scale. NaN counts as -infinity, and a sum of -infinity weighs 0.

    shape: a Phase-1 shape whose chunks the tokens are ([N, C, n]): ids are then absolute, chunk c's plus
    (c % P) * stream_offset, and idx, val can be Phase 1's k_idx, k_val (or q_idx, q_val)."""
    out = tuple(a.shape[:-1]) + (int(K),)
    if idx is None:
        idx = torch.empty(out, dtype=idx_dtype, device=a.device)
    if val is None:
        val = torch.empty(out, dtype=val_dtype, device=a.device)
    for name, t in (("idx", idx), ("val", val)):
        _shape("slot_topk", name, t, out)
        if not t.is_contiguous():
            raise ValueError("slot_topk: %s must be contiguous" % name)
    if idx.dtype not in (torch.int32, torch.int64):
        raise TypeError("slot_topk: idx must be int32 or int64")
    io = _slot_io("slot_topk", a, b, K, idx, val, scale, shape)
    _call(_lib.load().sdm_slot_topk, a.device, stream, io)
    return idx, val


def slot_topk_backward(d_val, idx, a, b, scale=1.0, shape=None, stream=None):
    """(d_a, d_b): the gradients of the scores, like a and b, from the gradients d_val [.., K] float32 of slot_topk's
    weights at its selection idx."""
    fn = "slot_topk_backward"
    K = idx.shape[-1]
    if idx.dtype not in (torch.int32, torch.int64) or not idx.is_contiguous():
        raise TypeError("%s: idx must be a contiguous int32 or int64 tensor" % fn)
    _shape(fn, "idx", idx, tuple(a.shape[:-1]) + (K,))
    _dense(fn, torch.float32, d_val=d_val)
    _shape(fn, "d_val", d_val, idx.shape)
    _same(fn, a, d_val=d_val)
    io = _slot_io(fn, a, b, K, idx, None, scale, shape)
    da, db = torch.empty(a.shape, dtype=a.dtype, device=a.device), torch.empty(b.shape, dtype=b.dtype, device=b.device)
    g = _lib.SlotTopkGrad(d_val.data_ptr(), da.data_ptr(), db.data_ptr(), a.shape[-1], b.shape[-1])
    _call(_lib.load().sdm_slot_topk_backward, a.device, stream, io, g)
    return da, db


# ------------------------------------------------------------------------- the gated linear recurrence

def _glr_io(fn, q, k, v, g, scale, state, lens, o, last):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("%s: q, k are [B, T, Hk, dk] and v is [B, T, H, dv]" % fn)
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2], v.shape[3]
    _same(fn, q, k=k, v=v, g=g, state=state, lens=lens, o=o, last=last)
    _shape(fn, "k", k, q.shape)
    _shape(fn, "v", v, (B, T, H, dv))
    _shape(fn, "g", g, (B, T, H))
    if k.dtype != q.dtype or v.dtype != q.dtype or g.dtype != torch.float32:
        raise TypeError("%s: q, k and v must have one dtype, and g must be float32" % fn)
    _columns(fn, q=q, k=k, v=v, o=o)
    _dense(fn, torch.float32, state=state, last=last)
    _dense(fn, torch.int32, lens=lens)
    for name, t in (("state", state), ("last", last)):
        if t is not None:
            _shape(fn, name, t, (B, H, dk, dv))
    if lens is not None:
        _shape(fn, "lens", lens, (B,))
    if o is not None:
        _shape(fn, "out", o, v.shape)
        if o.dtype != v.dtype:
            raise TypeError("%s: out must have v's dtype" % fn)
    return _lib.GlrIO(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), *q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *g.stride(),
        _ptr(state), _ptr(lens), _ptr(o), *((0, 0, 0) if o is None else o.stride()[:3]), _ptr(last), B, T, H, Hk, dk, dv,
        _code("%s: q, k and v" % fn, q), float(dk ** -0.5 if scale is None else scale), None, 0)


def _glr_space(fn, io, backward, workspace, device):
    lib = _lib.load()
    if workspace is None:
        need = int(lib.sdm_glr_workspace(ctypes.byref(io), backward))
        workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    elif workspace.device != device or not workspace.is_contiguous():
        raise TypeError("%s: workspace must be a contiguous tensor on %s" % (fn, device))
    if workspace is not None:
        io.workspace, io.workspace_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    return workspace


def glr_workspace_bytes(B, T, H, Hk, dk, dv, backward=False):
    """Bytes of the workspace of glr_forward (or glr_backward) for these sizes; 0 when it needs none."""
    io = _lib.GlrIO()
    io.B, io.T, io.H, io.Hk, io.dk, io.dv = int(B), int(T), int(H), int(Hk), int(dk), int(dv)
    return int(_lib.load().sdm_glr_workspace(ctypes.byref(io), int(bool(backward))))


def glr_forward(q, k, v, g, scale=None, state=None, lens=None, out=None, last=None, workspace=None, stream=None):
    """(out, last) of the gated linear recurrence: per stream and head, from S = state,
        S_t = exp(g_t) S_{t-1} + k_t v_t^T,    out_t = scale S_t^T q_t.

    q, k [B, T, Hk, dk], v [B, T, H, dv] float32 or bfloat16, g [B, T, H] float32 log gates (<= 0; -infinity resets the
    state). H is a multiple of Hk: value head h uses query and key head h // (H // Hk). dk, dv: 1..128. scale: dk^-0.5
    by default. state [B, H, dk, dv] float32 (None: zero). lens [B] int32 on the device: tokens of each stream, whose later tokens
    are not read and get zero outputs (None: T). last: the state after the last token. workspace: a uint8 tensor of
    glr_workspace_bytes (allocated per call by default)."""
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    if last is None:
        last = torch.empty((q.shape[0], v.shape[2], q.shape[3], v.shape[3]), dtype=torch.float32, device=v.device)
    io = _glr_io("glr_forward", q, k, v, g, scale, state, lens, out, last)
    keep = _glr_space("glr_forward", io, 0, workspace, q.device)  # noqa: F841
    _call(_lib.load().sdm_glr_forward, q.device, stream, io)
    return out, last


def glr_backward(d_out, q, k, v, g, scale=None, state=None, d_last=None, lens=None, workspace=None, stream=None):
    """The backward of glr_forward at its inputs, from the gradients d_out of out and d_last [B, H, dk, dv] float32 of the
    last state (None: zero): a dict of dq, dk, dv (contiguous, like q, k, v), dg [B, T, H] float32 and dstate (the
    gradient of the first state, [B, H, dk, dv] float32). Nothing of the forward is needed but its inputs."""
    fn = "glr_backward"
    io = _glr_io(fn, q, k, v, g, scale, state, lens, None, None)
    _same(fn, q, d_out=d_out, d_last=d_last)
    _shape(fn, "d_out", d_out, v.shape)
    if d_out.dtype != v.dtype:
        raise TypeError("%s: d_out must have v's dtype" % fn)
    _columns(fn, d_out=d_out)
    _dense(fn, torch.float32, d_last=d_last)
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    if d_last is not None:
        _shape(fn, "d_last", d_last, (B, H, dk, dv))
    r = dict(dq=torch.empty(q.shape, dtype=q.dtype, device=q.device), dk=torch.empty(k.shape, dtype=q.dtype, device=q.device),
             dv=torch.empty(v.shape, dtype=q.dtype, device=q.device), dg=torch.empty((B, T, H), dtype=torch.float32, device=q.device),
             dstate=torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device))
    keep = _glr_space(fn, io, 1, workspace, q.device)  # noqa: F841
    grad = _lib.GlrGrad(d_out.data_ptr(), *d_out.stride()[:3], _ptr(d_last), *[r[n].data_ptr() for n in ("dq", "dk", "dv", "dg", "dstate")])
    _call(_lib.load().sdm_glr_backward, q.device, stream, io, grad)
    return r


def glr_step(q, k, v, g, state, scale=None, new_state=None, slots=None, out=None, stream=None):
    """One token of B requests: their states updated in place (or into new_state, laid out the same) and the outputs.

    q, k [B, Hk, dk], v [B, H, dv], g [B, H] float32, state [rows, H, dk, dv] float32 contiguous. slots [B] int32 on the device:
    the row of each request (None: row b); rows must be distinct, and a request whose row is outside the
    tensor is left out (output 0). Returns out [B, H, dv]."""
    fn = "glr_step"
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("%s: q, k are [B, Hk, dk] and v is [B, H, dv]" % fn)
    B, Hk, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    if new_state is None:
        new_state = state
    _same(fn, q, k=k, v=v, g=g, state=state, new_state=new_state, slots=slots, out=out)
    if k.shape != q.shape or v.shape[0] != B or tuple(g.shape) != (B, H) or out.shape != v.shape:
        raise ValueError("%s: q %s, k %s, v %s, g %s, out %s do not fit" % (fn, tuple(q.shape), tuple(k.shape), tuple(v.shape), tuple(g.shape),
                                                                          tuple(out.shape)))
    if k.dtype != q.dtype or v.dtype != q.dtype or out.dtype != q.dtype or g.dtype != torch.float32:
        raise TypeError("%s: q, k, v and out must have one dtype, and g must be float32" % fn)
    _columns(fn, q=q, k=k, v=v, out=out)
    _dense(fn, torch.float32, state=state, new_state=new_state)
    if state.shape[1:] != (H, dk, dv) or new_state.shape != state.shape:
        raise ValueError("%s: state is %s, expected [rows, %d, %d, %d]" % (fn, tuple(state.shape), H, dk, dv))
    if slots is not None:
        _dense(fn, torch.int32, slots=slots)
        _shape(fn, "slots", slots, (B,))
    io = _lib.GlrStepIO(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), *q.stride()[:2], *k.stride()[:2], *v.stride()[:2], *g.stride(),
        state.data_ptr(), new_state.data_ptr(), state.shape[0], _ptr(slots), out.data_ptr(), *out.stride()[:2], B, H, Hk, dk, dv,
        _code("%s: q, k and v" % fn, q), float(dk ** -0.5 if scale is None else scale))
    _call(_lib.load().sdm_glr_step, q.device, stream, io)
    return out
