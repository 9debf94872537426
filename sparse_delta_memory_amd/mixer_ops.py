"""The mixer operators beside the bank: head norms with rotation, slot selection and the gated linear
recurrence. Argument marshalling only, as in the rest of the binding: torch provides device memory and
the current stream, the HIP kernels of libsdm_amd.so do every step, and there is no CPU fallback.

Heads are [.., heads, columns] device tensors with contiguous columns and any strides before them (views
of a packed projection, say), float32 or bfloat16. Outputs are allocated unless given. Every call takes
the current stream of the inputs' device, or `stream`: then the outputs and the workspace that the call allocates
are that stream's (no work still queued elsewhere uses their memory), the outputs kept for the current one too. Inputs
and outputs that another stream made or uses are the caller's to order, as everywhere in torch.
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


def _same(fn, first, *others):
    """Every tensor on the first one's GPU (any that are None are left out)."""
    dev = first.device
    if dev.type != "cuda":
        raise TypeError("%s: the tensors must be on a GPU" % fn)
    for t in others:
        if t is not None and t.device != dev:
            raise TypeError("%s: a tensor is on %s, not on %s" % (fn, t.device, dev))
    return dev


def _shape(fn, name, t, want):
    if t.shape != want:
        raise ValueError("%s: %s is %s, expected %s" % (fn, name, tuple(t.shape), tuple(want)))


def _columns(fn, *tensors):
    """Contiguous columns (a last dimension of one element has no stride to speak of)."""
    for t in tensors:
        if t is not None and t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError("%s: tensors must have contiguous columns" % fn)


def _dense(fn, dtype, *tensors):
    for t in tensors:
        if t is not None and (t.dtype is not dtype or not t.is_contiguous()):
            raise TypeError("%s: expected a contiguous %s tensor, got %s %s" % (fn, dtype, t.dtype, tuple(t.stride())))


def _ptr(t):
    return 0 if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it, where torch has that (2 us of a small call's 10).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _own(stream, shape, dtype, dev):
    """Memory of the stream that will use it: what a block freed on the current stream held may still be in use there, and
    `stream` does not wait for that."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _output(stream, shape, dtype, dev):
    """A tensor that the call returns: the caller goes on with it on the current stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    t = _own(stream, shape, dtype, dev)
    if t.is_cuda:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _output_like(stream, t):
    """The same with t's shape and type (on the current stream by the shortest way: small calls are this side's time)."""
    return t.new_empty(t.shape) if stream is None else _output(stream, t.shape, t.dtype, t.device)


def _call(fn, dev, stream, *packed, workspace=None):
    """Enqueues fn. workspace: the caller's, which the stream still needs when the call returns."""
    if stream is not None:
        if stream.device != dev:
            raise TypeError("the stream is on %s, the tensors are on %s" % (stream.device, dev))
        if workspace is not None:
            workspace.record_stream(stream)
    st = _raw_stream(dev.index) if stream is None else stream.cuda_stream
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            _lib.check(fn(*packed, st))
    else:
        _lib.check(fn(*packed, st))


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


def _head(fn, t, out, w, N, D, dt, rows):
    """Checks of one tensor of heads against the first one's N, D and dtype; appends its strides to rows."""
    if t.dim() != 3 or t.shape[0] != N or t.shape[2] != D:
        raise ValueError("%s: heads are %s, expected [%d, heads, %d]" % (fn, tuple(t.shape), N, D))
    if t.dtype is not dt or out.dtype is not dt:
        raise TypeError("%s: q, k and the outputs must have one dtype" % fn)
    _shape(fn, "an output", out, t.shape)
    if w is not None:
        _shape(fn, "a norm weight", w, (D,))
    _columns(fn, t, out, w)
    s, o = t.stride(), out.stride()
    rows.append((t.shape[1], s[0], s[1], o[0], o[1]))


def _norm_rope_io(fn, q, k, q_weight, k_weight, positions, table, interleaved, eps, q_out, k_out):
    one = q if q is not None else k
    dev = _same(fn, one, k, q_weight, k_weight, positions, table, q_out, k_out)
    if one.dim() != 3:
        raise ValueError("%s: heads are [tokens, heads, columns]" % fn)
    N, _, D = one.shape
    code = _code(fn, one)
    rows = []
    for t, o, w in ((q, q_out, q_weight), (k, k_out, k_weight)):
        if t is None:
            rows.append((0, 0, 0, 0, 0))
        else:
            _head(fn, t, o, w, N, D, one.dtype, rows)
    wd = _lib.SDM_F32
    if q is None:      # a weight without its heads is not used
        q_weight = None
    if k is None:
        k_weight = None
    w = q_weight if q_weight is not None else k_weight
    if w is not None:
        wd = _code(fn, w)
        if k_weight is not None and k_weight.dtype is not w.dtype:
            raise TypeError("%s: q_weight and k_weight must have one dtype" % fn)
    rot = trows = pos = tab = 0
    pb = 4
    if table is not None and table.shape[-1] > 0:
        _dense(fn, torch.float32, table)
        if table.dim() != 2:
            raise ValueError("%s: table must be [positions, rot]" % fn)
        trows, rot = table.shape
        if positions is None or positions.dtype not in (torch.int32, torch.int64) or not positions.is_contiguous():
            raise TypeError("%s: positions must be a contiguous int32 or int64 tensor" % fn)
        _shape(fn, "positions", positions, (N,))
        pb = 8 if positions.dtype is torch.int64 else 4
        pos, tab = positions.data_ptr(), table.data_ptr()
    (Hq, qr, qh, qor, qoh), (Hk, kr, kh, kor, koh) = rows
    return dev, _lib.pack_norm_rope(_ptr(q), _ptr(k), qr, qh, kr, kh, _ptr(q_out), _ptr(k_out), qor, qoh, kor, koh, _ptr(q_weight), _ptr(k_weight),
                                    pos, tab, trows, N, Hq, Hk, D, rot, 1 if interleaved else 0, code, wd, pb, float(eps))


def norm_rope(q, k, q_weight=None, k_weight=None, positions=None, table=None, interleaved=False, eps=1e-6, q_out=None, k_out=None,
              stream=None):
    """(q_out, k_out): every head of q [N, Hq, D] and k [N, Hk, D] divided by its root mean square (eps added
    to the mean), times the weights [D] (float32 or bfloat16; None: ones), and its first rot columns turned by
    the token's angles: row positions[t] of `table` [rows, rot] (rope_table; None: no rotation). Pairs are
    (i, i + rot/2), or (2i, 2i + 1) when interleaved. A position outside the table takes its nearest row. q or k may
    be None; an output may be its input."""
    if q is None and k is None:
        raise TypeError("norm_rope: q or k is required")
    if q_out is None and q is not None:
        q_out = _output_like(stream, q)
    if k_out is None and k is not None:
        k_out = _output_like(stream, k)
    dev, io = _norm_rope_io("norm_rope", q, k, q_weight, k_weight, positions, table, interleaved, eps, q_out, k_out)
    _call(_lib.load().sdm_norm_rope, dev, stream, io)
    return q_out, k_out


def norm_rope_backward(d_q, d_k, q, k, q_weight=None, k_weight=None, positions=None, table=None, interleaved=False, eps=1e-6,
                       stream=None):
    """The backward of norm_rope at its inputs, from the gradients d_q and d_k of its outputs: a dict of dq, dk (like
    q and k, contiguous) and dwq, dwk ([D] float32; None without that tensor)."""
    fn = "norm_rope_backward"
    if q is None and k is None:
        raise TypeError("%s: q or k is required" % fn)
    dq = None if q is None else _output_like(stream, q)
    dk = None if k is None else _output_like(stream, k)
    dev, io = _norm_rope_io(fn, q, k, q_weight, k_weight, positions, table, interleaved, eps, dq, dk)
    one = q if q is not None else k
    grads = []
    for name, t, d in (("d_q", q, d_q), ("d_k", k, d_k)):
        if t is None:
            grads.append((0, 0, 0))
            continue
        if d is None or d.dtype is not t.dtype or d.device != dev:
            raise TypeError("%s: %s must have the dtype and device of its heads" % (fn, name))
        _shape(fn, name, d, t.shape)
        _columns(fn, d)
        grads.append((d.data_ptr(), d.stride(0), d.stride(1)))
    lib = _lib.load()
    ws = _own(stream, max(int(lib.sdm_norm_rope_workspace(io)), 16), torch.uint8, dev)
    D = one.shape[-1]
    dw = _output(stream, (2, D), torch.float32, dev)
    at = dw.data_ptr()
    (gq, gqr, gqh), (gk, gkr, gkh) = grads
    g = _lib.pack_norm_rope_grad(gq, gk, gqr, gqh, gkr, gkh, 0 if q is None else at, 0 if k is None else at + 4 * D, ws.data_ptr(), ws.numel())
    _call(lib.sdm_norm_rope_backward, dev, stream, io, g)
    return dict(dq=dq, dk=dk, dwq=None if q is None else dw[0], dwk=None if k is None else dw[1])


# ------------------------------------------------------------------------------------- slot selection

def _row_stride(fn, t):
    """The stride between the rows of t [.., n], whose leading dimensions must fold into one (those of a view of a packed
    projection do)."""
    dims = [(n, s) for n, s in zip(t.shape[:-1], t.stride()[:-1]) if n != 1]
    for (_, s), (n, inner) in zip(dims, dims[1:]):
        if s != n * inner and t.numel() > 0:
            raise ValueError("%s: the rows of %s with strides %s are not evenly spaced" % (fn, tuple(t.shape), tuple(t.stride())))
    return dims[-1][1] if dims else t.shape[-1]


def _slot_io(fn, a, b, K, idx, val, scale, shape):
    dev = _same(fn, a, b, idx, val)
    if a.dim() < 2 or a.shape[:-1] != b.shape[:-1] or a.dtype is not b.dtype:
        raise ValueError("%s: a %s and b %s must be [.., n1] and [.., n2] of one dtype" % (fn, tuple(a.shape), tuple(b.shape)))
    _columns(fn, a, b)
    n1, n2 = a.shape[-1], b.shape[-1]
    ra, rb = (a.stride(0), b.stride(0)) if a.dim() == 2 else (_row_stride(fn, a), _row_stride(fn, b))
    C, P, off = (0, 1, 0) if shape is None else (shape.C, shape.P, shape.stream_offset)
    if shape is not None and a.shape[:-1].numel() != shape.N * C:
        raise ValueError("%s: %d rows of scores, the shape has %d chunks of %d tokens" % (fn, a.shape[:-1].numel(), shape.N, C))
    return dev, _lib.pack_slot_topk(a.data_ptr(), b.data_ptr(), ra, rb, _ptr(idx), _ptr(val), idx.numel() // K if K else 0, n1, n2, K, _code(fn, a),
                                    0 if val is None else _code(fn, val), 8 if idx.dtype is torch.int64 else 4, float(scale), C, P, off)


def slot_topk(a, b, K, scale=1.0, shape=None, idx=None, val=None, idx_dtype=torch.int32, val_dtype=torch.float32, stream=None):
    """(idx, val) [.., K]: ids and weights of each token's K best slots of a bank of n1 x n2, from its scores
    a [.., n1] and b [.., n2] (each with evenly spaced rows); a slot's score is a[i] + b[j], its id i * n2 + j. The
    K best of each row, then the K best sums of those, the best first (of equal ones the lower column; of equal sums the better a, then the better
    b), and the softmax of the K sums times scale. NaN counts as -infinity, and a sum of -infinity weighs 0.

    shape: a Phase-1 shape whose chunks the tokens are ([N, C, n], or N * C rows): ids are then absolute, chunk c's plus
    (c % P) * stream_offset, and idx, val can be Phase 1's k_idx, k_val (or q_idx, q_val)."""
    K = int(K)
    out = a.shape[:-1] + (K,)
    if idx is None:
        idx = _output(stream, out, idx_dtype, a.device)
    if val is None:
        val = _output(stream, out, val_dtype, a.device)
    for name, t in (("idx", idx), ("val", val)):
        _shape("slot_topk", name, t, out)
        if not t.is_contiguous():
            raise ValueError("slot_topk: %s must be contiguous" % name)
    if idx.dtype not in (torch.int32, torch.int64):
        raise TypeError("slot_topk: idx must be int32 or int64")
    dev, io = _slot_io("slot_topk", a, b, K, idx, val, scale, shape)
    _call(_lib.load().sdm_slot_topk, dev, stream, io)
    return idx, val


def slot_topk_backward(d_val, idx, a, b, scale=1.0, shape=None, stream=None):
    """(d_a, d_b): the gradients of the scores, like a and b, from the gradients d_val [.., K] float32 of slot_topk's
    weights at its selection idx."""
    fn = "slot_topk_backward"
    K = idx.shape[-1]
    if idx.dtype not in (torch.int32, torch.int64) or not idx.is_contiguous():
        raise TypeError("%s: idx must be a contiguous int32 or int64 tensor" % fn)
    _shape(fn, "idx", idx, a.shape[:-1] + (K,))
    _dense(fn, torch.float32, d_val)
    _shape(fn, "d_val", d_val, idx.shape)
    _same(fn, a, d_val)
    dev, io = _slot_io(fn, a, b, K, idx, None, scale, shape)
    da, db = _output_like(stream, a), _output_like(stream, b)
    g = _lib.pack_slot_topk_grad(d_val.data_ptr(), da.data_ptr(), db.data_ptr(), a.shape[-1], b.shape[-1])
    _call(_lib.load().sdm_slot_topk_backward, dev, stream, io, g)
    return da, db


# ------------------------------------------------------------------------- the gated linear recurrence

def _glr_io(fn, q, k, v, g, scale, state, lens, o, last, backward, workspace, stream):
    """The call's device and structure, and the workspace to keep until it is enqueued."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("%s: q, k are [B, T, Hk, dk] and v is [B, T, H, dv]" % fn)
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2], v.shape[3]
    dev = _same(fn, q, k, v, g, state, lens, o, last, workspace)
    _shape(fn, "k", k, q.shape)
    _shape(fn, "v", v, (B, T, H, dv))
    _shape(fn, "g", g, (B, T, H))
    if k.dtype is not q.dtype or v.dtype is not q.dtype or g.dtype is not torch.float32:
        raise TypeError("%s: q, k and v must have one dtype, and g must be float32" % fn)
    _columns(fn, q, k, v, o)
    _dense(fn, torch.float32, state, last)
    _dense(fn, torch.int32, lens)
    for name, t in (("state", state), ("last", last)):
        if t is not None:
            _shape(fn, name, t, (B, H, dk, dv))
    if lens is not None:
        _shape(fn, "lens", lens, (B,))
    if o is not None:
        _shape(fn, "out", o, v.shape)
        if o.dtype is not v.dtype:
            raise TypeError("%s: out must have v's dtype" % fn)
    if workspace is not None and not workspace.is_contiguous():
        raise TypeError("%s: workspace must be contiguous" % fn)
    fields = (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), *q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *g.stride(),
              _ptr(state), _ptr(lens), _ptr(o), *((0, 0, 0) if o is None else o.stride()[:3]), _ptr(last), B, T, H, Hk, dk, dv,
              _code(fn, q), float(dk ** -0.5 if scale is None else scale))
    if workspace is None:
        need = int(_lib.load().sdm_glr_workspace(_lib.pack_glr(*fields, 0, 0), backward))
        workspace = _own(stream, need, torch.uint8, dev) if need else None
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return dev, _lib.pack_glr(*fields, _ptr(workspace), size), workspace


def glr_workspace_bytes(B, T, H, Hk, dk, dv, backward=False):
    """Bytes of the workspace of glr_forward (or glr_backward) for these sizes; 0 when it needs none."""
    io = _lib.GlrIO()
    io.B, io.T, io.H, io.Hk, io.dk, io.dv = int(B), int(T), int(H), int(Hk), int(dk), int(dv)
    return int(_lib.load().sdm_glr_workspace(ctypes.byref(io), int(bool(backward))))


def glr_forward(q, k, v, g, scale=None, state=None, lens=None, out=None, last=None, workspace=None, stream=None):
    """(out, last) of the gated linear recurrence: per stream and head, from S = state,
        S_t = exp(g_t) S_{t-1} + k_t v_t^T,    out_t = scale S_t^T q_t.

    q, k [B, T, Hk, dk], v [B, T, H, dv] float32 or bfloat16, g [B, T, H] float32 log gates (<= 0; -infinity resets the
    state, whatever it held). H is a multiple of Hk: value head h uses query and key head h // (H // Hk). dk, dv: 1..128. scale: dk^-0.5
    by default. state [B, H, dk, dv] float32 (None: zero). lens [B] int32 on the device: tokens of each stream, whose later tokens
    are not read and get zero outputs (None: T). last: the state after the last token. workspace: a uint8 tensor of
    glr_workspace_bytes (allocated per call by default)."""
    if q.dim() == 4 and v.dim() == 4:
        if out is None:
            out = _output_like(stream, v)
        if last is None:
            last = _output(stream, (q.shape[0], v.shape[2], q.shape[3], v.shape[3]), torch.float32, v.device)
    dev, io, keep = _glr_io("glr_forward", q, k, v, g, scale, state, lens, out, last, 0, workspace, stream)
    _call(_lib.load().sdm_glr_forward, dev, stream, io, workspace=workspace)
    return out, last


def glr_backward(d_out, q, k, v, g, scale=None, state=None, d_last=None, lens=None, workspace=None, stream=None):
    """The backward of glr_forward at its inputs, from the gradients d_out of out and d_last [B, H, dk, dv] float32 of the
    last state (None: zero): a dict of dq, dk, dv (contiguous, like q, k, v), dg [B, T, H] float32 and dstate (the
    gradient of the first state, [B, H, dk, dv] float32). Nothing of the forward is needed but its inputs."""
    fn = "glr_backward"
    dev, io, keep = _glr_io(fn, q, k, v, g, scale, state, lens, None, None, 1, workspace, stream)
    _same(fn, q, d_out, d_last)
    _shape(fn, "d_out", d_out, v.shape)
    if d_out.dtype is not v.dtype:
        raise TypeError("%s: d_out must have v's dtype" % fn)
    _columns(fn, d_out)
    _dense(fn, torch.float32, d_last)
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    if d_last is not None:
        _shape(fn, "d_last", d_last, (B, H, dk, dv))
    new = lambda shape, dtype: _output(stream, shape, dtype, dev)  # noqa: E731
    r = dict(dq=new(q.shape, q.dtype), dk=new(k.shape, q.dtype), dv=new(v.shape, q.dtype), dg=new((B, T, H), torch.float32),
             dstate=new((B, H, dk, dv), torch.float32))
    grad = _lib.pack_glr_grad(d_out.data_ptr(), *d_out.stride()[:3], _ptr(d_last), *[t.data_ptr() for t in r.values()])
    _call(_lib.load().sdm_glr_backward, dev, stream, io, grad, workspace=workspace)
    return r


def glr_step(q, k, v, g, state, scale=None, new_state=None, slots=None, out=None, stream=None):
    """One token of B requests: their states updated in place (or into new_state, laid out the same) and the outputs.

    q, k [B, Hk, dk], v [B, H, dv], g [B, H] float32, state [rows, H, dk, dv] float32 contiguous. slots [B] int32 on the device:
    the row of each request (None: row b); rows must be distinct, and a request whose row is outside the
    tensor is left out (output 0). A gate of -infinity starts from nothing, whatever the row held. Returns out [B, H, dv]."""
    fn = "glr_step"
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("%s: q, k are [B, Hk, dk] and v is [B, H, dv]" % fn)
    B, Hk, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    if out is None:
        out = _output_like(stream, v)
    if new_state is None:
        new_state = state
    dev = _same(fn, q, k, v, g, state, new_state, slots, out)
    if k.shape != q.shape or v.shape[0] != B or g.shape != (B, H) or out.shape != v.shape:
        raise ValueError("%s: q %s, k %s, v %s, g %s, out %s do not fit" % (fn, tuple(q.shape), tuple(k.shape), tuple(v.shape), tuple(g.shape),
                                                                          tuple(out.shape)))
    dt = q.dtype
    if k.dtype is not dt or v.dtype is not dt or out.dtype is not dt or g.dtype is not torch.float32:
        raise TypeError("%s: q, k, v and out must have one dtype, and g must be float32" % fn)
    _columns(fn, q, k, v, out)
    _dense(fn, torch.float32, state, new_state)
    if state.shape[1:] != (H, dk, dv) or new_state.shape != state.shape:
        raise ValueError("%s: state is %s, expected [rows, %d, %d, %d]" % (fn, tuple(state.shape), H, dk, dv))
    if slots is not None:
        _dense(fn, torch.int32, slots)
        _shape(fn, "slots", slots, (B,))
    qs, ks, vs, os = q.stride(), k.stride(), v.stride(), out.stride()
    io = _lib.pack_glr_step(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], *g.stride(),
        state.data_ptr(), new_state.data_ptr(), state.shape[0], _ptr(slots), out.data_ptr(), os[0], os[1], B, H, Hk, dk, dv,
        _code(fn, q), float(dk ** -0.5 if scale is None else scale))
    _call(_lib.load().sdm_glr_step, dev, stream, io)
    return out
