"""What is measured of the operators that make a mixer layer with delta-rule heads.

Three operators, each in its plain form (elementary torch operations in 32 bits, rounded once at the end)
and through the package's entry points (`own`):

  gdr    gated delta rule with a dense state per head, forward, backward and for one token:
             u_t = beta_t (v_t - exp(g_t) S_{t-1}^T k_t),   S_t = exp(g_t) S_{t-1} + k_t u_t^T,   o_t = scale S_t^T q_t
  gn     RMS norm of every value head and its gate, y = x / rms(x) w silu(z), forward and backward
  rn     the norms around a block with its residual: h = x + scale (y or y / rms(y) wy), n = h / rms(h) w,
         forward and backward

Sizes are the package's workload shapes (streams, tokens, head dims 64 / 120 / 128) with ordinary head
counts and row widths.
"""

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One training step's mixing over 8 streams of 4096 tokens, and its gradients.
        dict(name="gdr_train_fwd", op="gdr_fwd", B=8, T=4096, H=16, Hk=16, dk=128, dv=128, dtype="bf16", ragged=False, state=False),
        dict(name="gdr_train_bwd", op="gdr_bwd", B=8, T=4096, H=16, Hk=16, dk=128, dv=128, dtype="bf16", ragged=False, state=False),
        # A long prompt of one request that continues a state: little to run side by side but the time axis.
        dict(name="gdr_prefill_long", op="gdr_fwd", B=1, T=16384, H=8, Hk=4, dk=128, dv=128, dtype="bf16", ragged=False, state=True),
        # Fine-tuning in float32 on ragged rows, four value heads on each query and key head, odd head dims.
        dict(name="gdr_ragged_shared_bwd", op="gdr_bwd", B=4, T=509, H=8, Hk=2, dk=64, dv=120, dtype="f32", ragged=True, state=True),
        # One new token: of a single request, where the call's latency counts, and of a full batch.
        dict(name="gdr_token_one", op="gdr_step", B=1, H=4, Hk=4, dk=64, dv=64, dtype="bf16"),
        dict(name="gdr_token_batch", op="gdr_step", B=256, H=16, Hk=16, dk=128, dv=128, dtype="bf16"),
        # Gated norm of a few new tokens' heads; of a training step's; gradients at an odd head dim and count.
        dict(name="gn_tokens_few", op="gn_fwd", N=8, H=16, D=128, dtype="bf16"),
        dict(name="gn_train_fwd", op="gn_fwd", N=32768, H=16, D=128, dtype="bf16"),
        dict(name="gn_odd_bwd", op="gn_bwd", N=16381, H=16, D=120, dtype="bf16"),
        # Residual and next norm of a few new tokens; a training step's rows with both norms; its gradients.
        dict(name="rn_tokens_few", op="rn_fwd", N=8, D=2048, y_norm=False, scaled=False, dtype="bf16"),
        dict(name="rn_train_fwd", op="rn_fwd", N=32768, D=2048, y_norm=True, scaled=True, dtype="bf16"),
        dict(name="rn_train_bwd", op="rn_bwd", N=16381, D=2048, y_norm=True, scaled=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["gdr_fwd", "gdr_fwd", "gdr_bwd", "gdr_bwd", "gdr_step", "gn_fwd", "gn_bwd", "rn_fwd", "rn_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("gdr_fwd", "gdr_bwd"):
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        H = Hk * rng.choice([1, 1, 2, 4])
        dk, dv = rng.choice([64, 64, 120, 128, 128, rng.randint(9, 128)]), rng.choice([64, 120, 128, 128, rng.randint(9, 128)])
        T = _log(rng, 1, 16384)
        # Float32 rows are twice as wide and their matrix products slower: a quarter of the tokens.
        most = (8 * 4096 * 16 if dtype == "bf16" else 2 * 4096 * 16) // H
        B = _log(rng, 1, max(1, min(64, most // T)))
        T = min(T, most // B)
        return dict(op=op, B=B, T=T, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, ragged=rng.random() < 0.4,
                    state=T < 16 or rng.random() < 0.5)   # from no state, the first token's gate reaches nothing
    if op == "gdr_step":
        Hk = rng.choice([1, 2, 4, 8, 16])
        H = Hk * rng.choice([1, 1, 2])
        dk, dv = rng.choice([64, 120, 128, rng.randint(9, 128)]), rng.choice([64, 120, 128, rng.randint(9, 128)])
        return dict(op=op, B=_log(rng, 1, 256 * 16 // H), H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype)
    if op in ("gn_fwd", "gn_bwd"):
        D = rng.choice([64, 120, 128, 128, rng.randint(9, 256)])
        H = rng.choice([1, 2, 4, 8, 16, 32])
        N = _log(rng, 1, max(1, min(65536, 32768 * 16 * 128 // (H * D) // (1 if dtype == "bf16" else 2))))
        return dict(op=op, N=N, H=H, D=D, dtype=dtype)
    D = rng.choice([256, 512, 1024, 2048, 4096, rng.randint(64, 8192)])
    N = _log(rng, 1, max(1, min(65536, 32768 * 2048 // D // (1 if dtype == "bf16" else 2))))
    return dict(op=op, N=N, D=D, y_norm=rng.random() < 0.5, scaled=rng.random() < 0.5, dtype=dtype)


def _lens(case):
    """Tokens of each row: all of them, or a ragged batch (the first row full, the others down to half)."""
    B, T = case["B"], case["T"]
    return [T - (i * 37) % (T // 2 + 1) for i in range(B)] if case["ragged"] else [T] * B


def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("gdr_fwd", "gdr_bwd"):
        n, H, Hk, dk, dv = sum(_lens(case)), case["H"], case["Hk"], case["dk"], case["dv"]
        st = case["B"] * H * dk * dv * 4
        one = n * (2 * Hk * dk + H * dv) * es + n * H * 8      # q, k, v, g and beta
        rows = n * H * dv * es                                  # o, or its gradient
        if op == "gdr_fwd":   # prediction, update and output of every token
            return dict(bytes=one + rows + st * (1 + case["state"]), flops=6.0 * n * H * dk * dv)
        # The states again (4), then dq, du, two parts of dk, and two updates of the state's gradient.
        return dict(bytes=2 * one + rows + st * (3 if case["state"] else 0), flops=16.0 * n * H * dk * dv)
    if op == "gdr_step":
        B, H, Hk, dk, dv = (case[k] for k in ("B", "H", "Hk", "dk", "dv"))
        return dict(bytes=B * H * dk * dv * 8 + B * (2 * Hk * dk + 2 * H * dv) * es + B * H * 8, flops=7.0 * B * H * dk * dv)
    if op in ("gn_fwd", "gn_bwd"):
        e = case["N"] * case["H"] * case["D"]
        return dict(bytes=(3 if op == "gn_fwd" else 5) * e * es, flops=(10.0 if op == "gn_fwd" else 25.0) * e)
    e = case["N"] * case["D"]
    if op == "rn_fwd":   # x, y; h, n
        return dict(bytes=4 * e * es, flops=(6.0 + 4.0 * case["y_norm"]) * e)
    # Gradients of h and n, h, y (where its norm or its scale needs it); gradients of x and y.
    return dict(bytes=(6 if case["y_norm"] or case["scaled"] else 5) * e * es, flops=(12.0 + 12.0 * case["y_norm"]) * e)


# --------------------------------------------------------------------------------------------- inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, op = _dtype(case), case["op"]

    def rnd(*shape, mul=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(mul)

    def unit(*shape):   # query and key heads come with a norm of one
        x = rnd(*shape)
        return x.mul_(x.square().sum(-1, keepdim=True).rsqrt())

    s = dict(case)
    if op.startswith("gdr"):
        B, H, Hk, dk, dv = (case[k] for k in ("B", "H", "Hk", "dk", "dv"))
        lead = (B,) if op == "gdr_step" else (B, case["T"])
        s["scale"] = dk ** -0.5
        s["q"], s["k"] = unit(*lead, Hk, dk).to(dt), unit(*lead, Hk, dk).to(dt)
        s["v"] = rnd(*lead, H, dv).to(dt)
        s["g"] = torch.nn.functional.logsigmoid(rnd(*lead, H) + 3.0)
        s["beta"] = rnd(*lead, H).sigmoid()
        s["s0"] = rnd(B, H, dk, dv, mul=0.3) if op == "gdr_step" or case["state"] else None
        if op == "gdr_step":
            # The new state goes to a buffer of its own, so that a pass can be repeated from the same state.
            s["s1"], s["o"] = torch.empty_like(s["s0"]), torch.empty_like(s["v"])
            return s
        s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        if op == "gdr_bwd":
            s["do"] = rnd(B, case["T"], H, dv).to(dt)
            s["ds"] = rnd(B, H, dk, dv, mul=0.1) if case["state"] else None
    elif op.startswith("gn"):
        N, H, D = (case[k] for k in ("N", "H", "D"))
        # The mixing's outputs, and gates that are a part of the rows of one projection.
        s["x"] = rnd(N, H, D, mul=0.2).to(dt)
        s["z"] = rnd(N, 2 * H * D).to(dt)[:, H * D:].view(N, H, D)
        s["w"] = 1.0 + rnd(D, mul=0.1)
        if op == "gn_bwd":
            s["d"] = rnd(N, H, D).to(dt)
    else:
        N, D = case["N"], case["D"]
        s["x"], s["y"] = rnd(N, D).to(dt), rnd(N, D, mul=0.5).to(dt)
        s["w"] = 1.0 + rnd(D, mul=0.1)
        s["wy"] = 1.0 + rnd(D, mul=0.1) if case["y_norm"] else None
        s["a"] = 0.3 + rnd(D, mul=0.1) if case["scaled"] else None
        if op == "rn_bwd":
            # h is what the forward pass returned.
            s["h"] = _rn_fwd(s)["h"]
            s["dh"], s["dn"] = rnd(N, D).to(dt), rnd(N, D).to(dt)
    return s


# --------------------------------------------------------------------------------------- plain forms

L = 64


def _chunks(x):
    """[B, H, T, ..] -> [B, H, n, L, ..], zeros behind the last token."""
    T = x.shape[2]
    n = (T + L - 1) // L
    pad = [0, 0] * (x.dim() - 3) + [0, n * L - T]
    return torch.nn.functional.pad(x, pad).unflatten(2, (n, L))


def _decays(g):
    """exp(g_{j+1} + .. + g_i) at [.., i, j] for j <= i, 0 above. The sums are taken per column, so that near steps
    keep their digits."""
    low = torch.ones(L, L, dtype=torch.bool, device=g.device).tril_()
    x = torch.where(low.tril(-1), g[..., :, None].expand(*g.shape, L), 0.0).cumsum(-2)
    return torch.where(low, x, float("-inf")).exp()


def _inverse(A):
    """(1 + A)^-1 of strictly lower triangular matrices, row after row."""
    t = torch.eye(L, device=A.device).expand_as(A).clone()
    for i in range(1, L):
        t[..., i, :i] = -(A[..., i, None, :i] @ t[..., :i, :i])[..., 0, :]
    return t


def _gdr_inputs(s):
    """The inputs as [B, H, T, *] float32, shared heads repeated, tokens past a row's length without effect."""
    r = s["H"] // s["Hk"]
    q, k = (s[n].float().repeat_interleave(r, 2).transpose(1, 2) for n in ("q", "k"))
    v, g, b = s["v"].float().transpose(1, 2), s["g"].transpose(1, 2), s["beta"].transpose(1, 2)
    do = s["do"].float().transpose(1, 2) if "do" in s else None
    if s["lens"] is not None:
        live = torch.arange(s["T"], device="cuda") < s["lens"][:, None, None]
        q, k, v = (torch.where(live[..., None], x, 0.0) for x in (q, k, v))
        g, b = torch.where(live, g, 0.0), torch.where(live, b, 0.0)
        do = torch.where(live[..., None], do, 0.0) if do is not None else None
    return q, k, v, g, b, do


def _first(s):
    return torch.zeros((s["B"], s["H"], s["dk"], s["dv"]), device="cuda") if s["s0"] is None else s["s0"]


def _gdr_fwd(s):
    q, k, v, g, b, _ = (None if x is None else _chunks(x) for x in _gdr_inputs(s))
    dec = _decays(g)
    into = g.cumsum(-1).exp()[..., None]                     # what of the state before reaches each token
    outof = dec[..., -1, :, None]                            # what of each token reaches the chunk's end
    t = _inverse(((k @ k.transpose(-1, -2)) * dec * b[..., None]).tril(-1)) * b[..., None, :]
    own_u, from_s = t @ v, t @ (k * into)                    # u = own_u - from_s S
    p = (q @ k.transpose(-1, -2)) * dec
    S = _first(s)
    o = torch.empty_like(v)
    for c in range(v.shape[2]):
        u = own_u[:, :, c] - from_s[:, :, c] @ S
        o[:, :, c] = (q[:, :, c] * into[:, :, c]) @ S + p[:, :, c] @ u
        S = S * into[:, :, c, -1, :, None] + (k[:, :, c] * outof[:, :, c]).transpose(-1, -2) @ u
    o = o.flatten(2, 3)[:, :, :s["T"]] * s["scale"]
    return dict(o=o.transpose(1, 2).to(_dtype(s)), state=S)


def _gdr_bwd(s):
    q, k, v, g, b, do = (_chunks(x) for x in _gdr_inputs(s))
    B, H, T, Hk, dt, n = s["B"], s["H"], s["T"], s["Hk"], _dtype(s), v.shape[2]
    do = do * s["scale"]
    tr = lambda x: x.transpose(-1, -2)  # noqa: E731
    dec = _decays(g)
    into, outof, bb = g.cumsum(-1).exp()[..., None], dec[..., -1, :, None], b[..., None]
    near = ((k @ tr(k)) * dec).tril(-1)
    t = _inverse(near * bb)
    p = (q @ tr(k)) * dec
    # The states before every chunk and the rows u again.
    own_u, from_s = (t * tr(bb)) @ v, (t * tr(bb)) @ (k * into)
    S = _first(s)
    states, u = [], torch.empty_like(v)
    for c in range(n):
        states.append(S)
        u[:, :, c] = own_u[:, :, c] - from_s[:, :, c] @ S
        S = S * into[:, :, c, -1, :, None] + tr(k[:, :, c] * outof[:, :, c]) @ u[:, :, c]
    # Back in time: the gradient of the state behind every chunk, and of the rows u.
    R = torch.zeros_like(S) if s["ds"] is None else s["ds"]
    grads, du = [None] * n, torch.empty_like(v)
    last, R_end, end = S, R, v.new_zeros((B, H, n))
    pd = tr(p) @ do
    for c in range(n - 1, -1, -1):
        grads[c] = R
        end[:, :, c] = (R * (states[c + 1] if c + 1 < n else last)).sum((-1, -2))
        du[:, :, c] = tr(t[:, :, c]) @ ((k[:, :, c] * outof[:, :, c]) @ R + pd[:, :, c])
        R = (R * into[:, :, c, -1, :, None] + tr(q[:, :, c] * into[:, :, c]) @ do[:, :, c]
             - tr(k[:, :, c] * into[:, :, c]) @ (bb[:, :, c] * du[:, :, c]))
    S, G = torch.stack(states, 2), torch.stack(grads, 2)
    dv = bb * du
    pred = into * (k @ S) + near @ u
    dbeta = (du * (v - pred)).sum(-1)
    dq = into * (do @ tr(S)) + ((do @ tr(u)) * dec) @ k
    cross = ((dv @ tr(u)) * dec).tril(-1)
    dk = outof * (u @ tr(G)) + tr((do @ tr(u)) * dec) @ q - into * (dv @ tr(S)) - (cross + tr(cross)) @ k
    # A gate scales everything that reaches its token or a later one from an earlier one.
    dg = ((q * dq).sum(-1) - (v * dv).sum(-1)).flip(-1).cumsum(-1).flip(-1) + end[..., None]
    rows = lambda x: x.flatten(2, 3)[:, :, :T]  # noqa: E731
    dq, dk, dv, dg, dbeta = (rows(x) for x in (dq * 1.0, dk, dv, dg, dbeta))
    if s["s0"] is None:
        dg[:, :, 0] = 0.0
    if s["lens"] is not None:
        live = torch.arange(T, device="cuda") < s["lens"][:, None, None]
        dg, dbeta = torch.where(live, dg, 0.0), torch.where(live, dbeta, 0.0)
        dq, dk, dv = (torch.where(live[..., None], x, 0.0) for x in (dq, dk, dv))
    fold = lambda x: x.reshape(B, Hk, H // Hk, T, -1).sum(2).transpose(1, 2).to(dt)  # noqa: E731
    out = dict(dq=fold(dq), dk=fold(dk), dv=dv.transpose(1, 2).to(dt), dg=dg.transpose(1, 2).contiguous(),
               dbeta=dbeta.transpose(1, 2).contiguous())
    if s["s0"] is not None:
        out["dstate"] = R
    return out


def _gdr_step(s):
    r = s["H"] // s["Hk"]
    q, k = (s[n].float().repeat_interleave(r, 1)[..., None] for n in ("q", "k"))
    S = s["s0"] * s["g"].exp()[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (S * k).sum(-2))
    S = S + k * u[..., None, :]
    return dict(o=((S * q).sum(-2) * s["scale"]).to(_dtype(s)), state=S)


def _rms(x):
    return (x.square().mean(-1, keepdim=True) + EPS).rsqrt()


def _norm_grad(d, x, w):
    """Gradients of x and w of y = x / rms(x) w, from d of y."""
    r = _rms(x)
    n, dn = x * r, d * w
    return (dn - n * (dn * n).mean(-1, keepdim=True)) * r, (d * n).flatten(0, -2).sum(0)


def _gn_fwd(s):
    x, z = s["x"].float(), s["z"].float()
    return dict(y=(x * _rms(x) * s["w"] * (z * z.sigmoid())).to(_dtype(s)))


def _gn_bwd(s):
    x, z, d = (s[n].float() for n in ("x", "z", "d"))
    sg = z.sigmoid()
    dx, dw = _norm_grad(d * (z * sg), x, s["w"])
    dz = d * (x * _rms(x) * s["w"]) * (sg * (1.0 + z * (1.0 - sg)))
    return dict(dx=dx.to(_dtype(s)), dz=dz.to(_dtype(s)), dw=dw)


def _rn_fwd(s):
    x, y = s["x"].float(), s["y"].float()
    if s["y_norm"]:
        y = y * _rms(y) * s["wy"]
    h = (x + (y if s["a"] is None else s["a"] * y)).to(_dtype(s))
    f = h.float()
    return dict(h=h, n=(f * _rms(f) * s["w"]).to(_dtype(s)))


def _rn_bwd(s):
    h, y, dh, dn = (s[n].float() for n in ("h", "y", "dh", "dn"))
    dx, dw = _norm_grad(dn, h, s["w"])
    dx = dh + dx
    out = dict(dx=dx.to(_dtype(s)), dw=dw)
    if s["scaled"]:
        out["da"] = (dx * (y * _rms(y) * s["wy"] if s["y_norm"] else y)).sum(0)
    dy = dx * s["a"] if s["scaled"] else dx
    if s["y_norm"]:
        dy, out["dwy"] = _norm_grad(dy, y, s["wy"])
    out["dy"] = dy.to(_dtype(s))
    return out


# ------------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if not own:
        return dict(gdr_fwd=_gdr_fwd, gdr_bwd=_gdr_bwd, gdr_step=_gdr_step, gn_fwd=_gn_fwd, gn_bwd=_gn_bwd, rn_fwd=_rn_fwd,
                    rn_bwd=_rn_bwd)[op](s)
    import sparse_delta_memory_amd as sdm

    if op == "gdr_fwd":
        o, last = sdm.gdr_forward(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], state=s["s0"], lens=s["lens"])
        return dict(o=o, state=last)
    if op == "gdr_bwd":
        r = sdm.gdr_backward(s["do"], s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], state=s["s0"], d_last=s["ds"],
                             lens=s["lens"])
        return {k: r[k] for k in ("dq", "dk", "dv", "dg", "dbeta") + (("dstate",) if s["s0"] is not None else ())}
    if op == "gdr_step":
        sdm.gdr_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["s0"], scale=s["scale"], new_state=s["s1"], out=s["o"])
        return dict(o=s["o"], state=s["s1"])
    if op == "gn_fwd":
        return dict(y=sdm.gate_norm(s["x"], s["z"], s["w"], eps=EPS))
    if op == "gn_bwd":
        return sdm.gate_norm_backward(s["d"], s["x"], s["z"], s["w"], eps=EPS)
    more = dict(scale=s["a"], norm_y=s["y_norm"], y_weight=s["wy"], eps=EPS)
    if op == "rn_fwd":
        h, n = sdm.residual_norm(s["x"], s["y"], s["w"], **more)
        return dict(h=h, n=n)
    r = sdm.residual_norm_backward(s["dh"], s["dn"], s["h"], s["y"], s["w"], **more)
    out = dict(dx=r["dx"], dw=r["dw"])
    if s["scaled"]:
        out["da"] = r["dscale"]
    if s["y_norm"]:
        out["dwy"] = r["dwy"]
    out["dy"] = r["dy"]
    return out


# ------------------------------------------------------------------------------- the values in 64 bits

def exact(case, seed):
    """From the definitions, in 64 bits: the rule token by token, its gradients by going back through the tokens, the
    norms with their gradients written out per row."""
    s = prepare(case, seed)
    op, f8 = case["op"], torch.float64

    if op.startswith("gdr"):
        B, H, Hk, dk, dv = (case[n] for n in ("B", "H", "Hk", "dk", "dv"))
        head = torch.arange(H, device="cuda") // (H // Hk)
        if op == "gdr_step":
            q, k, v = s["q"].to(f8)[:, head], s["k"].to(f8)[:, head], s["v"].to(f8)
            S = torch.exp(s["g"].to(f8))[:, :, None, None] * s["s0"].to(f8)
            miss = v - (k[:, :, None, :] @ S)[:, :, 0]
            S = S + k[:, :, :, None] * (s["beta"].to(f8)[:, :, None] * miss)[:, :, None, :]
            return dict(o=(q[:, :, None, :] @ S)[:, :, 0] * s["scale"], state=S)
        T = case["T"]
        alive = torch.arange(T, device="cuda")[None] < torch.tensor(_lens(case), device="cuda")[:, None]
        on = alive.to(f8)[:, :, None, None]
        q, k, v = s["q"].to(f8)[:, :, head], s["k"].to(f8)[:, :, head] * on, s["v"].to(f8) * on
        a = torch.exp(torch.where(alive[..., None], s["g"], 0.0).to(f8))[..., None, None]
        beta = s["beta"].to(f8)[..., None]
        S = torch.zeros(B, H, dk, dv, dtype=f8, device="cuda") if s["s0"] is None else s["s0"].to(f8).clone()

        def onward(S, t):
            """The state after token t, in place; the token's miss v - S^T k before it."""
            S.mul_(a[:, t])
            miss = v[:, t] - (k[:, t, :, None] @ S)[:, :, 0]
            S.addcmul_(k[:, t, :, :, None], (beta[:, t] * miss)[:, :, None])
            return miss

        if op == "gdr_fwd":
            o = torch.empty(B, T, H, dv, dtype=f8, device="cuda")
            for t in range(T):
                onward(S, t)
                o[:, t] = (q[:, t, :, None] @ S)[:, :, 0]
            return dict(o=o * on * s["scale"], state=S)
        do = s["do"].to(f8) * on * s["scale"]
        # The states before every 128th token, and those between again when the way back comes to them.
        step = 128
        marks = []
        for t in range(T):
            if t % step == 0:
                marks.append(S.clone())
            onward(S, t)
        R = torch.zeros_like(S) if s["ds"] is None else s["ds"].to(f8).clone()
        dq, dkk = (torch.empty(B, T, H, dk, dtype=f8, device="cuda") for _ in range(2))
        dvv = torch.empty(B, T, H, dv, dtype=f8, device="cuda")
        dg, db = (torch.empty(B, T, H, dtype=f8, device="cuda") for _ in range(2))
        for first in range((T - 1) // step * step, -1, -step):
            S = marks.pop()
            between, misses = [], []
            for t in range(first, min(T, first + step)):
                between.append(S.clone())
                misses.append(onward(S, t))
            between.append(S)
            for t in range(min(T, first + step) - 1, first - 1, -1):
                before, after, miss = between[t - first], between[t - first + 1], misses[t - first]
                dq[:, t] = (after @ do[:, t, :, :, None])[..., 0]
                R.addcmul_(q[:, t, :, :, None], do[:, t, :, None])
                du = (k[:, t, :, None] @ R)[:, :, 0]
                d = beta[:, t] * du
                db[:, t] = (du * miss).sum(-1)
                dvv[:, t] = d
                dkk[:, t] = (R @ (beta[:, t] * miss)[..., None])[..., 0] - ((before * a[:, t]) @ d[..., None])[..., 0]
                R.addcmul_(k[:, t, :, :, None], d[:, :, None], value=-1.0).mul_(a[:, t])
                dg[:, t] = (R * before).sum((-1, -2))
        live = on[..., 0]
        fold = lambda x: (x * on).view(B, T, Hk, H // Hk, dk).sum(3)  # noqa: E731
        out = dict(dq=fold(dq), dk=fold(dkk), dv=dvv * on, dg=dg * live, dbeta=db * live)
        if s["s0"] is not None:
            out["dstate"] = R
        return out

    if op.startswith("gn"):
        x, z, w = s["x"].to(f8), s["z"].to(f8), s["w"].to(f8)
        D = x.shape[-1]
        rms = torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS)
        gate = z / (1.0 + torch.exp(-z))
        if op == "gn_fwd":
            return dict(y=x / rms * w * gate)
        d = s["d"].to(f8)
        slope = (1.0 + torch.exp(-z) + z * torch.exp(-z)) / (1.0 + torch.exp(-z)) ** 2
        dy = d * gate
        inner = (dy * w * x).sum(-1, keepdim=True) / D
        return dict(dx=dy * w / rms - x * inner / rms ** 3, dz=d * slope * w * x / rms, dw=(dy * x / rms).sum((0, 1)))

    x, y, w = s["x"].to(f8), s["y"].to(f8), s["w"].to(f8)
    D = x.shape[-1]
    ry = torch.sqrt((y * y).sum(-1, keepdim=True) / D + EPS)
    part = y / ry * s["wy"].to(f8) if s["y_norm"] else y
    a = s["a"].to(f8) if s["scaled"] else torch.ones(D, dtype=f8, device="cuda")
    if op == "rn_fwd":
        h = x + a * part
        f = h.to(_dtype(s)).to(f8)   # the norm is that of h as it is returned
        return dict(h=h, n=f / torch.sqrt((f * f).sum(-1, keepdim=True) / D + EPS) * w)
    h, dh, dn = s["h"].to(f8), s["dh"].to(f8), s["dn"].to(f8)
    rh = torch.sqrt((h * h).sum(-1, keepdim=True) / D + EPS)
    dx = dh + dn * w / rh - h * ((dn * w * h).sum(-1, keepdim=True) / D) / rh ** 3
    out = dict(dx=dx, dw=(dn * h / rh).sum(0))
    if s["scaled"]:
        out["da"] = (dx * part).sum(0)
    dy = dx * a
    if s["y_norm"]:
        wy = s["wy"].to(f8)
        out["dwy"] = (dy * y / ry).sum(0)
        dy = dy * wy / ry - y * ((dy * wy * y).sum(-1, keepdim=True) / D) / ry ** 3
    out["dy"] = dy
    return out
