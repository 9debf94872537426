"""What is measured of the mixer operators that stand beside the sparse bank.

Three operators of one mixer layer, each in its plain form (elementary torch operations in 32 bits,
rounded once at the end) and through the package's entry points (`own`):

  glr    gated linear recurrence with a dense state per head, forward, backward and for one token:
             S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = scale S_t^T q_t
  nr     RMS norm of every query and key head and the rotation by its position, forward and backward
  slot   slot ids and weights of a bank of n1 x n2 slots from two rows of scores per token: the K best
         of each row, the K best of their pair sums, and the softmax of those, forward and backward

Sizes are the package's workload shapes (streams, tokens, head dims 64 / 120 / 128, 4..32 slots per token,
banks of 4096 .. 4194304 slots) with ordinary head counts.
"""

import torch

own = False


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One training step's mixing over 8 streams of 4096 tokens, and its gradients.
        dict(name="glr_train_fwd", op="glr_fwd", B=8, T=4096, H=16, Hk=16, dk=128, dv=128, dtype="bf16", ragged=False, state=False),
        dict(name="glr_train_bwd", op="glr_bwd", B=8, T=4096, H=16, Hk=16, dk=128, dv=128, dtype="bf16", ragged=False, state=False),
        # A long prompt of one request that continues a state: little to run side by side but the time axis.
        dict(name="glr_prefill_long", op="glr_fwd", B=1, T=16384, H=8, Hk=8, dk=128, dv=128, dtype="bf16", ragged=False, state=True),
        # Fine-tuning in float32 on ragged rows, four value heads on each query and key head, odd head dims.
        dict(name="glr_ragged_shared_bwd", op="glr_bwd", B=4, T=509, H=8, Hk=2, dk=64, dv=120, dtype="f32", ragged=True, state=True),
        # One new token: of a single request, where the call's latency counts, and of a full batch.
        dict(name="glr_token_one", op="glr_step", B=1, H=4, Hk=4, dk=64, dv=64, dtype="bf16"),
        dict(name="glr_token_batch", op="glr_step", B=256, H=16, Hk=16, dk=128, dv=128, dtype="bf16"),
        # Heads of a few new tokens; of a training step's tokens (16 query and 4 key heads).
        dict(name="nr_tokens_few", op="nr_fwd", N=8, Hq=16, Hk=4, D=128, rot=128, inter=False, dtype="bf16"),
        dict(name="nr_train_fwd", op="nr_fwd", N=32768, Hq=16, Hk=4, D=128, rot=128, inter=False, dtype="bf16"),
        # Gradients, rotation of part of the head in the interleaved layout, an odd count of tokens.
        dict(name="nr_part_bwd", op="nr_bwd", N=16381, Hq=16, Hk=4, D=128, rot=64, inter=True, dtype="bf16"),
        # Slots of a few tokens in a small bank; of a step's tokens in the largest bank; gradients.
        dict(name="slot_few", op="slot_fwd", N=64, n1=64, n2=64, K=4, dtype="f32"),
        dict(name="slot_large", op="slot_fwd", N=65536, n1=2048, n2=2048, K=32, dtype="bf16"),
        dict(name="slot_bwd", op="slot_bwd", N=32768, n1=512, n2=512, K=32, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["glr_fwd", "glr_fwd", "glr_bwd", "glr_bwd", "glr_step", "nr_fwd", "nr_bwd", "slot_fwd", "slot_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("glr_fwd", "glr_bwd"):
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
    if op == "glr_step":
        Hk = rng.choice([1, 2, 4, 8, 16])
        H = Hk * rng.choice([1, 1, 2])
        dk, dv = rng.choice([64, 120, 128, rng.randint(9, 128)]), rng.choice([64, 120, 128, rng.randint(9, 128)])
        return dict(op=op, B=_log(rng, 1, 256 * 16 // H), H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype)
    if op in ("nr_fwd", "nr_bwd"):
        D = rng.choice([64, 120, 128, 128, 2 * rng.randint(8, 128)])
        rot = rng.choice([D, D, D // 2 // 2 * 2, 0])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4, 8])
        N = _log(rng, 1, max(1, min(65536, 32768 * 20 * 128 // ((Hq + Hk) * D) // (1 if dtype == "bf16" else 2))))
        return dict(op=op, N=N, Hq=Hq, Hk=Hk, D=D, rot=rot, inter=rng.random() < 0.5, dtype=dtype)
    n1 = rng.choice([64, 128, 256, 512, 1024, 2048, rng.randint(16, 2048)])
    n2 = rng.choice([n1, n1, rng.randint(16, 2048)])
    K = rng.choice([4, 8, 16, 32, rng.randint(2, 64)])
    N = _log(rng, 1, max(1, min(65536, 65536 * 4096 // (n1 + n2) // (1 if dtype == "bf16" else 2))))
    return dict(op=op, N=N, n1=n1, n2=n2, K=K, dtype=dtype)


def _lens(case):
    """Tokens of each row: all of them, or a ragged batch (the first row full, the others down to half)."""
    B, T = case["B"], case["T"]
    return [T - (i * 37) % (T // 2 + 1) for i in range(B)] if case["ragged"] else [T] * B


def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("glr_fwd", "glr_bwd"):
        n, H, Hk, dk, dv = sum(_lens(case)), case["H"], case["Hk"], case["dk"], case["dv"]
        st = case["B"] * H * dk * dv * 4
        one = n * (2 * Hk * dk + H * dv) * es + n * H * 4      # q, k, v and g
        rows = n * H * dv * es                                  # o, or its gradient
        if op == "glr_fwd":
            return dict(bytes=one + rows + st * (1 + case["state"]), flops=4.0 * n * H * dk * dv)
        return dict(bytes=2 * one + rows + st * (3 if case["state"] else 0), flops=10.0 * n * H * dk * dv)
    if op == "glr_step":
        B, H, Hk, dk, dv = (case[k] for k in ("B", "H", "Hk", "dk", "dv"))
        return dict(bytes=B * H * dk * dv * 8 + B * (2 * Hk * dk + 2 * H * dv) * es + B * H * 4, flops=5.0 * B * H * dk * dv)
    if op in ("nr_fwd", "nr_bwd"):
        e = case["N"] * (case["Hq"] + case["Hk"]) * case["D"]
        tab = min(case["N"], 4096) * case["rot"] * 4 + case["N"] * 4      # rows of at most 4096 positions
        return dict(bytes=(2 if op == "nr_fwd" else 3) * e * es + tab, flops=(6.0 if op == "nr_fwd" else 14.0) * e)
    N, n, K = case["N"], case["n1"] + case["n2"], case["K"]
    if op == "slot_fwd":
        return dict(bytes=N * n * es + N * K * 8, flops=1.0 * N * n)
    return dict(bytes=N * n * es + N * K * (8 + 2 * es), flops=1.0 * N * n)


# --------------------------------------------------------------------------------------------- inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _table(rows, rot, base=10000.0):
    """cos | sin of every position's angles, [rows, rot] float32."""
    if rot == 0:
        return torch.zeros((rows, 0), device="cuda")
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, op = _dtype(case), case["op"]

    def rnd(*shape, mul=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(mul)

    s = dict(case)
    if op.startswith("glr"):
        B, H, Hk, dk, dv = (case[k] for k in ("B", "H", "Hk", "dk", "dv"))
        lead = (B,) if op == "glr_step" else (B, case["T"])
        s["scale"] = dk ** -0.5
        s["q"], s["k"] = rnd(*lead, Hk, dk).to(dt), rnd(*lead, Hk, dk, mul=dk ** -0.5).to(dt)
        s["v"] = rnd(*lead, H, dv).to(dt)
        s["g"] = torch.nn.functional.logsigmoid(rnd(*lead, H) + 2.0)
        s["s0"] = rnd(B, H, dk, dv, mul=0.3) if op == "glr_step" or case["state"] else None
        if op == "glr_step":
            # The new state goes to a buffer of its own, so that a pass can be repeated from the same state.
            s["s1"], s["o"] = torch.empty_like(s["s0"]), torch.empty_like(s["v"])
            return s
        s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        if op == "glr_bwd":
            s["do"] = rnd(B, case["T"], H, dv).to(dt)
            s["ds"] = rnd(B, H, dk, dv, mul=0.1) if case["state"] else None
    elif op.startswith("nr"):
        N, Hq, Hk, D, rot = (case[k] for k in ("N", "Hq", "Hk", "D", "rot"))
        # Query and key heads are views of one projection's rows, the value heads behind them.
        rows = rnd(N, (Hq + 2 * Hk) * D).to(dt)
        s["q"], s["k"] = rows[:, :Hq * D].view(N, Hq, D), rows[:, Hq * D:(Hq + Hk) * D].view(N, Hk, D)
        s["wq"], s["wk"] = 1.0 + rnd(D, mul=0.1), 1.0 + rnd(D, mul=0.1)
        s["pos"] = torch.randint(0, 16384, (N,), generator=gen, device="cuda", dtype=torch.int32)
        if N >= 4096:   # rows of whole sequences
            s["pos"] = (torch.arange(N, device="cuda", dtype=torch.int32) + s["pos"][:1]) % 4096
        s["table"] = _table(16384, rot)
        if op == "nr_bwd":
            s["dq"], s["dk"] = rnd(N, Hq, D).to(dt), rnd(N, Hk, D).to(dt)
    else:
        N, n1, n2, K = (case[k] for k in ("N", "n1", "n2", "K"))
        s["a"], s["b"] = rnd(N, n1).to(dt), rnd(N, n2).to(dt)
        s["scale"] = 1.0
        if op == "slot_bwd":
            s["idx"] = _slots(s["a"], s["b"], K)[0].to(torch.int32)
            s["dval"] = rnd(N, K)
    return s


# --------------------------------------------------------------------------------------- plain forms

def _decays(g):
    """exp of the sums of gates after each earlier step: [..., n] -> [..., n + 1, n + 1], where [i, j] holds
    exp(g_{j+1} + .. + g_i) for j <= i (index 0 is the start) and 0 above. The sums are taken per column, so
    that near steps keep their digits."""
    n = g.shape[-1] + 1
    x = torch.cat([g.new_zeros(g.shape[:-1] + (1,)), g], -1)
    low = torch.ones(n, n, dtype=torch.bool, device=g.device).tril_()
    x = torch.where(low.tril(-1), x[..., :, None].expand(*x.shape, n), 0.0).cumsum(-2)
    return torch.where(low, x, float("-inf")).exp()


def _mix(q, k, v, g, s0):
    """o [B, H, T, dv] and the last state of the recurrence over time, in chunks of 64 tokens: the tokens of a
    chunk with each other, the chunks' contributions to the state, and every chunk's state from those.
    q, k [B, H, T, dk], v [B, H, T, dv], g [B, H, T] float32, s0 [B, H, dk, dv] or None."""
    B, H, T, dk = q.shape
    L, n = 64, (T + 63) // 64
    pad = n * L - T
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)).view(B, H, n, L, x.shape[-1]) for x in (q, k, v))
    g = torch.nn.functional.pad(g, (0, pad)).view(B, H, n, L)
    dec = _decays(g)                                                      # [B, H, n, L + 1, L + 1]
    o = ((q @ k.transpose(-1, -2)) * dec[..., 1:, 1:]) @ v
    add = (k * dec[..., -1, 1:, None]).transpose(-1, -2) @ v              # what a chunk leaves in the state
    s0 = add.new_zeros((B, H, dk, v.shape[-1])) if s0 is None else s0
    add = torch.cat([s0[:, :, None], add], 2).view(B, H, n + 1, -1)
    states = (_decays(g.sum(-1)) @ add).view(B, H, n + 1, dk, -1)         # before each chunk, and after the last
    o = o + dec[..., 1:, 0, None] * (q @ states[:, :, :-1])
    return o.reshape(B, H, n * L, -1)[:, :, :T], states[:, :, -1]


def _glr_inputs(s):
    """The inputs as [B, H, T, *] float32, shared heads repeated, tokens past a row's length without effect."""
    r = s["H"] // s["Hk"]
    q, k = (s[n].float().repeat_interleave(r, 2).transpose(1, 2) for n in ("q", "k"))
    v, g = s["v"].float().transpose(1, 2), s["g"].transpose(1, 2)
    do = s["do"].float().transpose(1, 2) if "do" in s else None
    if s["lens"] is not None:
        live = torch.arange(s["T"], device="cuda") < s["lens"][:, None, None]
        q, k, v = (torch.where(live[..., None], x, 0.0) for x in (q, k, v))
        g = torch.where(live, g, 0.0)
        do = torch.where(live[..., None], do, 0.0) if do is not None else None
    return q, k, v, g, do


def _glr_fwd(s):
    q, k, v, g, _ = _glr_inputs(s)
    o, last = _mix(q, k, v, g, s["s0"])
    return dict(o=(o * s["scale"]).transpose(1, 2).to(_dtype(s)), state=last)


def _glr_bwd(s):
    q, k, v, g, do = _glr_inputs(s)
    B, H, T, Hk, dt = s["B"], s["H"], s["T"], s["Hk"], _dtype(s)
    do = do * s["scale"]
    # dq_t = S_t do_t: the recurrence with keys and values exchanged. dk and dv: the same recurrences back in
    # time on the state's gradient, whose step t decays by the next token's gate.
    dq = _mix(do, v, k, g, None if s["s0"] is None else s["s0"].transpose(-1, -2))[0]
    back = torch.cat([torch.zeros_like(g[..., :1]), g.flip(-1)[..., :-1]], -1)
    qf, kf, vf, df = (x.flip(2) for x in (q, k, v, do))
    dk = _mix(vf, df, qf, back, None if s["ds"] is None else s["ds"].transpose(-1, -2))[0].flip(2)
    dv, first = _mix(kf, qf, df, back, s["ds"])
    dv = dv.flip(2)
    # A gate scales everything that reaches a later token from an earlier one.
    dg = ((q * dq).sum(-1) - (k * dk).sum(-1)).flip(-1).cumsum(-1).flip(-1)
    if s["ds"] is not None:
        dg = dg + (_mix(q, k, v, g, s["s0"])[1] * s["ds"]).sum((-1, -2))[..., None]
        if s["lens"] is not None:
            dg = torch.where(torch.arange(T, device="cuda") < s["lens"][:, None, None], dg, 0.0)
    fold = lambda x: x.view(B, Hk, H // Hk, T, -1).sum(2).transpose(1, 2).to(dt)  # noqa: E731
    out = dict(dq=fold(dq), dk=fold(dk), dv=dv.transpose(1, 2).to(dt), dg=dg.transpose(1, 2).contiguous())
    if s["s0"] is not None:
        out["dstate"] = first * g[..., 0, None, None].exp()
    return out


def _glr_step(s):
    r = s["H"] // s["Hk"]
    q, k = (s[n].float().repeat_interleave(r, 1) for n in ("q", "k"))
    new = s["s0"] * s["g"].exp()[..., None, None] + k[..., :, None] * s["v"].float()[..., None, :]
    return dict(o=((new * q[..., :, None]).sum(-2) * s["scale"]).to(_dtype(s)), state=new)


def _turn(y, table, pos, inter):
    """The rotation of the first rot columns of y [N, H, D] by its tokens' angles."""
    rot = table.shape[1]
    if rot == 0:
        return y
    c, n = (t[:, None, :] for t in table[pos.long()].chunk(2, 1))
    x = y[..., :rot]
    x1, x2 = (x[..., 0::2], x[..., 1::2]) if inter else x.chunk(2, -1)
    p = (x1 * c - x2 * n, x2 * c + x1 * n)
    x = torch.stack(p, -1).flatten(-2) if inter else torch.cat(p, -1)
    return torch.cat([x, y[..., rot:]], -1)


EPS = 1e-6


def _nr_fwd(s):
    def one(x, w):
        x = x.float()
        return _turn(x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w, s["table"], s["pos"], s["inter"]).to(_dtype(s))
    return dict(q=one(s["q"], s["wq"]), k=one(s["k"], s["wk"]))


def _nr_bwd(s):
    back = torch.cat([s["table"][:, :s["rot"] // 2], -s["table"][:, s["rot"] // 2:]], 1)   # the rotation's transpose

    def one(x, w, d):
        x, d = x.float(), _turn(d.float(), back, s["pos"], s["inter"])
        r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        n = x * r
        dn = d * w
        return ((dn - n * (dn * n).mean(-1, keepdim=True)) * r).to(_dtype(s)), (d * n).sum((0, 1))
    dq, dwq = one(s["q"], s["wq"], s["dq"])
    dk, dwk = one(s["k"], s["wk"], s["dk"])
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


def _best(x, K):
    """The K best of each row and their places, the best first; of equal ones the lowest place first."""
    v, i = torch.sort(x, dim=-1, descending=True, stable=True)
    return v[:, :K], i[:, :K]


def _slots(a, b, K):
    """(ids, sums) of the K best pairs, the best first, from the K best of each row (of equal sums, the pair
    with the better first half, then the better second half)."""
    a, b = a.float() + 0.0, b.float() + 0.0
    va, ia = _best(a, min(K, a.shape[1]))
    vb, ib = _best(b, min(K, b.shape[1]))
    kb = vb.shape[1]
    v, p = _best((va[:, :, None] + vb[:, None, :]).flatten(1), K)
    return ia.gather(1, p // kb) * b.shape[1] + ib.gather(1, p % kb), v


def _slot_fwd(s):
    idx, v = _slots(s["a"], s["b"], s["K"])
    e = ((v - v[:, :1]) * s["scale"]).exp()
    return dict(idx=idx.to(torch.int32), val=e / e.sum(-1, keepdim=True))


def _slot_bwd(s):
    a, b, i = s["a"].float(), s["b"].float(), s["idx"].long()
    i, j = i // s["n2"], i % s["n2"]
    v = a.gather(1, i) + b.gather(1, j)
    e = ((v - v.amax(-1, keepdim=True)) * s["scale"]).exp()
    p = e / e.sum(-1, keepdim=True)
    d = p * (s["dval"] - (p * s["dval"]).sum(-1, keepdim=True)) * s["scale"]
    return dict(da=torch.zeros_like(a).scatter_add_(1, i, d).to(_dtype(s)), db=torch.zeros_like(b).scatter_add_(1, j, d).to(_dtype(s)))


# ------------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if not own:
        return dict(glr_fwd=_glr_fwd, glr_bwd=_glr_bwd, glr_step=_glr_step, nr_fwd=_nr_fwd, nr_bwd=_nr_bwd,
                    slot_fwd=_slot_fwd, slot_bwd=_slot_bwd)[op](s)
    import sparse_delta_memory_amd as sdm

    if op == "glr_fwd":
        o, last = sdm.glr_forward(s["q"], s["k"], s["v"], s["g"], scale=s["scale"], state=s["s0"], lens=s["lens"])
        return dict(o=o, state=last)
    if op == "glr_bwd":
        r = sdm.glr_backward(s["do"], s["q"], s["k"], s["v"], s["g"], scale=s["scale"], state=s["s0"], d_last=s["ds"], lens=s["lens"])
        return {k: r[k] for k in ("dq", "dk", "dv", "dg") + (("dstate",) if s["s0"] is not None else ())}
    if op == "glr_step":
        sdm.glr_step(s["q"], s["k"], s["v"], s["g"], s["s0"], scale=s["scale"], new_state=s["s1"], out=s["o"])
        return dict(o=s["o"], state=s["s1"])
    if op == "nr_fwd":
        q, k = sdm.norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["table"], interleaved=s["inter"], eps=EPS)
        return dict(q=q, k=k)
    if op == "nr_bwd":
        return sdm.norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["table"],
                                      interleaved=s["inter"], eps=EPS)
    if op == "slot_fwd":
        idx, val = sdm.slot_topk(s["a"], s["b"], s["K"], scale=s["scale"])
        return dict(idx=idx, val=val)
    da, db = sdm.slot_topk_backward(s["dval"], s["idx"], s["a"], s["b"], scale=s["scale"])
    return dict(da=da, db=db)


# ------------------------------------------------------------------------------- the values in 64 bits

def exact(case, seed):
    """From the definitions, in 64 bits: the recurrence token by token, the rotation as a complex product, the
    slots from a full ordering of the pairs that can win."""
    s = prepare(case, seed)
    op = case["op"]
    f8 = torch.float64

    if op.startswith("glr"):
        B, H, Hk, dk, dv = (case[n] for n in ("B", "H", "Hk", "dk", "dv"))
        head = torch.arange(H, device="cuda") // (H // Hk)
        if op == "glr_step":
            q, k, v = s["q"].to(f8)[:, head], s["k"].to(f8)[:, head], s["v"].to(f8)
            S = torch.exp(s["g"].to(f8))[:, :, None, None] * s["s0"].to(f8) + k[:, :, :, None] * v[:, :, None, :]
            return dict(o=(q[:, :, :, None] * S).sum(2) * s["scale"], state=S)
        T = case["T"]
        q, k, v = s["q"].to(f8)[:, :, head], s["k"].to(f8)[:, :, head], s["v"].to(f8)
        lens = torch.tensor(_lens(case), device="cuda")
        live = (torch.arange(T, device="cuda")[None] < lens[:, None]).to(f8)[:, :, None, None]
        a = torch.exp(s["g"].to(f8))[..., None, None]
        a = a * live[..., None] + (1.0 - live[..., None])
        k, v = k * live, v * live
        S = torch.zeros(B, H, dk, dv, dtype=f8, device="cuda") if s["s0"] is None else s["s0"].to(f8).clone()
        if op == "glr_fwd":
            o = torch.empty(B, T, H, dv, dtype=f8, device="cuda")
            for t in range(T):
                S.mul_(a[:, t]).addcmul_(k[:, t, :, :, None], v[:, t, :, None, :])
                o[:, t] = (q[:, t, :, None] @ S)[:, :, 0]
            return dict(o=o * live * s["scale"], state=S)
        do = s["do"].to(f8) * live * s["scale"]
        dqh = torch.empty(B, T, H, dk, dtype=f8, device="cuda")
        dkh, dvh = torch.empty_like(dqh), torch.empty(B, T, H, dv, dtype=f8, device="cuda")
        for t in range(T):
            S.mul_(a[:, t]).addcmul_(k[:, t, :, :, None], v[:, t, :, None, :])
            dqh[:, t] = (S @ do[:, t, :, :, None])[..., 0]
        R = torch.zeros_like(S) if s["ds"] is None else s["ds"].to(f8).clone()
        run_ = (S * R).sum((-1, -2))               # everything that passes the end of the row
        dg = torch.empty(B, T, H, dtype=f8, device="cuda")
        for t in range(T - 1, -1, -1):
            R.addcmul_(q[:, t, :, :, None], do[:, t, :, None, :])
            dkh[:, t] = (R @ v[:, t, :, :, None])[..., 0]
            dvh[:, t] = (k[:, t, :, None] @ R)[:, :, 0]
            run_ = run_ + (q[:, t] * dqh[:, t]).sum(-1) - (k[:, t] * dkh[:, t]).sum(-1)
            dg[:, t] = run_
            R.mul_(a[:, t])
        dkh, dvh = dkh * live, dvh * live
        out = dict(dq=dqh.view(B, T, Hk, H // Hk, dk).sum(3), dk=dkh.view(B, T, Hk, H // Hk, dk).sum(3), dv=dvh,
                   dg=dg * live[..., 0])
        if s["s0"] is not None:
            out["dstate"] = R
        return out

    if op.startswith("nr"):
        D, rot = case["D"], case["rot"]
        h = rot // 2
        ang = torch.complex(s["table"][:, :h].to(f8), s["table"][:, h:].to(f8))[s["pos"].long()][:, None]
        lo = torch.arange(h, device="cuda") * (2 if case["inter"] else 1)
        hi = lo + (1 if case["inter"] else h)

        def spin(x, by):
            z = torch.complex(x[..., lo], x[..., hi]) * by
            x = x.clone()
            x[..., lo], x[..., hi] = z.real, z.imag
            return x

        out = {}
        for n in ("q", "k"):
            x, w = s[n].to(f8), s["w" + n].to(f8)
            rms = torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS)
            if op == "nr_fwd":
                out[n] = spin(x / rms * w, ang)
                continue
            d = spin(s["d" + n].to(f8), ang.conj())
            out["dw" + n] = (d * x / rms).sum(0).sum(0)
            d = d * w
            out["d" + n] = d / rms - x * (d * x).sum(-1, keepdim=True) / (D * rms ** 3)
        return out

    N, n2, K = case["N"], case["n2"], case["K"]
    a, b = s["a"].to(f8), s["b"].to(f8)
    if op == "slot_fwd":
        # The sums of any K pairs that win are the K largest sums: their weights need no ids.
        va, vb = torch.topk(a, min(K, case["n1"])).values, torch.topk(b, min(K, n2)).values
        top = torch.topk((va[:, :, None] + vb[:, None, :]).view(N, -1), K).values
        return dict(idx=None, val=torch.softmax(top * s["scale"], -1))
    i = s["idx"].long()
    p = torch.softmax((a.gather(1, i // n2) + b.gather(1, i % n2)) * s["scale"], -1)
    dval = s["dval"].to(f8)
    d = (p * dval - p * (p * dval).sum(-1, keepdim=True)) * s["scale"]
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for m in range(K):      # no two entries of one column share a row
        da.scatter_add_(1, i[:, m:m + 1] // n2, d[:, m:m + 1])
        db.scatter_add_(1, i[:, m:m + 1] % n2, d[:, m:m + 1])
    return dict(da=da, db=db)
