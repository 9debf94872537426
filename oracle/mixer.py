"""float64 oracle of the mixer operators, from their definitions: plain loops over tokens and rows in numpy.

Each function also returns, where a float32 evaluation is compared with it, the magnitude of what it adds
up: the same sums over absolute values, which the tests' bounds are multiples of."""

from __future__ import annotations

import numpy as np


def _live(lens, B, T):
    n = np.full(B, T) if lens is None else np.clip(np.asarray(lens), 0, T)
    return np.arange(T)[None, :] < n[:, None]


def glr_forward(q, k, v, g, scale, state=None, lens=None):
    """(o, last, |o|, |last|): q, k [B, T, Hk, dk], v [B, T, H, dv], g [B, T, H]."""
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    head = np.arange(H) // (H // Hk)
    live = _live(lens, B, T)
    S = np.zeros((B, H, dk, dv)) if state is None else np.array(state, dtype=np.float64)
    M = np.abs(S)
    o, mo = np.zeros((B, T, H, dv)), np.zeros((B, T, H, dv))
    for b in range(B):
        for t in range(T):
            if not live[b, t]:
                continue
            for h in range(H):
                a = np.exp(np.float64(g[b, t, h]))
                kk, qq, vv = (x.astype(np.float64) for x in (k[b, t, head[h]], q[b, t, head[h]], v[b, t, h]))
                # A reset leaves nothing, whatever was there.
                S[b, h] = (a * S[b, h] if a > 0 else 0.0) + np.outer(kk, vv)
                M[b, h] = (a * M[b, h] if a > 0 else 0.0) + np.abs(np.outer(kk, vv))
                o[b, t, h] = scale * (qq @ S[b, h])
                mo[b, t, h] = abs(scale) * (np.abs(qq) @ M[b, h])
    return o, S, mo, M


def glr_backward(d_o, q, k, v, g, scale, state=None, d_last=None, lens=None):
    """Gradients from the chain rule, token by token, dg_t = <exp(g_t) S_{t-1}, R_t>: (grads, magnitudes), dicts of dq, dk,
    dv, dg and dstate. dg's magnitude is that of the sums a chunked evaluation adds up to it,
    sum over s >= t of |q_s| |dq_s| + |k_s| |dk_s|, plus |S_T| |R_T|."""
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    head = np.arange(H) // (H // Hk)
    live = _live(lens, B, T)
    z = lambda *s: np.zeros(s)  # noqa: E731
    r = dict(dq=z(B, T, Hk, dk), dk=z(B, T, Hk, dk), dv=z(B, T, H, dv), dg=z(B, T, H), dstate=z(B, H, dk, dv))
    m = {n: np.zeros_like(x) for n, x in r.items()}
    for b in range(B):
        n = int(live[b].sum())
        for h in range(H):
            S = np.zeros((dk, dv)) if state is None else np.array(state[b, h], dtype=np.float64)
            M = np.abs(S)
            before = []
            part = np.zeros(n)
            for t in range(n):
                a = np.exp(np.float64(g[b, t, h]))
                kk, vv, dd = (x.astype(np.float64) for x in (k[b, t, head[h]], v[b, t, h], d_o[b, t, h]))
                before.append(S)
                S = (a * S if a > 0 else 0.0) + np.outer(kk, vv)
                M = (a * M if a > 0 else 0.0) + np.abs(np.outer(kk, vv))
                x, mx = scale * (S @ dd), abs(scale) * (M @ np.abs(dd))
                r["dq"][b, t, head[h]] += x
                m["dq"][b, t, head[h]] += mx
                part[t] += np.abs(q[b, t, head[h]].astype(np.float64)) @ mx
            R = np.zeros((dk, dv)) if d_last is None else np.array(d_last[b, h], dtype=np.float64)
            N = np.abs(R)
            rest = float((M * N).sum())
            for t in range(n - 1, -1, -1):
                a = np.exp(np.float64(g[b, t, h]))
                kk, vv, qq, dd = (x.astype(np.float64) for x in (k[b, t, head[h]], v[b, t, h], q[b, t, head[h]], d_o[b, t, h]))
                R = R + scale * np.outer(qq, dd)
                N = N + abs(scale) * np.abs(np.outer(qq, dd))
                r["dk"][b, t, head[h]] += R @ vv
                m["dk"][b, t, head[h]] += N @ np.abs(vv)
                part[t] += np.abs(kk) @ (N @ np.abs(vv))
                r["dv"][b, t, h] = kk @ R
                m["dv"][b, t, h] = np.abs(kk) @ N
                r["dg"][b, t, h] = a * (before[t] * R).sum() if a > 0 else 0.0
                rest += part[t]
                m["dg"][b, t, h] = rest
                R, N = (a * R, a * N) if a > 0 else (np.zeros_like(R), np.zeros_like(N))
            r["dstate"][b, h], m["dstate"][b, h] = R, N
    return r, m


def _angles(table, pos, h):
    p = np.clip(np.asarray(pos), 0, table.shape[0] - 1)
    t = np.asarray(table, dtype=np.float64)[p]
    return t[:, :h], t[:, h:]


def _pairs(D, rot, interleaved):
    h = rot // 2
    return (np.arange(h) * 2, np.arange(h) * 2 + 1) if interleaved else (np.arange(h), np.arange(h) + h)


def norm_rope(x, w, pos, table, rot, interleaved, eps):
    """y of heads x [N, H, D]: float64."""
    x = x.astype(np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * w.astype(np.float64)
    out = y.copy()
    if rot:
        c, s = _angles(table, pos, rot // 2)
        i, j = _pairs(x.shape[-1], rot, interleaved)
        out[..., i] = y[..., i] * c[:, None] - y[..., j] * s[:, None]
        out[..., j] = y[..., j] * c[:, None] + y[..., i] * s[:, None]
    return out


def norm_rope_backward(d, x, w, pos, table, rot, interleaved, eps):
    """(dx, dw, |dx|, |dw|): the Jacobian of norm_rope applied to d, the magnitudes of the sums."""
    x, d = x.astype(np.float64), d.astype(np.float64)
    e, me = d.copy(), np.abs(d)
    if rot:
        c, s = _angles(table, pos, rot // 2)
        c, s = c[:, None], s[:, None]
        i, j = _pairs(x.shape[-1], rot, interleaved)
        e[..., i] = d[..., i] * c + d[..., j] * s
        e[..., j] = d[..., j] * c - d[..., i] * s
        me[..., i] = np.abs(d[..., i] * c) + np.abs(d[..., j] * s)
        me[..., j] = np.abs(d[..., j] * c) + np.abs(d[..., i] * s)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dw, mw = (e * n).sum((0, 1)), (me * np.abs(n)).sum((0, 1))
    if w is not None:
        e, me = e * w.astype(np.float64), me * np.abs(w.astype(np.float64))
    dx = r * (e - n * (e * n).mean(-1, keepdims=True))
    return dx, dw, r * (me + np.abs(n) * (me * np.abs(n)).mean(-1, keepdims=True)), mw


def slot_topk(a, b, K, scale, n2=None):
    """(idx, val) of rows a [N, n1], b [N, n2]: ids by sorting, sums rounded to float32 as they are compared, the
    softmax in float64."""
    N, n2 = a.shape[0], b.shape[1]
    a = np.where(np.isnan(a), -np.inf, a).astype(np.float32)
    b = np.where(np.isnan(b), -np.inf, b).astype(np.float32)
    idx, val = np.zeros((N, K), np.int64), np.zeros((N, K))
    for t in range(N):
        ia = sorted(range(a.shape[1]), key=lambda c: (-a[t, c], c))[:K]
        ib = sorted(range(n2), key=lambda c: (-b[t, c], c))[:K]
        pairs = []
        for x, i in enumerate(ia):
            for y, j in enumerate(ib):
                with np.errstate(invalid="ignore", over="ignore"):
                    s = np.float32(a[t, i]) + np.float32(b[t, j])
                s = np.float32(-np.inf) if np.isnan(s) else s
                pairs.append((-s, x, y, i * n2 + j))
        pairs.sort()
        pairs = pairs[:K]
        idx[t] = [p[3] for p in pairs]
        s = np.array([-np.float64(p[0]) for p in pairs])
        val[t] = _softmax(s, scale)
    return idx, val


def _softmax(s, scale):
    if np.isneginf(s.max()):
        return np.zeros_like(s)
    e = np.exp((s - s.max()) * scale)
    return e / e.sum()


def slot_topk_backward(d_val, idx, a, b, scale):
    """(da, db, |da|, |db|) at the selection idx."""
    N, K = idx.shape
    n2 = b.shape[1]
    out = [np.zeros(a.shape), np.zeros(b.shape), np.zeros(a.shape), np.zeros(b.shape)]
    for t in range(N):
        i, j = idx[t] // n2, idx[t] % n2
        with np.errstate(invalid="ignore"):
            s = a[t, i].astype(np.float64) + b[t, j].astype(np.float64)
        # Sums are float32 by definition: those below its range are -infinity.
        s = np.where(np.isnan(s) | (s <= -(2.0 - 2.0 ** -24) * 2.0 ** 127), -np.inf, s)
        p = _softmax(s, scale)
        y = np.where(p > 0, d_val[t].astype(np.float64), 0.0)
        d = scale * p * (y - (p * y).sum())
        m = scale * p * (np.abs(y) + (p * np.abs(y)).sum())
        for c, (x, z) in enumerate(zip(i, j)):
            out[0][t, x] += d[c]
            out[1][t, z] += d[c]
            out[2][t, x] += m[c]
            out[3][t, z] += m[c]
    return out


def _heads(x, H):
    """Query or key heads [.., Hk, d] of every value head."""
    return np.repeat(x.astype(np.float64), H // x.shape[-2], axis=-2)


def _kept(a, x):
    """a x for a factor per row and head; 0 where the factor is 0, whatever x."""
    return np.where(a[..., None, None] > 0, a[..., None, None] * np.where(a[..., None, None] > 0, x, 0.0), 0.0)


def gdr_forward(q, k, v, g, beta, scale, state=None, lens=None, chunk=64):
    """(o, last, |o|, |last|) of u = beta (v - S'^T k), S = S' + k u^T, o = scale S^T q, with S' = exp(g) S: q, k [B, T, Hk, dk],
    v [B, T, H, dv], g and beta [B, T, H].

    The magnitudes bound what the rounding errors of an evaluation add up to, in units of one rounding: per column of a
    state, the root of the sum of squares of the norms that every token's step handles (its errors are independent
    in sign), decayed as the state is; later steps do not enlarge them where beta |k|^2 <= 2. (o: times |q|.) They are scaled up by
    what solving a chunk's tokens enlarges, the square of the norm of (1 + A diag(beta))^-1, A_ij = exp(g_{j+1} + .. + g_i) k_i . k_j."""
    B, T, _, dk = q.shape
    H, dv = v.shape[2:]
    live = _live(lens, B, T)
    q, k, v = _heads(q, H), _heads(k, H), v.astype(np.float64)
    S = np.zeros((B, H, dk, dv)) if state is None else np.array(state, dtype=np.float64)
    E2 = (S * S).sum(2)                                       # [B, H, dv]
    amp = np.ones((B, H))
    o, mo = np.zeros((B, T, H, dv)), np.zeros((B, T, H, dv))
    for t in range(T):
        on = live[:, t]
        a, be = np.exp(g[:, t].astype(np.float64)), beta[:, t].astype(np.float64)
        kk = k[:, t]
        S1 = _kept(a, S)
        pred = np.einsum("bhk,bhkv->bhv", kk, S1)
        u = be[..., None] * (v[:, t] - pred)
        S1 = S1 + kk[..., None] * u[:, :, None]
        n = np.sqrt((kk * kk).sum(-1))[..., None]
        local = np.abs(be)[..., None] * n * (np.abs(v[:, t]) + n * np.sqrt((S1 * S1).sum(2)) + np.abs(u))
        E1 = _kept(a * a, E2[..., None])[..., 0] + local ** 2 + (S1 * S1).sum(2)
        S, E2 = np.where(on[:, None, None, None], S1, S), np.where(on[:, None, None], E1, E2)
        o[:, t] = np.where(on[:, None, None], scale * np.einsum("bhk,bhkv->bhv", q[:, t], S), 0.0)
        mo[:, t] = np.where(on[:, None, None], abs(scale) * np.sqrt((q[:, t] ** 2).sum(-1))[..., None] * np.sqrt(E2), 0.0)
        if t % chunk == chunk - 1 or t == T - 1:
            amp = np.maximum(amp, _solve_norm(k, g, beta, live, t - t % chunk, t + 1))
    amp = amp[:, None, :, None]
    return o, S, mo * amp, np.sqrt(E2)[:, :, None] * amp[:, 0, :, :, None] * np.ones((1, 1, dk, 1))


def _solve_norm(k, g, beta, live, t0, t1):
    on = live[:, t0:t1, None]
    kk = np.where(on[..., None], k[:, t0:t1], 0.0).transpose(0, 2, 1, 3)
    G = np.cumsum(np.where(on, np.maximum(g[:, t0:t1].astype(np.float64), -1e4), 0.0), 1).transpose(0, 2, 1)
    be = np.where(on, beta[:, t0:t1], 0.0).transpose(0, 2, 1).astype(np.float64)
    n = t1 - t0
    D = np.exp(np.minimum(G[..., :, None] - G[..., None, :], 0.0)) * np.tril(np.ones((n, n)), -1)
    A = D * np.einsum("bhik,bhjk->bhij", kk, kk) * be[..., None, :]
    return np.maximum(np.abs(np.linalg.inv(np.eye(n) + A)).sum(-1).max(-1) ** 2, 1.0)


def gdr_backward(d_o, q, k, v, g, beta, scale, state=None, d_last=None, lens=None, chunk=64):
    """Gradients from the chain rule, token by token: (grads, magnitudes), dicts of dq, dk, dv, dg, dbeta and dstate. Magnitudes
    as in gdr_forward; dg's are of the sums a chunked evaluation adds up to it, q . dq and v . dv of the later tokens of its chunk."""
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    live = _live(lens, B, T)
    fold = lambda x: x.reshape(B, T, Hk, H // Hk, dk).sum(3)  # noqa: E731
    q, k, v, d_o = _heads(q, H), _heads(k, H), v.astype(np.float64), d_o.astype(np.float64)
    S = np.zeros((B, H, dk, dv)) if state is None else np.array(state, dtype=np.float64)
    E2, amp = (S * S).sum(2), np.ones((B, H))
    seen = []
    for t in range(T):
        on = live[:, t]
        a, be, kk = np.exp(g[:, t].astype(np.float64)), beta[:, t].astype(np.float64), k[:, t]
        S1 = _kept(a, S)
        r = v[:, t] - np.einsum("bhk,bhkv->bhv", kk, S1)
        S2 = S1 + kk[..., None] * (be[..., None] * r)[:, :, None]
        n = np.sqrt((kk * kk).sum(-1))[..., None]
        local = np.abs(be)[..., None] * n * (np.abs(v[:, t]) + n * np.sqrt((S2 * S2).sum(2)) + np.abs(be[..., None] * r))
        E1 = _kept(a * a, E2[..., None])[..., 0] + local ** 2 + (S2 * S2).sum(2)
        seen.append((S1, S2, r, np.sqrt(E2), np.sqrt(E1)))
        S, E2 = np.where(on[:, None, None, None], S2, S), np.where(on[:, None, None], E1, E2)
        if t % chunk == chunk - 1 or t == T - 1:
            amp = np.maximum(amp, _solve_norm(k, g, beta, live, t - t % chunk, t + 1))
    z = lambda *s: np.zeros(s)  # noqa: E731
    r_ = dict(dq=z(B, T, H, dk), dk=z(B, T, H, dk), dv=z(B, T, H, dv), dg=z(B, T, H), dbeta=z(B, T, H))
    m = {n: np.zeros_like(x) for n, x in r_.items()}
    R = z(B, H, dk, dv) if d_last is None else np.array(d_last, dtype=np.float64)
    F2 = (R * R).sum(2)
    rest = z(B, H)
    for t in range(T - 1, -1, -1):
        on = live[:, t]
        a, be, kk, qq, do = np.exp(g[:, t].astype(np.float64)), beta[:, t].astype(np.float64), k[:, t], q[:, t], d_o[:, t] * scale
        S1, S2, r, E0, E = seen[t]
        norm = lambda x: np.sqrt((x * x).sum(2))  # noqa: E731
        nk, nq = (np.sqrt((x * x).sum(-1))[..., None] for x in (kk, qq))
        if t % chunk == chunk - 1 or t == T - 1:
            rest = (E0 * np.sqrt(F2)).sum(-1) + (E * np.sqrt(F2)).sum(-1)
        Rt = R + qq[..., None] * do[:, :, None]
        du = np.einsum("bhk,bhkv->bhv", kk, Rt)
        d = be[..., None] * du
        u = be[..., None] * r
        F = np.sqrt(F2 + (nq * np.abs(do)) ** 2 + (nk * np.abs(d)) ** 2 + (Rt * Rt).sum(2))
        new = dict(dq=np.einsum("bhkv,bhv->bhk", S2, do), dk=np.einsum("bhkv,bhv->bhk", Rt, u) - np.einsum("bhkv,bhv->bhk", S1, d),
                   dv=d, dbeta=(du * r).sum(-1))
        ab = np.abs(be)[..., None]
        one = np.ones((1, 1, dk))
        mags = dict(dq=(E * np.abs(do)).sum(-1)[..., None] * one, dv=ab * nk * F, dbeta=(nk * F * np.abs(r) + np.abs(du) * (np.abs(v[:, t]) + nk * E)).sum(-1),
                    dk=(F * np.abs(u) + E * np.abs(d) + 2 * ab * nk * E * F).sum(-1)[..., None] * one)
        rest = rest + nq[..., 0] * mags["dq"][..., 0] + (np.abs(v[:, t]) * mags["dv"]).sum(-1)
        mags["dg"] = rest
        R1 = Rt - kk[..., None] * d[:, :, None]
        new["dg"] = (R1 * S1).sum((2, 3))   # S1 is already decayed; 0 past a reset
        for n, x in new.items():
            w = on.reshape((B,) + (1,) * (x.ndim - 1))
            r_[n][:, t], m[n][:, t] = np.where(w, x, 0.0), np.where(w, mags[n], 0.0)
        R = np.where(on[:, None, None, None], _kept(a, R1), R)
        F2 = np.where(on[:, None, None], _kept(a * a, (F ** 2)[..., None])[..., 0], F2)
    for n in ("dq", "dk"):
        r_[n], m[n] = fold(r_[n]), fold(m[n] * amp[:, None, :, None])
    m["dv"], m["dg"], m["dbeta"] = m["dv"] * amp[:, None, :, None], m["dg"] * amp[:, None], m["dbeta"] * amp[:, None]
    r_["dstate"], m["dstate"] = R, np.sqrt(F2)[:, :, None] * amp[..., None, None] * np.ones((1, 1, dk, 1))
    return r_, m


def _rms(x, eps):
    return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def _norm_back(d, x, w, eps):
    """(dx, dw, |dx|, |dw|) of y = x / rms(x) w per row [.., D], and of the sums over absolute values."""
    w = np.ones(x.shape[-1]) if w is None else w.astype(np.float64)
    r = _rms(x, eps)
    n, dn = x * r, d * w
    lead = tuple(range(x.ndim - 1))
    dx = r * (dn - n * (dn * n).mean(-1, keepdims=True))
    return dx, (d * n).sum(lead), r * (np.abs(dn) + np.abs(n) * (np.abs(dn * n)).mean(-1, keepdims=True)), np.abs(d * n).sum(lead)


def _sigmoid(z):
    return np.exp(-np.logaddexp(0.0, -z))


def gate_norm(x, z, w, eps):
    x, z = x.astype(np.float64), z.astype(np.float64)
    return x * _rms(x, eps) * (1.0 if w is None else w.astype(np.float64)) * z * _sigmoid(z)


def gate_norm_backward(d, x, z, w, eps):
    """(grads, magnitudes), dicts of dx, dz and dw."""
    d, x, z = (t.astype(np.float64) for t in (d, x, z))
    s = _sigmoid(z)
    dx, dw, mx, mw = _norm_back(d * z * s, x, w, eps)
    n = x * _rms(x, eps) * (1.0 if w is None else w.astype(np.float64))
    dz = d * n * s * (1.0 + z * (1.0 - s))
    return dict(dx=dx, dz=dz, dw=dw), dict(dx=mx, dz=np.abs(d * n * s) * (1.0 + np.abs(z) * (1.0 - s)), dw=mw)


def residual_norm(x, y, w, a, norm_y, wy, eps, rounded):
    """(h, n, |h|): n is that of `rounded`, the h that was returned."""
    x, y = x.astype(np.float64), y.astype(np.float64)
    if norm_y:
        y = y * _rms(y, eps) * (1.0 if wy is None else wy.astype(np.float64))
    y = y * (1.0 if a is None else a.astype(np.float64))
    f = rounded.astype(np.float64)
    return x + y, f * _rms(f, eps) * (1.0 if w is None else w.astype(np.float64)), np.abs(x) + np.abs(y)


def residual_norm_backward(dh, dn, h, y, w, a, norm_y, wy, eps):
    """(grads, magnitudes), dicts of dx, dy, dw, dscale and dwy."""
    h, y, dn = (t.astype(np.float64) for t in (h, y, dn))
    aa = np.ones(h.shape[-1]) if a is None else a.astype(np.float64)
    dx, dw, mx, mw = _norm_back(dn, h, w, eps)
    if dh is not None:
        dx, mx = dx + dh.astype(np.float64), mx + np.abs(dh)
    part = y * _rms(y, eps) * (1.0 if wy is None else wy.astype(np.float64)) if norm_y else y
    r, m = dict(dx=dx, dw=dw, dscale=(dx * part).sum(0)), dict(dx=mx, dw=mw, dscale=(mx * np.abs(part)).sum(0))
    if norm_y:
        r["dy"], r["dwy"], _, _ = _norm_back(dx * aa, y, wy, eps)
        _, _, m["dy"], m["dwy"] = _norm_back(mx * np.abs(aa), np.abs(y), None if wy is None else np.abs(wy), eps)
    else:
        r["dy"], m["dy"] = dx * aa, mx * np.abs(aa)
    return r, m
