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
