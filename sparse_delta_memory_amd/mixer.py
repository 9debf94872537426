"""A mixer layer step made of the package's operators: a dense gated state per head beside the sparse bank.

    python -m sparse_delta_memory_amd.mixer        # a short prompt, then single tokens, on cuda:0

One projection of the token rows x [P, T, model] gives everything:

  query and key heads  -> norm_rope                      -> glr_forward / glr_step  (the dense state, value heads v)
  write scores a, b    -> slot_topk -> k_idx, k_val      -> phase1, read_step, dw_step (the bank, value rows u)
  read scores a, b     -> slot_topk -> q_idx, q_val         (absolute ids, in Phase 1's chunks)
  gates, beta                        (log-sigmoid per token and head, sigmoid per token)

and the layer's output is the dense heads' outputs and the bank's reads, side by side. Streams are rows of
the batch; the bank is worked through in chunks of C tokens (phase1 of all chunks at once, then read side and
DW step by step), so prompts are whole chunks here. A single token of every stream is a chunk of one.
"""

from __future__ import annotations

import torch

from . import alloc_dw_workspace, dw_step, glr_forward, glr_step, make_shape, norm_rope, phase1, read_step, rope_table, slot_topk


class Mixer:
    """The layer's sizes and weights. P streams share nothing but the weights: stream p owns the bank's rows
    p * S .. (p + 1) * S - 1, S = n * n slots."""

    def __init__(self, model=256, heads=4, key_heads=2, d=64, hd=64, n=32, W=4, R=4, C=32, rot=32, positions=4096, seed=0, device="cuda",
                 dtype=torch.bfloat16):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.key_heads, self.d, self.hd, self.n, self.W, self.R, self.C = heads, key_heads, d, hd, n, W, R, C
        # q, k, v heads; scores of the writes and of the reads (two rows each); bank values; gates of the heads, the bank, and beta
        self.split = [key_heads * d, key_heads * d, heads * d, n, n, n, n, hd, heads + 2]
        w = (torch.randn((model, sum(self.split)), generator=gen, device=device) * model ** -0.5).to(dtype)
        # Each part starts on 16 bytes in every row, rows included (unused columns between): views of the projection's rows
        # then take the operators' wide loads. Without it one odd part, the gates', puts all of them on the element paths.
        unit = 16 // dtype.itemsize
        self.padded = [-(-c // unit) * unit for c in self.split]
        self.w = torch.cat([torch.nn.functional.pad(c, (0, wide - c.shape[1])) for c, wide in zip(w.split(self.split, 1), self.padded)], 1)
        self.q_norm, self.k_norm = torch.ones(d, device=device), torch.ones(d, device=device)
        self.table = rope_table(positions, rot, device=device)

    def rows(self, x, pos):
        """x [P, T, model], pos [P * T] -> what the two memories take before slots are chosen, rows in x's order: q, k, v, their
        gates, the score rows (score_rows), and the bank's gate, beta and values."""
        P, T = x.shape[:2]
        parts = self.padded[:3] + [sum(self.padded[3:7])] + self.padded[7:]      # the four score rows stay side by side
        q, k, v, scores, u, g = (x.flatten(0, 1) @ self.w).split(parts, 1)
        q, k, v, u, g = (t[:, :c] for t, c in zip((q, k, v, u, g), self.split[:3] + self.split[7:]))
        heads = lambda t, h: t.view(P * T, h, self.d)  # noqa: E731
        q, k = norm_rope(heads(q, self.key_heads), heads(k, self.key_heads), self.q_norm, self.k_norm, pos, self.table)
        g = g.float()
        gates, gate, beta = torch.nn.functional.logsigmoid(g[:, :self.heads] + 3), torch.nn.functional.logsigmoid(g[:, -2] + 3), g[:, -1].sigmoid()
        return q, k, heads(v, self.heads), gates, scores, gate, beta, u.float()

    def score_rows(self, scores):
        """a and b of the writes, then of the reads."""
        return [t[:, :self.n] for t in scores.split(self.padded[3], 1)]

    def project(self, x, pos):
        """The same with the slots of every row, ids within its stream, in place of the scores."""
        q, k, v, gates, scores, gate, beta, u = self.rows(x, pos)
        wa, wb, ra, rb = self.score_rows(scores)
        return q, k, v, gates, *slot_topk(wa, wb, self.W), *slot_topk(ra, rb, self.R), gate, beta, u

    def check_positions(self, fn, start, T):
        """norm_rope takes a position outside its table to the nearest row: tokens there would turn by the wrong angles."""
        if start < 0 or start + T > self.table.shape[0]:
            raise ValueError("Mixer.%s: positions %d .. %d of a table of %d" % (fn, start, start + T - 1, self.table.shape[0]))

    def bank(self, P, dtype=torch.float32, device="cuda"):
        return torch.zeros((P * self.n * self.n, self.hd), dtype=dtype, device=device)

    def sparse(self, bank, P, T, C, scores, gate, beta, u):
        """The bank over T tokens of P streams, in chunks of C: reads [P * T, hd], the bank updated in place."""
        steps, S = T // C, self.n * self.n
        # Chunk ti * P + p holds the tokens ti * C .. of stream p.
        chunks = lambda t: t.unflatten(0, (P, steps, C)).transpose(0, 1).reshape(-1, *t.shape[1:])  # noqa: E731
        N = steps * P
        shape = make_shape(N, C, self.W, self.R, P=P, key_bits=max(1, (S - 1).bit_length()), stream_offset=S)
        # Slots in Phase 1's layouts and absolute ids, from the score rows in the chunks' order.
        wa, wb, ra, rb = self.score_rows(chunks(scores))
        (ki, kv), (qi, qv) = ([t.view(N, C, K) for t in slot_topk(a, b, K, shape=shape)] for a, b, K in ((wa, wb, self.W), (ra, rb, self.R)))
        g, b = chunks(gate).view(N, C), chunks(beta).view(N, C)
        out = phase1(shape, ki, qi, kv, qv, g)
        v = chunks(u).contiguous()
        dv, pred, read = torch.empty_like(v), torch.empty_like(v), torch.empty_like(v)
        ws = alloc_dw_workspace(shape, self.hd, bank.device)
        for ti in range(steps):
            read_step(bank, out, ki, qi, v, b, dv, pred, read, shape, ti, step_rows=P * C)
            dw_step(bank, dv, out["krec"], shape, ti, dv_step_rows=P * C, workspace=ws)
        return read.view(steps, P, C, self.hd).transpose(0, 1).reshape(P * T, self.hd)

    def prompt(self, x, bank, state=None, start=0):
        """x [P, T, model] (T a multiple of C): (y [P, T, heads * d + hd] float32, the dense state [P, heads, d, d]). The bank is
        updated in place. start: the position of the first token."""
        P, T = x.shape[:2]
        if T % self.C:
            raise ValueError("Mixer.prompt: %d tokens are no whole chunks of %d" % (T, self.C))
        self.check_positions("prompt", start, T)
        pos = (torch.arange(start, start + T, dtype=torch.int32, device=x.device)).repeat(P)
        q, k, v, gates, *sparse = self.rows(x, pos)
        seq = lambda t: t.unflatten(0, (P, T))  # noqa: E731
        o, state = glr_forward(seq(q), seq(k), seq(v), seq(gates), state=state)
        read = self.sparse(bank, P, T, self.C, *sparse)
        return torch.cat([o.flatten(2).float(), seq(read)], 2), state

    def token(self, x, bank, state, pos):
        """One token of every stream: x [P, model] -> y [P, heads * d + hd]; the bank and the state are updated in place."""
        P = x.shape[0]
        self.check_positions("token", pos, 1)
        q, k, v, gates, *sparse = self.rows(x[:, None], torch.full((P,), pos, dtype=torch.int32, device=x.device))
        o = glr_step(q, k, v, gates, state)
        return torch.cat([o.flatten(1).float(), self.sparse(bank, P, 1, 1, *sparse)], 1)


def main():
    m = Mixer()
    P, T, more = 2, 4 * m.C, 8
    x = torch.randn((P, T + more, m.w.shape[0]), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(m.w.dtype)
    bank = m.bank(P)
    y, state = m.prompt(x[:, :T], bank)
    print("prompt: %d streams of %d tokens, outputs %s, rms %.3f" % (P, T, tuple(y.shape), y.square().mean().sqrt()))
    for t in range(T, T + more):
        y = m.token(x[:, t], bank, state, t)
    print("%d more tokens: outputs %s, rms %.3f, %d slots written" % (more, tuple(y.shape), y.square().mean().sqrt(),
                                                                    int((bank != 0).any(1).sum())))


if __name__ == "__main__":
    main()
