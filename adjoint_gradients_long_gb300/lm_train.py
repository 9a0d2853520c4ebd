"""A small language model on the operators of lm.py: training on a token sequence and answering
one token at a time.  Run ``python -m adjoint_gradients_long_gb300.lm_train``.

One residual layer of linear attention with a decay for each head:
    x_t  = E[token_t]
    [q|k|v|z] = x W_in,  g = log sigmoid(z + 3)      (one decay a head and token)
    y    = x + attention(q, k, v, g) W_o,   logits = y E^T
A training step runs LinAttn forward, TokenLogProbs with the loss's gradient, LinAttn backward and
GradClip over all gradients, then plain gradient descent.  An answer runs the prompt through
LinAttn, keeps its final state, and goes on with LinStep and the top of TokenLogProbs.
The dense projections are torch products.
"""
from __future__ import annotations

import torch

from . import lm


class TinyLm:
    """vocab tokens, width P = H * D, bf16 activations, fp32 weights.  B rows of T tokens a step."""

    def __init__(self, vocab, B, T, H=4, D=64, Hk=None, device="cuda", seed=0):
        self.V, self.B, self.T, self.H, self.D, self.Hk = vocab, B, T, H, D, Hk or H
        P, gen = H * D, torch.Generator().manual_seed(seed)
        wide = 2 * self.Hk * D + H * D + H
        def w(*s):
            return (torch.randn(*s, generator=gen) / s[0] ** 0.5).to(device)
        self.E, self.W_in, self.W_o = w(vocab, P) * vocab ** 0.5 / P ** 0.5, w(P, wide), w(P, P) * 0.5
        self.params = [self.E, self.W_in, self.W_o]
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.scale = D ** -0.5
        self.att = lm.LinAttn(B, T, H, D, D, Hk=self.Hk, scale=self.scale, backward=True, device=device)
        self.probs = lm.TokenLogProbs(B * T, vocab, device=device)
        self.clipper = lm.GradClip(self.grads)
        self.device = device

    def _project(self, x):
        """q, k, v as slices of one projection (bf16), and the decay's argument z (fp32)."""
        h = x @ self.W_in
        wq, wv = self.Hk * self.D, self.H * self.D
        qkv = h[..., :2 * wq + wv].bfloat16()
        split = lambda t, n: t.unflatten(-1, (n, self.D))  # noqa: E731
        q, k, v = split(qkv[..., :wq], self.Hk), split(qkv[..., wq:2 * wq], self.Hk), split(qkv[..., 2 * wq:], self.H)
        return q, k, v, h[..., -self.H:].contiguous()

    def _decay(self, z):
        return torch.nn.functional.logsigmoid(z + 3.0)

    def loss_and_grads(self, tokens):
        """Mean negative log probability of the next tokens (a device scalar); fills self.grads."""
        B, T, P = self.B, self.T, self.H * self.D
        x = self.E[tokens[:, :-1]]
        q, k, v, z = self._project(x)
        g = self._decay(z)
        o, _ = self.att.forward(q, k, v, g)
        o2 = o.reshape(B * T, P).float()
        y = x.reshape(B * T, P) + o2 @ self.W_o
        logits = (y @ self.E.T).bfloat16()
        targets = tokens[:, 1:].reshape(-1)
        glp = torch.full((B * T,), -1.0 / (B * T), device=self.device)
        r = self.probs.gradient(logits, targets, glp, dlogits=logits)     # in place
        dl = r.dlogits.float()
        dy = dl @ self.E
        dE, dW_in, dW_o = self.grads
        torch.mm(dl.T, y, out=dE)
        torch.mm(o2.T, dy, out=dW_o)
        go = (dy @ self.W_o.T).bfloat16().reshape(B, T, self.H, self.D)
        dq, dk, dv, dg, _ = self.att.backward(q, k, v, g, go)
        dz = dg * torch.sigmoid(-(z + 3.0))
        dh = torch.cat([t.reshape(B * T, -1).float() for t in (dq, dk, dv, dz)], -1)
        torch.mm(x.reshape(B * T, P).T, dh, out=dW_in)
        dx = dy + dh @ self.W_in.T
        # sorted sums: a token that occurs often gets the same bits every time
        dE.index_put_((tokens[:, :-1].reshape(-1),), dx, accumulate=True)
        return -r.logp.mean()

    def step(self, tokens, lr=0.5, max_norm=1.0):
        """One training step on tokens [B, T+1]: (loss, gradient norm) as device scalars."""
        loss = self.loss_and_grads(tokens)
        norm, _ = self.clipper.clip(max_norm)
        for p, g in zip(self.params, self.grads):
            p.add_(g, alpha=-lr)
        return loss, norm

    def prompt(self, tokens):
        """Logits after the last token of one prompt [n], and the state that goes on from there."""
        x = self.E[tokens][None]
        q, k, v, z = self._project(x)
        att = lm.LinAttn(1, len(tokens), self.H, self.D, self.D, Hk=self.Hk, scale=self.scale, device=self.device)
        o, s1 = att.forward(q, k, v, self._decay(z))
        y = x[0, -1] + o[0, -1].reshape(-1).float() @ self.W_o
        return (y @ self.E.T).bfloat16()[None], s1

    def answer(self, tokens, n, top=4):
        """The n likeliest next tokens, one by one, with their log probabilities and alternatives:
        lists of (token, logp, [(token, logp), ...])."""
        logits, state = self.prompt(tokens)
        step = lm.LinStep(1, self.H, self.D, self.D, Hk=self.Hk, scale=self.scale, device=self.device)
        probs = lm.TokenLogProbs(1, self.V, top=top, device=self.device)
        nobody = torch.full((1,), -1, dtype=torch.int64, device=self.device)
        out = []
        for i in range(n):
            r = probs.forward(logits, nobody)
            ids, lps = r.top_id[0].tolist(), r.top_logp[0].tolist()
            out.append((ids[0], lps[0], list(zip(ids[1:], lps[1:]))))
            x = self.E[torch.tensor([ids[0]], device=self.device)]
            q, k, v, z = self._project(x)
            o = step.step(q, k, v, self._decay(z), state)
            y = x + o.reshape(1, -1).float() @ self.W_o
            logits = (y @ self.E.T).bfloat16()
        return out


def cycle_tokens(B, T, period, vocab, seed=0, device="cuda"):
    """Rows that repeat one random sequence of `period` distinct tokens, each from its own place."""
    gen = torch.Generator().manual_seed(seed)
    base = torch.randperm(vocab, generator=gen)[:period]
    at = torch.randint(0, period, (B, 1), generator=gen) + torch.arange(T + 1)
    return base[at % period].to(device)


def main():
    B, T, vocab, period = 4, 512, 1000, 37
    model = TinyLm(vocab, B, T)
    for i in range(100):
        loss, norm = model.step(cycle_tokens(B, T, period, vocab))
        if i % 20 == 19:
            print(f"step {i + 1}: loss {loss.item():.4f}, gradient norm {norm.item():.3f}")
    seq = cycle_tokens(1, 100, period, vocab)[0]
    got = model.answer(seq[:60], 12)
    right = sum(t == s for (t, _, _), s in zip(got, seq[60:72].tolist()))
    print(f"answers: {right} of 12 as in the sequence; first alternatives of the last: {got[-1][2]}")


if __name__ == "__main__":
    main()
