"""Small language models on the operators of lm.py: training on token sequences and answering one
token at a time.  Run ``python -m adjoint_gradients_long_gb300.lm_train``.

TinyLm: one residual layer of linear attention with a decay for each head,
    x_t  = E[token_t]
    [q|k|v|z] = x W_in,  g = log sigmoid(z + 3)      (one decay a head and token)
    y    = x + attention(q, k, v, g) W_o,   logits = y E^T
A training step runs LinAttn forward, TokenLogProbs with the loss's gradient, LinAttn backward and
GradClip over all gradients, then plain gradient descent.  An answer runs the prompt through
LinAttn, keeps its final state, and goes on with LinStep and the top of TokenLogProbs, or a Sampler.

SelLm: one residual layer of the selective recurrence behind its short convolution,
    [u|z] = x W_in,  c = silu(conv(u)),  [dt|B|C] = c W_x,  y = x + scan(c, dt, B, C, z) W_o
trained on documents of different lengths packed one behind the other (ShortConv, SelScan and their
gradients) and answering from the states that its prompt left (ShortConvStep, SelScanStep).
The dense projections are torch products.
"""
from __future__ import annotations

import torch

from . import lm


class Chooser:
    """The next token of one row of logits, as TinyLm.answer gives it."""

    def __init__(self, vocab, top, sampling, seed, device):
        self.probs = lm.TokenLogProbs(1, vocab, top=top, device=device)
        self.nobody = torch.full((1,), -1, dtype=torch.int64, device=device)
        self.sampler = None if sampling is None else lm.Sampler(1, vocab, device=device)
        self.settings = {n: torch.full((1,), v, device=device, dtype=torch.int32 if n == "top_k" else torch.float32)
                         for n, v in (sampling or {}).items()}
        self.gen, self.device = torch.Generator().manual_seed(seed), device

    def __call__(self, logits):
        r = self.probs.forward(logits, self.nobody)
        best = list(zip(r.top_id[0].tolist(), r.top_logp[0].tolist()))
        if self.sampler is None:
            return best[0][0], best[0][1], best[1:]
        token, logp = self.sampler.sample(logits, torch.rand(1, generator=self.gen).to(self.device), **self.settings)
        return token.item(), logp.item(), best


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

    def answer(self, tokens, n, top=4, sampling=None, seed=0):
        """The n next tokens, one by one, with their log probabilities and the `top` likeliest ones:
        lists of (token, logp, [(token, logp), ...]).  sampling None: the likeliest each time (the list
        then holds the others); else a dict of settings for Sampler.sample, one number each, and logp is
        that of the distribution drawn from."""
        logits, state = self.prompt(tokens)
        step = lm.LinStep(1, self.H, self.D, self.D, Hk=self.Hk, scale=self.scale, device=self.device)
        chooser = Chooser(self.V, top, sampling, seed, self.device)
        out = []
        for i in range(n):
            out.append(chooser(logits))
            x = self.E[torch.tensor([out[-1][0]], device=self.device)]
            q, k, v, z = self._project(x)
            o = step.step(q, k, v, self._decay(z), state)
            y = x + o.reshape(1, -1).float() @ self.W_o
            logits = (y @ self.E.T).bfloat16()
        return out


class SelLm:
    """vocab tokens, width P, N states a channel, W taps; bf16 activations, fp32 weights.  A step takes up
    to T tokens of up to B documents, packed."""

    def __init__(self, vocab, B, T, P=128, N=16, W=4, device="cuda", seed=0):
        self.V, self.B, self.T, self.P, self.N, self.W, self.device = vocab, B, T, P, N, W, device
        gen = torch.Generator().manual_seed(seed)
        def w(*s):
            return (torch.randn(*s, generator=gen) / s[0] ** 0.5).to(device)
        self.E, self.W_in, self.W_x, self.W_o = w(vocab, P) * vocab ** 0.5 / P ** 0.5, w(P, 2 * P), w(P, P + 2 * N), w(P, P) * 0.5
        self.w, self.b = w(W, P).T.contiguous(), torch.zeros(P, device=device)
        self.A = -(torch.arange(N, device=device) + 1.0).repeat(P, 1)
        self.D = torch.ones(P, device=device)
        rate = torch.exp(torch.rand(P, generator=gen) * 4.6 - 6.9).to(device)          # steps of 0.001 to 0.1
        self.dt_bias = rate + torch.log(-torch.expm1(-rate))
        self.params = [self.E, self.W_in, self.W_x, self.W_o, self.w, self.b, self.A, self.D, self.dt_bias]
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.conv = lm.ShortConv(B, T, P, W, packed=True, backward=True, device=device)
        self.scan = lm.SelScan(B, T, P, N, packed=True, backward=True, device=device)
        self.probs = lm.TokenLogProbs(T, vocab, device=device)
        self.clipper = lm.GradClip(self.grads)

    def _split(self, h):
        P, N = self.P, self.N
        return h[..., :P], h[..., P:P + N], h[..., P + N:]

    def loss_and_grads(self, tokens, targets, offsets):
        """Mean negative log probability of the targets (a device scalar) over packed tokens [T], targets
        [T] (-1: none, as for rows of no document) and offsets [B+1]; fills self.grads."""
        P, T = self.P, self.T
        # The operators leave rows of no document as they were: an older batch's values, which the products below, over
        # all rows, must not see
        t = torch.arange(T, device=self.device)
        nobody = ((t < offsets[0]) | (t >= offsets[-1]))[:, None]
        x = self.E[tokens]
        uz = (x @ self.W_in).bfloat16()
        u, z = uz[:, :P], uz[:, P:]
        c = self.conv.forward(u, self.w, self.b, None, offsets)[0].masked_fill(nobody, 0)
        cf = c.float()
        dt, Bm, Cm = self._split((cf @ self.W_x).bfloat16())
        s = self.scan.forward(c, dt, self.A, Bm, Cm, self.D, z, self.dt_bias, None, offsets)[0].float().masked_fill_(nobody, 0)
        y = x + s @ self.W_o
        logits = (y @ self.E.T).bfloat16()
        count = (targets >= 0).sum()
        glp = (-1.0 / count.float()).expand(T).contiguous()
        r = self.probs.gradient(logits, targets, glp, dlogits=logits)
        dl = r.dlogits.float()
        dy = dl @ self.E
        dE, dW_in, dW_x, dW_o, dw, db, dA, dD, ddt_bias = self.grads
        torch.mm(dl.T, y, out=dE)
        torch.mm(s.T, dy, out=dW_o)
        g = self.scan.backward(c, dt, self.A, Bm, Cm, (dy @ self.W_o.T).bfloat16(), self.D, z, self.dt_bias, None, None, offsets)
        dA.copy_(g.dA), dD.copy_(g.dD), ddt_bias.copy_(g.ddt_bias)
        dh = torch.cat([g.ddt.float(), g.dB.float(), g.dC.float()], -1).masked_fill_(nobody, 0)
        torch.mm(cf.T, dh, out=dW_x)
        dc = (g.dx.float() + dh @ self.W_x.T).bfloat16()
        du, gw, gb, _ = self.conv.backward(u, self.w, dc, self.b, None, None, offsets)
        dw.copy_(gw), db.copy_(gb)
        duz = torch.cat([du.float(), g.dz.float()], -1).masked_fill_(nobody, 0)
        torch.mm(x.T, duz, out=dW_in)
        dx = dy + duz @ self.W_in.T
        # sorted sums: a token that occurs often gets the same bits every time
        dE.index_put_((tokens,), dx, accumulate=True)
        return -r.logp.sum() / count

    def step(self, tokens, targets, offsets, lr=0.5, max_norm=1.0):
        """One training step: (loss, gradient norm) as device scalars."""
        loss = self.loss_and_grads(tokens, targets, offsets)
        norm, _ = self.clipper.clip(max_norm)
        for p, g in zip(self.params, self.grads):
            p.add_(g, alpha=-lr)
        return loss, norm

    def prompts(self, tokens, offsets):
        """Logits after the last token of every prompt, packed tokens [n] with offsets [k+1] (none of them
        empty), and the states that go on from there: (logits [k,V], inputs [k,W-1,P], states [k,P,N])."""
        k, n = len(offsets) - 1, len(tokens)
        x = self.E[tokens]
        uz = (x @ self.W_in).bfloat16()
        conv = lm.ShortConv(k, n, self.P, self.W, packed=True, device=self.device)
        scan = lm.SelScan(k, n, self.P, self.N, packed=True, device=self.device)
        c, taps = conv.forward(uz[:, :self.P], self.w, self.b, None, offsets)
        dt, Bm, Cm = self._split((c.float() @ self.W_x).bfloat16())
        s, state = scan.forward(c, dt, self.A, Bm, Cm, self.D, uz[:, self.P:], self.dt_bias, None, offsets)
        last = offsets[1:] - 1
        y = x[last] + s[last].float() @ self.W_o
        return (y @ self.E.T).bfloat16(), taps, state

    def answers(self, tokens, offsets, n, sampling=None, seed=0):
        """n tokens after each of k packed prompts: tokens [k,n] and their log probabilities [k,n].  sampling:
        settings for Sampler.sample, one number each; None: the likeliest each time."""
        logits, taps, state = self.prompts(tokens, offsets)
        k = len(offsets) - 1
        conv = lm.ShortConvStep(k, self.P, self.W, device=self.device)
        scan = lm.SelScanStep(k, self.P, self.N, device=self.device)
        sampler = lm.Sampler(k, self.V, device=self.device)
        settings = {n_: torch.full((k,), v, device=self.device, dtype=torch.int32 if n_ == "top_k" else torch.float32)
                    for n_, v in (sampling or dict(temperature=0.0)).items()}
        u = torch.rand(n, k, generator=torch.Generator().manual_seed(seed)).to(self.device)
        out, lps = [], []
        for i in range(n):
            token, logp = sampler.sample(logits, u[i], **settings)
            out.append(token.clone()), lps.append(logp.clone())
            x = self.E[token]
            uz = (x @ self.W_in).bfloat16()
            c = conv.step(uz[:, :self.P], self.w, taps, self.b)
            dt, Bm, Cm = self._split((c.float() @ self.W_x).bfloat16())
            s = scan.step(c, dt, self.A, Bm, Cm, state, self.D, uz[:, self.P:], self.dt_bias)
            logits = ((x + s.float() @ self.W_o) @ self.E.T).bfloat16()
        return torch.stack(out, 1), torch.stack(lps, 1)


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
    drawn = model.answer(seq[:60], 12, sampling=dict(temperature=0.8, top_k=50, top_p=0.95))
    print(f"drawn with temperature, top-k and top-p: {[t for t, _, _ in drawn]}")

    # the same sequences as documents of different lengths, packed into one row of tokens
    lengths = [512, 100, 0, 700, 400]
    offsets = torch.tensor([0, *lengths], device="cuda").cumsum(0)
    sel = SelLm(vocab, len(lengths), 2048)
    seq = cycle_tokens(len(lengths), 1024, period, vocab)
    def pack(shift):
        rows = [seq[i, shift:shift + n] for i, n in enumerate(lengths)]
        tail = torch.full((sel.T - sum(lengths),), -shift, dtype=torch.int64, device="cuda")     # no document: no target
        return torch.cat([*rows, tail])
    for i in range(100):
        loss, norm = sel.step(pack(0), pack(1), offsets)
        if i % 20 == 19:
            print(f"selective layer, step {i + 1}: loss {loss.item():.4f}, gradient norm {norm.item():.3f}")
    k = torch.tensor([0, 40, 75], device="cuda")
    tokens, _ = sel.answers(torch.cat([seq[0, :40], seq[1, :35]]), k, 12)
    want = torch.stack([seq[0, 40:52], seq[1, 35:47]])
    print(f"answers of two prompts: {(tokens == want).sum().item()} of 24 as in the sequences")


if __name__ == "__main__":
    main()
