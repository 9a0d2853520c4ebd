"""The measured cases of the language-model operators: linear attention with a decay for each
head (prompt, training and single-token forms), log probabilities of tokens with entropy, top
alternatives and gradient, and clipping gradients by their global norm.

`run` computes them in their plain form (elementary torch operations in 32 bits) or, with `own`
set, by the calls of adjoint_gradients_long_gb300.lm.  `exact` gives the same results in 64
bits from the definitions, written apart from the plain form.
"""
import math

import torch

own = False

EPS = 1e-6          # added to the norm in the clipping coefficient
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_NAME = {True: "bf16", False: "f32"}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one sequence being answered, one layer of 16 heads (2048 channels): latency only
        dict(name="step_one", op="step", B=1, H=16, Hk=16, Dk=128, Dv=128, dtype="bf16", pool=1),
        # a full serving batch whose states lie scattered in a pool of slots
        dict(name="step_batch", op="step", B=256, H=16, Hk=16, Dk=128, Dv=128, dtype="bf16", pool=300),
        # a short follow-up prompt that continues from a stored state
        dict(name="prompt_short", op="fwd", B=1, T=77, H=16, Hk=16, Dk=64, Dv=64, dtype="bf16", s0=True, docs=0),
        # a whole long context: 131072 tokens of 2048 channels in heads of 128
        dict(name="prompt_long", op="fwd", B=1, T=131072, H=16, Hk=16, Dk=128, Dv=128, dtype="bf16", s0=False, docs=0),
        # fp32 storage, groups of four heads sharing q and k, documents packed into rows
        dict(name="prompt_f32_shared", op="fwd", B=4, T=2000, H=16, Hk=4, Dk=64, Dv=128, dtype="f32", s0=True, docs=600),
        # a small training batch: ragged length, shared heads, unequal head sizes, packed documents
        dict(name="train_ragged", op="bwd", B=3, T=1531, H=8, Hk=2, Dk=96, Dv=64, dtype="bf16", s0=True, docs=400),
        # an ordinary training batch of one layer
        dict(name="train_batch", op="bwd", B=2, T=8192, H=16, Hk=16, Dk=128, Dv=128, dtype="bf16", s0=False, docs=0),
        # the answers of a small decode batch: log probability and eight alternatives a row
        dict(name="logp_decode", op="logp", N=4, V=32000, dtype="bf16", top=8, grad=False, mask=0),
        # scoring given text: fp32 logits of an odd vocabulary with masked entries
        dict(name="logp_score", op="logp", N=2048, V=50001, dtype="f32", top=5, grad=False, mask=37),
        # the loss of a training step with its gradient, the entropy's included
        dict(name="loss_train", op="logp", N=8192, V=32768, dtype="bf16", top=0, grad=True, mask=0),
        # gradients of one small layer
        dict(name="clip_small", op="clip", tensors=24, total=100003, max_norm=1.0),
        # gradients of a whole model, weights in bf16 and norms and biases in fp32
        dict(name="clip_large", op="clip", tensors=300, total=220000000, max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "fwd", "bwd", "logp", "logp", "clip"])
    if op == "logp":
        V, top, grad = _log(rng, 1000, 131072), rng.choice([0, 1, 5, 16, 32]), rng.random() < 0.5
        return dict(op="logp", N=_log(rng, 1, min(8192, 260000000 // V)), V=V, dtype=rng.choice(["bf16", "f32"]),
                    top=top, grad=grad, mask=rng.choice([0, 0, 3, 500]))
    if op == "clip":
        n = _log(rng, 1, 400)
        return dict(op="clip", tensors=n, total=max(n, _log(rng, 2000, 200000000)), max_norm=rng.choice([0.5, 1.0, 5.0]))
    Hk = rng.choice([1, 2, 4, 8, 16])
    H = Hk * rng.choice([1, 1, 1, 2, 4])
    c = dict(op=op, H=H, Hk=Hk, Dk=8 * rng.randint(2, 16), Dv=8 * rng.randint(2, 16),
             dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]))
    if op == "step":
        c["B"] = _log(rng, 1, max(1, 4000 // H))
        c["pool"] = c["B"] + rng.randint(0, 9)
        return c
    c["B"] = rng.choice([1, 1, 2, 3, 8])
    rows = 1000000 if op == "fwd" else 250000               # tokens times heads
    if c["dtype"] == "f32":
        rows //= 4
    c["T"] = _log(rng, 1, max(2, min(100000, rows // (H * c["B"]))))
    c["s0"], c["docs"] = rng.random() < 0.5, rng.choice([0, 0, 300])
    return c


def work(case):
    c = case
    if c["op"] == "logp":
        n, e = c["N"] * c["V"], 2 if c["dtype"] == "bf16" else 4
        return {"bytes": n * e * (2 if c["grad"] else 1) + c["N"] * (24 + 8 * c["top"]), "flops": n * (8 if c["grad"] else 4)}
    if c["op"] == "clip":
        b = sum(n * (2 if bf else 4) for n, bf in _tensors(c))
        return {"bytes": 2 * b + 8, "flops": 3 * c["total"]}
    e = 2 if c["dtype"] == "bf16" else 4
    rows = c["B"] * c.get("T", 1)
    qk, vo, st = rows * c["Hk"] * c["Dk"] * e, rows * c["H"] * c["Dv"] * e, c["B"] * c["H"] * c["Dk"] * c["Dv"] * 4
    mm = rows * c["H"] * c["Dk"] * c["Dv"]
    if c["op"] == "step":
        return {"bytes": 2 * qk + 2 * vo + 2 * st + rows * c["H"] * 4, "flops": 5 * mm}
    if c["op"] == "fwd":
        return {"bytes": 2 * qk + 2 * vo + st * (2 if c["s0"] else 1) + rows * c["H"] * 4, "flops": 4 * mm}
    return {"bytes": 4 * qk + 3 * vo + rows * c["H"] * 8 + st * (3 if c["s0"] else 0), "flops": 10 * mm}


# ---------------------------------------------------------------- inputs
def _tensors(c):
    """(values, bf16?) of every tensor: four matrices to each small vector, sizes uneven and odd."""
    n = c["tensors"]
    w = [0.001 * (1 + i % 3) if i % 5 == 4 else 1.0 + 0.37 * (i % 7) for i in range(n)]
    s = sum(w)
    sizes = [int(c["total"] * x / s) for x in w]
    sizes[0] += c["total"] - sum(sizes)
    return [(m, i % 5 != 4) for i, m in enumerate(sizes)]


def _inputs(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    def uniform(*s):
        return torch.rand(*s, device="cuda", generator=gen)

    if c["op"] == "clip":
        parts = _tensors(c)
        flat = {bf: (normal(sum(m for m, b in parts if b == bf)) * 0.01).to(torch.bfloat16 if bf else torch.float32)
                for bf in (True, False) if any(b == bf for _, b in parts)}
        grads, at = [], {True: 0, False: 0}
        for m, bf in parts:
            grads.append(flat[bf][at[bf]:at[bf] + m])
            at[bf] += m
        return {"grads": grads, "flat": flat}
    dt = _DT[c["dtype"]]
    if c["op"] == "logp":
        N, V = c["N"], c["V"]
        x = normal(N, V) * 2.0
        x[torch.arange(N, device="cuda"), (uniform(N) * V).long()] += 6.0          # a confident guess
        if c["mask"]:
            x[:, V - c["mask"]:] = -math.inf                                       # padding of the vocabulary
        y = (uniform(N) * (V - c["mask"])).long()
        y[uniform(N) < 0.05] = -1                                                   # tokens that are not scored
        s = {"logits": x.to(dt), "targets": y}
        if c["grad"]:
            s["glp"], s["gent"] = -(0.5 + uniform(N)) / N, 0.01 * normal(N) / N
        return s
    B, H, Hk, Dk, Dv = c["B"], c["H"], c["Hk"], c["Dk"], c["Dv"]
    lead = (B,) if c["op"] == "step" else (B, c["T"])
    s = {"q": normal(*lead, Hk, Dk).to(dt), "k": (normal(*lead, Hk, Dk) / math.sqrt(Dk)).to(dt),
         "v": normal(*lead, H, Dv).to(dt),
         "g": torch.log(torch.sigmoid(normal(*lead, H) + 3.0))}
    if c["op"] == "step":
        s["state"] = normal(c["pool"], H, Dk, Dv)
        s["slots"] = torch.randperm(c["pool"], device="cuda", generator=gen)[:B].int()
        return s
    if c["docs"]:                        # a document starts with an empty state: its first decay is zero
        s["g"].masked_fill_((uniform(B, c["T"]) < 1.0 / c["docs"])[..., None], -math.inf)
    s["s0"] = normal(B, H, Dk, Dv) if c["s0"] else None
    if c["op"] == "bwd":
        s["do"] = normal(*lead, H, Dv).to(dt)
        s["ds1"] = normal(B, H, Dk, Dv) if c["s0"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    c = s["case"] = dict(case)
    if c["op"] == "clip":
        s["out_flat"] = {bf: torch.zeros_like(x) for bf, x in s["flat"].items()}
        at, s["outs"] = {True: 0, False: 0}, []
        for m, bf in _tensors(c):
            s["outs"].append(s["out_flat"][bf][at[bf]:at[bf] + m])
            at[bf] += m
    if own:
        from adjoint_gradients_long_gb300 import lm
        bf = c.get("dtype") == "bf16"
        if c["op"] == "clip":
            s["plan"] = lm.GradClip(s["grads"], s["outs"])
        elif c["op"] == "logp":
            s["plan"] = lm.TokenLogProbs(c["N"], c["V"], x_bf16=bf, top=c["top"])
        elif c["op"] == "step":
            s["plan"] = lm.LinStep(c["B"], c["H"], c["Dk"], c["Dv"], Hk=c["Hk"], x_bf16=bf, scale=c["Dk"] ** -0.5)
        else:
            s["plan"] = lm.LinAttn(c["B"], c["T"], c["H"], c["Dk"], c["Dv"], Hk=c["Hk"], x_bf16=bf,
                                   scale=c["Dk"] ** -0.5, backward=c["op"] == "bwd")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    c, plan = s["case"], s["plan"]
    if c["op"] == "clip":
        norm, _ = plan.clip(c["max_norm"])
        return {"norm": norm, **{_NAME[bf]: x for bf, x in s["out_flat"].items()}}
    if c["op"] == "logp":
        if c["grad"]:
            r = plan.gradient(s["logits"], s["targets"], s["glp"], s["gent"])
        else:
            r = plan.forward(s["logits"], s["targets"])
        out = {"logp": r.logp, "entropy": r.entropy, "lse": r.lse}
        if c["top"]:
            out.update(top_id=r.top_id, top_logp=r.top_logp)
        if c["grad"]:
            out["dlogits"] = r.dlogits
        return out
    if c["op"] == "step":
        return {"o": plan.step(s["q"], s["k"], s["v"], s["g"], s["state"], s["slots"]), "state": s["state"]}
    if c["op"] == "fwd":
        o, s1 = plan.forward(s["q"], s["k"], s["v"], s["g"], s["s0"])
        return {"o": o, "s1": s1}
    dq, dk, dv, dg, ds0 = plan.backward(s["q"], s["k"], s["v"], s["g"], s["do"], s["s0"], s["ds1"])
    out = {"dq": dq, "dk": dk, "dv": dv, "dg": dg}
    if c["s0"]:
        out["ds0"] = ds0
    return out


def _run_plain(s):
    c = s["case"]
    if c["op"] == "clip":
        norm = torch.stack([x.float().square().sum() for x in s["grads"]]).sum().sqrt()
        coef = (c["max_norm"] / (norm + EPS)).clamp(max=1.0)
        [y.copy_(x.float() * coef) for x, y in zip(s["grads"], s["outs"])]
        return {"norm": norm, **{_NAME[bf]: x for bf, x in s["out_flat"].items()}}
    if c["op"] == "logp":
        return _plain_logp(c, s)
    if c["op"] == "step":
        return _plain_step(c, s)
    q, k, v, g = (s[n].float() for n in ("q", "k", "v", "g"))
    s0 = s["s0"] if c["s0"] else torch.zeros(c["B"], c["H"], c["Dk"], c["Dv"], device=q.device)
    if c["op"] == "fwd":
        o, s1 = _plain_lin(c, q, k, v, g, s0)
        return {"o": o.to(s["v"].dtype), "s1": s1}
    leaves = [x.detach().clone().requires_grad_() for x in (q, k, v, g, s0)]
    o, s1 = _plain_lin(c, *leaves)
    loss = (o * s["do"].float()).sum()
    if c["s0"]:
        loss = loss + (s1 * s["ds1"]).sum()
    dq, dk, dv, dg, ds0 = torch.autograd.grad(loss, leaves)
    out = {"dq": dq.to(s["q"].dtype), "dk": dk.to(s["q"].dtype), "dv": dv.to(s["q"].dtype), "dg": dg}
    if c["s0"]:
        out["ds0"] = ds0
    return out


def _plain_logp(c, s):
    x, y = s["logits"].float(), s["targets"]
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    lse = m + torch.log(z)
    p = e / z
    lp = x - lse
    plp = torch.where(p > 0, p * lp, 0.0)
    ent = -plp.sum(-1)
    scored = (y >= 0) & (y < c["V"])
    at = torch.where(scored, y, 0)
    logp = torch.where(scored, lp.gather(-1, at[:, None])[:, 0], 0.0)
    out = {"logp": logp, "entropy": ent, "lse": lse[:, 0]}
    if c["top"]:
        i = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :c["top"]]
        out.update(top_id=i.int(), top_logp=lp.gather(-1, i))
    if c["grad"]:
        gl = torch.where(scored, s["glp"], 0.0)
        d = -gl[:, None] * p - s["gent"][:, None] * (plp + p * ent[:, None])
        d.scatter_add_(-1, at[:, None], gl[:, None])
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


def _plain_step(c, s):
    r = c["H"] // c["Hk"]
    q, k, v = s["q"].float().repeat_interleave(r, 1), s["k"].float().repeat_interleave(r, 1), s["v"].float()
    at = s["slots"].long()
    S = s["state"][at] * torch.exp(s["g"])[..., None, None] + k[..., :, None] * v[..., None, :]
    s["state"][at] = S
    o = (q[..., :, None] * S).sum(-2) * c["Dk"] ** -0.5
    return {"o": o.to(s["v"].dtype), "state": s["state"]}


def _segment_sums(x):
    """L[..., i, j] = sum of x over (j, i], minus infinity for j > i."""
    n = x.shape[-1]
    below = torch.ones(n, n, dtype=torch.bool, device=x.device).tril(-1)
    L = x[..., :, None].expand(*x.shape, n).masked_fill(~below, 0.0).cumsum(-2)
    return L.masked_fill(below.T, -math.inf)


def _plain_lin(c, q, k, v, g, s0, C=64):
    """The chunked form: pairs inside a chunk of C tokens, and states carried between chunks by
    the matrix of the decays between them."""
    B, T, H, Dk, Dv = c["B"], c["T"], c["H"], c["Dk"], c["Dv"]
    n, r = -(-T // C), H // c["Hk"]

    def chunks(x, rep=1):
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * C - T))
        x = x.repeat_interleave(rep, 2) if rep > 1 else x
        return x.reshape(B, n, C, H, x.shape[-1]).permute(0, 3, 1, 2, 4)

    q, k, v = chunks(q, r), chunks(k, r), chunks(v)
    g = chunks(g[..., None])[..., 0]
    D = torch.exp(_segment_sums(g))
    intra = ((q @ k.transpose(-1, -2)) * D) @ v
    U = (k * D[..., -1, :, None]).transpose(-1, -2) @ v
    G = g.cumsum(-1)
    U = torch.cat([s0[:, :, None], U], 2).reshape(B, H, n + 1, Dk * Dv)
    between = torch.exp(_segment_sums(torch.nn.functional.pad(G[..., -1], (1, 0))))
    S = (between @ U).reshape(B, H, n + 1, Dk, Dv)
    inter = (q * torch.exp(G)[..., None]) @ S[:, :, :n]
    o = ((intra + inter) * Dk ** -0.5).permute(0, 2, 3, 1, 4).reshape(B, n * C, H, Dv)[:, :T]
    return o, S[:, :, n]


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    if c["op"] == "clip":
        norm = math.sqrt(sum(float(x.double().pow(2).sum()) for x in s["grads"] if x.numel()))
        f = min(1.0, c["max_norm"] / (norm + EPS))
        return {"norm": torch.tensor(norm, dtype=torch.float64),
                **{_NAME[bf]: x.double() * f for bf, x in s["flat"].items()}}
    if c["op"] == "logp":
        return _exact_logp(c, s)
    if c["op"] == "step":
        S, o, r = s["state"].double(), [], c["H"] // c["Hk"]
        for b in range(c["B"]):
            i = int(s["slots"][b])
            q, k = (s[n][b].double().repeat_interleave(r, 0) for n in ("q", "k"))
            S[i] = torch.exp(s["g"][b].double())[:, None, None] * S[i] + torch.einsum("hd,he->hde", k, s["v"][b].double())
            o.append(torch.einsum("hd,hde->he", q, S[i]) / math.sqrt(c["Dk"]))
        return {"o": torch.stack(o), "state": S}
    return _exact_lin(c, s)


def _exact_logp(c, s):
    N, V = c["N"], c["V"]
    out = {n: [] for n in ("logp", "entropy", "lse", "top_logp", "dlogits")}
    for a in range(0, N, 512):                                   # rows at a time, to bound the memory
        x, y = s["logits"][a:a + 512].double(), s["targets"][a:a + 512]
        lse = torch.logsumexp(x, -1)
        lp = x - lse[:, None]
        p = torch.exp(lp)
        ent = torch.special.entr(p).sum(-1)
        ok = y >= 0
        hot = torch.zeros_like(x)
        hot[ok.nonzero()[:, 0], y[ok]] = 1.0
        out["logp"].append(torch.where(ok, x.gather(-1, y.clamp(min=0)[:, None])[:, 0] - lse, 0.0))
        out["entropy"].append(ent)
        out["lse"].append(lse)
        if c["top"]:
            out["top_logp"].append(torch.topk(lp, c["top"], -1).values)
        if c["grad"]:
            gl = (s["glp"][a:a + 512].double() * ok)[:, None]
            d = gl * (hot - p) + s["gent"][a:a + 512].double()[:, None] * (torch.special.entr(p) - p * ent[:, None])
            out["dlogits"].append(d)
    got = {n: torch.cat(v) for n, v in out.items() if v}
    if c["top"]:
        got["top_id"] = None
    return got


def _exact_lin(c, s, C=128):
    """Block by block: the pairs of a block by the sums of their decays, the rest by the state
    that enters it; the gradient by the adjoint state, blocks taken from the last one back."""
    B, T, H, Dk, Dv = c["B"], c["T"], c["H"], c["Dk"], c["Dv"]
    r, scale = H // c["Hk"], 1.0 / math.sqrt(Dk)

    def block(n, a, rep):
        x = s[n][:, a:a + C].double()
        return x.repeat_interleave(rep, 2).transpose(1, 2)

    def decays(a):
        g = s["g"][:, a:a + C].double().transpose(1, 2)           # [B, H, c]
        cut = torch.isinf(g)
        G, seg = torch.where(cut, 0.0, g).cumsum(-1), cut.cumsum(-1)
        n = G.shape[-1]
        pair = torch.ones(n, n, dtype=torch.bool, device=g.device).tril() & (seg[..., :, None] == seg[..., None, :])
        D = torch.where(pair, torch.exp((G[..., :, None] - G[..., None, :]).clamp(max=0)), 0.0)
        first = torch.where(seg == 0, torch.exp(G), 0.0)          # from before the block to each token
        last = D[..., -1, :]                                      # from each token to the block's end
        return D, first, last, cut

    S = s["s0"].double() if c["s0"] else torch.zeros(B, H, Dk, Dv, dtype=torch.float64, device=s["q"].device)
    outs, states = [], []
    for a in range(0, T, C):
        q, k, v = block("q", a, r), block("k", a, r), block("v", a, 1)
        D, first, last, _ = decays(a)
        if c["op"] == "fwd":
            o = (torch.einsum("bhid,bhjd->bhij", q, k) * D) @ v + first[..., None] * (q @ S)
            outs.append((o * scale).transpose(1, 2))
        else:
            states.append(S)
        S = first[..., -1, None, None] * S + torch.einsum("bhj,bhjd,bhje->bhde", last, k, v)
    if c["op"] == "fwd":
        return {"o": torch.cat(outs, 1), "s1": S}
    dS = s["ds1"].double() if c["s0"] else torch.zeros_like(S)
    grads = []
    for a in reversed(range(0, T, C)):
        q, k, v, do = block("q", a, r), block("k", a, r), block("v", a, 1), block("do", a, 1) * scale
        D, first, last, cut = decays(a)
        S0 = states.pop()
        R = (do @ v.transpose(-1, -2)) * D
        P = (q @ k.transpose(-1, -2)) * D
        dq = R @ k + first[..., None] * (do @ S0.transpose(-1, -2))
        dk = R.transpose(-1, -2) @ q + last[..., None] * (v @ dS.transpose(-1, -2))
        dv = P.transpose(-1, -2) @ do + last[..., None] * (k @ dS)
        dG = (q * dq).sum(-1) - (k * dk).sum(-1)
        dg = dG.flip(-1).cumsum(-1).flip(-1) + (dS * S).sum((-1, -2))[..., None]
        dg = torch.where(cut, 0.0, dg)
        if a == 0 and not c["s0"]:
            dg[..., 0] = 0.0                                      # the first decay meets an empty state
        n = dq.shape[-2]
        share = lambda x: x.transpose(1, 2).reshape(B, n, c["Hk"], r, Dk).sum(3)  # noqa: E731
        grads.append((share(dq), share(dk), dv.transpose(1, 2), dg.transpose(1, 2)))
        dS = first[..., -1, None, None] * dS + torch.einsum("bhi,bhid,bhie->bhde", first, q, do)
        S = S0
    dq, dk, dv, dg = (torch.cat([x[n] for x in reversed(grads)], 1) for n in range(4))
    out = {"dq": dq, "dk": dk, "dv": dv, "dg": dg}
    if c["s0"]:
        out["ds0"] = dS
    return out
