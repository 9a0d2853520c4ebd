"""The measured cases of what stands around a recurrent layer: its short causal convolution and its
selective scan (prompts with states and packed sequences, gradients, single tokens), and sampling the
next token with temperature, top-k, top-p and min-p from given random numbers.

`run` computes them in their plain form (elementary torch operations in 32 bits; sampling, where a
token hangs on a border between two sums, in 64) or, with `own` set, by the calls of
adjoint_gradients_long_gb300.lm.  `exact` gives the same results in 64 bits from the definitions,
token by token, written apart from the plain form.
"""
import math

import torch

own = False

UNIT = 2.0 ** 40                     # weight of the likeliest token in the sampler's whole numbers
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a full serving batch, states in a pool of slots: the convolution's last inputs are shifted by one
        dict(name="conv_step", op="conv_step", B=256, P=2048, W=4, dtype="bf16", pool=300),
        # a batch of prompts of different lengths packed one behind the other, continued from stored states
        dict(name="conv_prompts", op="conv_fwd", B=24, T=32768, P=2048, W=4, dtype="bf16", packed=True, s0=True, act=True),
        # an ordinary training batch of one layer
        dict(name="conv_train", op="conv_bwd", B=8, T=2048, P=2048, W=4, dtype="bf16", packed=False, s0=False, act=True),
        # one sequence being answered: latency only
        dict(name="scan_step_one", op="scan_step", B=1, P=2048, N=16, dtype="bf16", pool=1, gate=True),
        # a full serving batch whose states lie scattered in a pool of slots
        dict(name="scan_step_batch", op="scan_step", B=256, P=2048, N=16, dtype="bf16", pool=300, gate=True),
        # a short follow-up prompt that continues from a stored state
        dict(name="scan_prompt_short", op="scan_fwd", B=1, T=77, P=2048, N=16, dtype="bf16", packed=False, s0=True, gate=True),
        # a whole long context of one layer
        dict(name="scan_prompt_long", op="scan_fwd", B=1, T=65536, P=1024, N=16, dtype="bf16", packed=False, s0=False, gate=True),
        # a small training batch: fp32, packed documents of uneven length, a channel count that fills no tile
        dict(name="scan_train_ragged", op="scan_bwd", B=5, T=1531, P=200, N=8, dtype="f32", packed=True, s0=True, gate=False),
        # an ordinary training batch of one layer
        dict(name="scan_train_batch", op="scan_bwd", B=2, T=8192, P=2048, N=16, dtype="bf16", packed=False, s0=False, gate=True),
        # the next token of one answer
        dict(name="sample_one", op="sample", N=1, V=32000, dtype="bf16", mix="usual", mask=0),
        # a decode batch whose requests each have their own settings, an odd vocabulary with masked entries
        dict(name="sample_batch", op="sample", N=256, V=50001, dtype="f32", mix="each", mask=37),
        # the widest vocabulary, top-p alone: nothing short of the whole row says where it ends
        dict(name="sample_wide", op="sample", N=64, V=131072, dtype="bf16", mix="top_p", mask=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step",
                     "sample", "sample", "sample"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "sample":
        V = _log(rng, 100, 131072)
        return dict(op=op, N=_log(rng, 1, min(512, 8000000 // V)), V=V, dtype=dtype,
                    mix=rng.choice(["usual", "each", "each", "top_p", "plain"]), mask=rng.choice([0, 0, 3, 50]))
    c = dict(op=op, P=8 * _log(rng, 1, 256), dtype=dtype)
    if op.startswith("conv"):
        c["W"] = rng.choice([2, 3, 4, 4])
    else:
        c["N"], c["gate"] = rng.choice([8, 16, 16, 32, 64]), rng.random() < 0.6
    if op.endswith("step"):
        c["B"] = _log(rng, 1, 256)
        c["pool"] = c["B"] + rng.randint(0, 9)
        return c
    # tokens: as many values as the largest case of the same direction, fewer in fp32
    most = {"conv_fwd": 60e6, "conv_bwd": 30e6, "scan_fwd": 0.8e9, "scan_bwd": 0.3e9}[op]
    rows = most / (c["P"] * c.get("N", 1) * (2 if dtype == "f32" else 1))
    tokens = _log(rng, 1, max(2, min(30000 if op == "scan_fwd" else 8000, rows)))
    c["packed"] = rng.random() < 0.5
    if c["packed"]:
        c["B"], c["T"] = _log(rng, 1, 40), tokens
    else:
        c["B"] = rng.choice([1, 1, 2, 3, 8])
        c["T"] = max(1, tokens // c["B"])
    c["s0"] = rng.random() < 0.5
    if op.startswith("conv"):
        c["act"] = rng.random() < 0.8
    return c


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "sample":
        return {"bytes": c["N"] * (c["V"] * e + 32), "flops": 8 * c["N"] * c["V"]}
    P, B = c["P"], c["B"]
    if c["op"].endswith("step"):
        if c["op"] == "conv_step":
            return {"bytes": B * P * e * 2 * c["W"] + P * (c["W"] + 1) * 4, "flops": B * P * (2 * c["W"] + 5)}
        vec = B * P * e * (4 if c["gate"] else 3) + 2 * B * c["N"] * e
        return {"bytes": vec + 8 * B * P * c["N"] + P * (c["N"] + 2) * 4, "flops": B * P * (7 * c["N"] + 12)}
    R = c["T"] if c["packed"] else c["B"] * c["T"]
    if c["op"].startswith("conv"):
        st = B * (c["W"] - 1) * P * e if c["s0"] else 0
        if c["op"] == "conv_fwd":
            return {"bytes": 2 * R * P * e + 2 * st + P * (c["W"] + 1) * 4, "flops": R * P * (2 * c["W"] + 5)}
        return {"bytes": 3 * R * P * e + 3 * st + 2 * P * (c["W"] + 1) * 4, "flops": R * P * (6 * c["W"] + 12)}
    N, st, par = c["N"], B * P * c["N"] * 4, P * (c["N"] + 2) * 4
    if c["op"] == "scan_fwd":
        return {"bytes": R * P * e * (4 if c["gate"] else 3) + 2 * R * N * e + st * (2 if c["s0"] else 1) + par,
                "flops": R * P * (7 * N + 12)}
    return {"bytes": R * P * e * (7 if c["gate"] else 5) + 4 * R * N * e + st * (3 if c["s0"] else 0) + 2 * par,
            "flops": R * P * (22 * N + 30)}


# ---------------------------------------------------------------- inputs
def _offsets(c, gen):
    """Where the sequences begin, and the end of the last: B + 1 whole numbers from 0 to the tokens."""
    if not c["packed"]:
        return torch.arange(c["B"] + 1, device="cuda") * c["T"]
    cuts = (torch.rand(c["B"] - 1, device="cuda", generator=gen) * (c["T"] + 1)).long().sort().values
    return torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), c["T"])])


def _inputs(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    def uniform(*s):
        return torch.rand(*s, device="cuda", generator=gen)

    dt = _DT[c["dtype"]]
    if c["op"] == "sample":
        N, V = c["N"], c["V"]
        x = normal(N, V) * 2.0
        x[torch.arange(N, device="cuda"), (uniform(N) * V).long().clamp(max=V - 1)] += 6.0     # a confident guess
        if c["mask"]:
            x[:, V - c["mask"]:] = -math.inf                                     # padding of the vocabulary
        s = {"logits": x.to(dt), "u": uniform(N)}
        pick = lambda *v: torch.tensor(v, device="cuda")[(uniform(N) * len(v)).long().clamp(max=len(v) - 1)]  # noqa: E731
        if c["mix"] == "usual":
            s["temperature"], s["top_k"], s["top_p"] = pick(0.8), pick(50).int(), pick(0.95)
        elif c["mix"] == "top_p":
            s["temperature"], s["top_p"] = pick(1.0, 1.2), pick(0.9, 0.99)
        elif c["mix"] == "each":
            s["temperature"] = pick(0.0, 0.6, 0.8, 1.0, 1.5)
            s["top_k"] = pick(0, 1, 20, 50, 1000).int()
            s["top_p"], s["min_p"] = pick(0.5, 0.9, 0.95, 1.0), pick(0.0, 0.0, 0.02, 0.1)
        return s
    P, B = c["P"], c["B"]
    step = c["op"].endswith("step")
    lead = (B,) if step else (c["T"],) if c["packed"] else (B, c["T"])
    s = {}
    if not step:
        s["offsets"] = _offsets(c, gen)
    else:
        s["slots"] = torch.randperm(c["pool"], device="cuda", generator=gen)[:B].int()
    if c["op"].startswith("conv"):
        W = c["W"]
        s["x"] = normal(*lead, 2 * P).to(dt)[..., :P]                            # half of a projection
        s["w"], s["bias"] = (uniform(P, W) * 2 - 1) / math.sqrt(W), (uniform(P) * 2 - 1) / math.sqrt(W)
        if step:
            s["state"] = normal(c["pool"], W - 1, P).to(dt)
            return s
        s["s0"] = normal(B, W - 1, P).to(dt) if c["s0"] else None
        if c["op"] == "conv_bwd":
            s["go"] = normal(*lead, P).to(dt)
            s["ds1"] = normal(B, W - 1, P).to(dt) if c["s0"] else None
        return s
    N = c["N"]
    s["x"] = normal(*lead, P).to(dt)
    parts = (normal(*lead, P + 2 * N) * 0.7).to(dt)                              # one projection: dt, B, C
    s["dt"], s["Bm"], s["Cm"] = parts[..., :P], parts[..., P:P + N], parts[..., P + N:]
    s["z"] = normal(*lead, P).to(dt) if c["gate"] else None
    # steps between 0.001 and 0.1, decays of one to N of them a token, as such layers begin with
    rate = torch.exp(math.log(0.001) + uniform(P) * math.log(100.0))
    s["dt_bias"] = rate + torch.log(-torch.expm1(-rate))
    s["A"] = -(torch.arange(N, device="cuda") + 1.0) * (0.8 + 0.4 * uniform(P, N))
    s["D"] = 1.0 + 0.1 * normal(P)
    if step:
        s["state"] = normal(c["pool"], P, N)
        return s
    s["s0"] = normal(B, P, N) if c["s0"] else None
    if c["op"] == "scan_bwd":
        s["go"] = normal(*lead, P).to(dt)
        s["ds1"] = normal(B, P, N) if c["s0"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    c = s["case"] = dict(case)
    if own:
        from adjoint_gradients_long_gb300 import lm
        bf = c["dtype"] == "bf16"
        if c["op"] == "sample":
            s["plan"] = lm.Sampler(c["N"], c["V"], x_bf16=bf)
        elif c["op"] == "conv_step":
            s["plan"] = lm.ShortConvStep(c["B"], c["P"], c["W"], x_bf16=bf)
        elif c["op"] == "scan_step":
            s["plan"] = lm.SelScanStep(c["B"], c["P"], c["N"], x_bf16=bf)
        elif c["op"].startswith("conv"):
            s["plan"] = lm.ShortConv(c["B"], c["T"], c["P"], c["W"], x_bf16=bf, act=c["act"], packed=c["packed"],
                                     backward=c["op"] == "conv_bwd")
        else:
            s["plan"] = lm.SelScan(c["B"], c["T"], c["P"], c["N"], x_bf16=bf, packed=c["packed"],
                                   backward=c["op"] == "scan_bwd")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    c, plan = s["case"], s["plan"]
    if c["op"] == "sample":
        token, logp = plan.sample(s["logits"], s["u"], s.get("temperature"), s.get("top_k"), s.get("top_p"), s.get("min_p"))
        return {"token": token, "logp": logp}
    if c["op"] == "conv_step":
        return {"y": plan.step(s["x"], s["w"], s["state"], s["bias"], s["slots"]), "state": s["state"]}
    if c["op"] == "scan_step":
        y = plan.step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["state"], s["D"], s["z"], s["dt_bias"], s["slots"])
        return {"y": y, "state": s["state"]}
    off = s["offsets"] if c["packed"] else None
    if c["op"] == "conv_fwd":
        y, s1 = plan.forward(s["x"], s["w"], s["bias"], s["s0"], off)
        return {"y": y, "s1": s1}
    if c["op"] == "conv_bwd":
        dx, dw, dbias, ds0 = plan.backward(s["x"], s["w"], s["go"], s["bias"], s["s0"], s["ds1"], off)
        out = {"dx": dx, "dw": dw, "dbias": dbias}
        if c["s0"]:
            out["ds0"] = ds0
        return out
    at = s["x"], s["dt"], s["A"], s["Bm"], s["Cm"]
    if c["op"] == "scan_fwd":
        y, s1 = plan.forward(*at, s["D"], s["z"], s["dt_bias"], s["s0"], off)
        return {"y": y, "s1": s1}
    r = plan.backward(*at, s["go"], s["D"], s["z"], s["dt_bias"], s["s0"], s["ds1"], off)
    out = {"dx": r.dx, "ddt": r.ddt, "dA": r.dA, "dB": r.dB, "dC": r.dC, "dD": r.dD, "ddt_bias": r.ddt_bias}
    if c["gate"]:
        out["dz"] = r.dz
    if c["s0"]:
        out["ds0"] = r.ds0
    return out


def _run_plain(s):
    c = s["case"]
    if c["op"] == "sample":
        return _plain_sample(c, s)
    if c["op"] == "conv_step":
        at, dt = s["slots"].long(), s["x"].dtype
        taps = torch.cat([s["state"][at], s["x"][:, None]], 1)
        p = s["bias"] + (taps.float() * s["w"].T).sum(1)
        s["state"][at] = taps[:, 1:]
        return {"y": (p * torch.sigmoid(p)).to(dt), "state": s["state"]}
    if c["op"] == "scan_step":
        at = s["slots"].long()
        x, d = s["x"].float(), _softplus(s["dt"].float() + s["dt_bias"])
        h = torch.exp(d[..., None] * s["A"]) * s["state"][at] + (d * x)[..., None] * s["Bm"].float()[:, None]
        s["state"][at] = h
        v = (h * s["Cm"].float()[:, None]).sum(-1) + s["D"] * x
        return {"y": _gated(c, v, s["z"]).to(s["x"].dtype), "state": s["state"]}
    if c["op"].startswith("conv"):
        return _plain_conv(c, s)
    return _plain_scan(c, s)


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _gated(c, v, z):
    return v * (z.float() * torch.sigmoid(z.float())) if c["gate"] else v


def _sequences(s, rows):
    """For every token its sequence, and whether it is the first or the last one of it."""
    off = s["offsets"]
    t = torch.arange(rows, device=off.device)
    seq = torch.searchsorted(off, t, right=True) - 1
    return seq, t == off[seq], t + 1 == off[seq + 1]


def _plain_conv(c, s):
    """Taps gathered from one long list: the tokens, the stored states, and a row of zeros."""
    B, P, W, dt = c["B"], c["P"], c["W"], s["x"].dtype
    x = s["x"].reshape(-1, P)
    R, off = x.shape[0], s["offsets"]
    s0 = s["s0"] if c["s0"] else x.new_zeros(B, W - 1, P)
    rows = torch.cat([x, s0.reshape(-1, P)]).float()
    seq, _, _ = _sequences(s, R)

    def at(seq, i):
        """Row of entry i of a sequence's list: its state (i < W - 1), then its tokens."""
        return torch.where(i < W - 1, R + seq * (W - 1) + i, off[seq] + i - (W - 1))

    here = torch.arange(R, device=x.device) - off[seq]
    tap = [at(seq, here + j) for j in range(W)]
    p = s["bias"].expand(R, P).clone()
    for j in range(W):
        p += s["w"][:, j] * rows[tap[j]]
    b = torch.arange(B, device=x.device)
    last = at(b[:, None], (off[1:] - off[:-1])[:, None] + torch.arange(W - 1, device=x.device))
    if c["op"] == "conv_fwd":
        y = p * torch.sigmoid(p) if c["act"] else p
        return {"y": y.to(dt).reshape(s["x"].shape), "s1": rows[last].to(dt)}
    dp = s["go"].reshape(-1, P).float()
    if c["act"]:
        g = torch.sigmoid(p)
        dp = dp * (g * (1 + p * (1 - g)))
    d = torch.zeros_like(rows)
    dw = torch.empty_like(s["w"])
    for j in range(W):
        d[tap[j]] += s["w"][:, j] * dp
        dw[:, j] = (dp * rows[tap[j]]).sum(0)
    if c["s0"]:
        for i in range(W - 1):
            d[last[:, i]] += s["ds1"][:, i].float()
    out = {"dx": d[:R].to(dt).reshape(s["x"].shape), "dw": dw, "dbias": dp.sum(0)}
    if c["s0"]:
        out["ds0"] = d[R:].to(dt).reshape(B, W - 1, P)
    return out


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t from zero over the first dimension: in blocks side by side, then from
    block to block."""
    T = a.shape[0]
    C = 1 << (T.bit_length() // 2)
    n = -(-T // C)
    if n * C > T:
        tail = a.new_zeros(n * C - T, *a.shape[1:])
        a, b = torch.cat([a, tail]), torch.cat([b, tail])
    a, b = a.reshape(n, C, *a.shape[1:]), b.reshape(n, C, *b.shape[1:])
    h, p = torch.empty_like(b), torch.empty_like(a)
    h[:, 0], p[:, 0] = b[:, 0], a[:, 0]
    for i in range(1, C):
        torch.addcmul(b[:, i], a[:, i], h[:, i - 1], out=h[:, i])
        torch.mul(a[:, i], p[:, i - 1], out=p[:, i])
    enter = torch.zeros_like(h[:, 0])
    for j in range(1, n):
        enter[j] = p[j - 1, -1] * enter[j - 1] + h[j - 1, -1]
    h += p * enter[:, None]
    return h.reshape(n * C, *h.shape[2:])[:T]


def _plain_scan(c, s):
    B, P, N, dt = c["B"], c["P"], c["N"], s["x"].dtype
    shape = s["x"].shape
    x, raw = s["x"].reshape(-1, P).float(), s["dt"].reshape(-1, P).float() + s["dt_bias"]
    Bm, Cm = s["Bm"].reshape(-1, N).float(), s["Cm"].reshape(-1, N).float()
    R, off = x.shape[0], s["offsets"]
    z = s["z"].reshape(-1, P).float() if c["gate"] else None
    s0 = s["s0"] if c["s0"] else x.new_zeros(B, P, N)
    seq, first, last = _sequences(s, R)
    d = _softplus(raw)
    a = torch.exp(d[..., None] * s["A"])
    b = (d * x)[..., None] * Bm[:, None]
    b[first] += a[first] * s0[seq[first]]
    cut = a.clone()
    cut[first] = 0.0                                   # nothing comes in from the sequence before
    h = _recur(cut, b)
    del b
    v = (h * Cm[:, None]).sum(-1) + s["D"] * x
    if c["op"] == "scan_fwd":
        s1 = s0.clone()
        s1[seq[last]] = h[last]
        return {"y": _gated(c, v, z).to(dt).reshape(shape), "s1": s1}
    g = s["go"].reshape(-1, P).float()
    out = {}
    if c["gate"]:
        sg = torch.sigmoid(z)
        out["dz"] = (g * v * sg * (1 + z * (1 - sg))).to(dt).reshape(shape)
        g = g * z * sg
    src = g[..., None] * Cm[:, None]
    if c["s0"]:
        src[last] += s["ds1"][seq[last]]
    nxt = torch.cat([cut[1:], cut.new_zeros(1, P, N)])
    m = _recur(nxt.flip(0), src.flip(0)).flip(0)
    del nxt, src, cut
    out["dC"] = (g[..., None] * h).sum(1).to(dt).reshape(*shape[:-1], N)
    out["dB"] = (m * (d * x)[..., None]).sum(1).to(dt).reshape(*shape[:-1], N)
    mb = (m * Bm[:, None]).sum(-1)
    out["dx"] = (d * mb + s["D"] * g).to(dt).reshape(shape)
    out["dD"] = (g * x).sum(0)
    m *= a                                             # what reaches the state before
    if c["s0"]:
        ds0 = s["ds1"].clone()
        ds0[seq[first]] = m[first]
        out["ds0"] = ds0
    before = torch.cat([h.new_zeros(1, P, N), h[:-1]])
    before[first] = s0[seq[first]]
    m *= before
    out["dA"] = (m * d[..., None]).sum(0)
    ddt = (x * mb + (m * s["A"]).sum(-1)) * torch.sigmoid(raw)
    out["ddt"], out["ddt_bias"] = ddt.to(dt).reshape(shape), ddt.sum(0)
    return out


def _plain_sample(c, s):
    N, V = c["N"], c["V"]
    x = s["logits"].double()
    row = lambda n, off: s[n].double()[:, None] if n in s else x.new_full((N, 1), off)  # noqa: E731
    T, top_p, min_p = row("temperature", 1.0), row("top_p", 1.0), row("min_p", 0.0)
    top_k = s["top_k"].long()[:, None] if "top_k" in s else torch.zeros(N, 1, dtype=torch.long, device=x.device)
    m = x.amax(-1, keepdim=True)
    greedy = T == 0
    far = (x - m) / torch.where(greedy, 1.0, T)
    w = torch.round(torch.exp(far) * UNIT).long()
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, torch.arange(V, device=x.device).expand(N, V))
    keep = w.double() >= min_p * UNIT
    keep &= (rank < top_k) | (top_k <= 0)
    keep &= (rank < 1) | ~greedy
    w = torch.where(keep, w, 0)
    sorted_w = w.gather(-1, order)
    before = sorted_w.cumsum(-1) - sorted_w
    nucleus = (before.double() < top_p * w.sum(-1, keepdim=True).double()) | (top_p >= 1)
    w = torch.where(nucleus.gather(-1, rank), w, 0)
    Z = w.sum(-1, keepdim=True)
    past = w.cumsum(-1).double() > s["u"].double()[:, None] * Z.double()
    token = past.int().argmax(-1)
    logp = far.gather(-1, token[:, None]) - torch.log(Z.double() / UNIT)
    return {"token": token, "logp": logp[:, 0].float()}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    if c["op"] == "sample":
        return _exact_sample(c, s)
    if c["op"] == "conv_step":
        at, y = s["slots"].long(), []
        state = s["state"].double()
        for b in range(c["B"]):
            taps = torch.cat([state[at[b]], s["x"][b:b + 1].double()])
            p = s["bias"].double() + torch.einsum("jp,pj->p", taps, s["w"].double())
            y.append(p / (1 + torch.exp(-p)))
            state[at[b]] = taps[1:]
        return {"y": torch.stack(y), "state": state}
    if c["op"].startswith("conv"):
        return _exact_conv(c, s)
    return _exact_scan(c, s)


def _exact_conv(c, s):
    """Each sequence alone: its state and tokens in one list, gradients by automatic differentiation."""
    B, P, W = c["B"], c["P"], c["W"]
    off = s["offsets"].tolist()
    grad = c["op"] == "conv_bwd"
    x = s["x"].reshape(-1, P).double().requires_grad_(grad)
    s0 = (s["s0"].double() if c["s0"] else x.new_zeros(B, W - 1, P).detach()).requires_grad_(grad)
    w, bias = s["w"].double().requires_grad_(grad), s["bias"].double().requires_grad_(grad)
    ys, s1 = [], []
    for b in range(B):
        n = off[b + 1] - off[b]
        rows = torch.cat([s0[b], x[off[b]:off[b + 1]]])
        p = bias + sum(rows[j:j + n] * w[:, j] for j in range(W))
        ys.append(p / (1 + torch.exp(-p)) if c["act"] else p)
        s1.append(rows[n:])
    y, s1 = torch.cat(ys), torch.stack(s1)
    if not grad:
        return {"y": y.reshape(s["x"].shape), "s1": s1}
    loss = (y * s["go"].reshape(-1, P).double()).sum()
    if c["s0"]:
        loss = loss + (s1 * s["ds1"].double()).sum()
    dx, dw, dbias, ds0 = torch.autograd.grad(loss, (x, w, bias, s0))
    out = {"dx": dx.reshape(s["x"].shape), "dw": dw, "dbias": dbias}
    if c["s0"]:
        out["ds0"] = ds0
    return out


def _exact_scan(c, s):
    """Token by token: all sequences of a batch at once, packed ones one after the other."""
    B, P, N = c["B"], c["P"], c["N"]
    if c["op"] != "scan_step" and (c["T"] > 70000 or (c["op"] == "scan_bwd" and c["T"] * P * N * (1 if c["packed"] else B) > 6e8)):
        return None
    A, D, bias = s["A"].double(), s["D"].double(), s["dt_bias"].double()
    step = c["op"] == "scan_step"
    if step:
        at = s["slots"].long()
        start, runs, lead = s["state"].double()[at], [(None, 0, 1)], (B, 1)
    else:
        start = s["s0"].double() if c["s0"] else torch.zeros(B, P, N, dtype=torch.float64, device="cuda")
        off = s["offsets"].tolist()
        runs = [(b, off[b], off[b + 1]) for b in range(B)] if c["packed"] else [(None, 0, c["T"])]
        lead = (1, c["T"]) if c["packed"] else (B, c["T"])
    get = lambda n: s[n].reshape(*lead, -1)  # noqa: E731
    xs, dts, Bs, Cs = (get(n) for n in ("x", "dt", "Bm", "Cm"))
    zs = get("z").double() if c["gate"] else None
    # softplus from both sides of zero: log(1 + e^v), which loses nothing in 64 bits below 30
    v = dts.double() + bias
    ds = torch.where(v > 30, v, torch.log(1 + torch.exp(v.clamp(max=30))))
    grad = c["op"] == "scan_bwd"
    vs, end = torch.zeros(*lead, P, dtype=torch.float64, device="cuda"), start.clone()
    hist = torch.zeros(lead[1], lead[0], P, N, dtype=torch.float64, device="cuda") if grad else None
    for b, t0, t1 in runs:
        rows = slice(None) if b is None else slice(b, b + 1)
        h = start[rows]
        for t in range(t0, t1):
            if grad:
                hist[t] = h
            d = ds[:, t]
            h = torch.exp(d[..., None] * A) * h
            h += (d * xs[:, t].double())[..., None] * Bs[:, t, None].double()
            vs[:, t] = torch.einsum("bpn,bn->bp", h, Cs[:, t].double())
        end[rows] = h
    x = xs.double()
    vs += D * x
    if not grad:
        y = vs * zs / (1 + torch.exp(-zs)) if c["gate"] else vs
        if step:
            state = s["state"].double()
            state[at] = end
            return {"y": y[:, 0], "state": state}
        return {"y": y.reshape(s["x"].shape), "s1": end}
    go = get("go").double()
    out, g = {}, go
    if c["gate"]:
        sg = 1 / (1 + torch.exp(-zs))
        out["dz"] = (go * vs * (sg + zs * sg * (1 - sg))).reshape(s["x"].shape)
        g = go * zs * sg
    ds1 = s["ds1"].double() if c["s0"] else torch.zeros_like(start)
    ds0, dA = ds1.clone(), torch.zeros_like(A)
    dx, dd = D * g, torch.zeros_like(x)
    dB, dC = torch.zeros_like(Bs, dtype=torch.float64), torch.zeros_like(Cs, dtype=torch.float64)
    for b, t0, t1 in runs:
        rows = slice(None) if b is None else slice(b, b + 1)
        m = ds1[rows].clone()
        for t in reversed(range(t0, t1)):
            d, hp, Bt = ds[:, t], hist[t], Bs[:, t].double()
            a, u = torch.exp(d[..., None] * A), d * x[:, t]
            m = m + g[:, t, :, None] * Cs[:, t, None].double()
            dC[:, t] = torch.einsum("bp,bpn->bn", g[:, t], a * hp + u[..., None] * Bt[:, None])
            dB[:, t] = torch.einsum("bpn,bp->bn", m, u)
            mb = torch.einsum("bpn,bn->bp", m, Bt)
            m = m * a
            q = m * hp
            dd[:, t] = x[:, t] * mb + (q * A).sum(-1)
            dx[:, t] += d * mb
            dA += torch.einsum("bpn,bp->pn", q, d)
        ds0[rows] = m
    ddt = dd / (1 + torch.exp(-v))
    out.update(dx=dx.reshape(s["x"].shape), ddt=ddt.reshape(s["x"].shape), dA=dA, dB=dB.reshape(s["Bm"].shape),
               dC=dC.reshape(s["Cm"].shape), dD=(g * x).sum((0, 1)), ddt_bias=ddt.sum((0, 1)))
    if c["s0"]:
        out["ds0"] = ds0
    return out


def _exact_sample(c, s):
    """Row by row: the order first, then how far down it each limit reaches."""
    token, logp = [], []
    get = lambda n, i, off: float(s[n][i]) if n in s else off  # noqa: E731
    for i in range(c["N"]):
        T, p, q, k = (get("temperature", i, 1.0), get("top_p", i, 1.0), get("min_p", i, 0.0), int(get("top_k", i, 0)))
        val, idx = torch.sort(s["logits"][i].double(), descending=True, stable=True)
        e = (val - val[0]) / (T or 1.0)
        w = (torch.exp(e) * UNIT).round()
        n = int((w >= max(q * UNIT, 1.0)).sum())
        n = min(n, k) if k > 0 else n
        n = 1 if T == 0 else n
        run = w[:n].cumsum(0)
        if p < 1:
            n = min(n, 1 + int((run < p * run[-1]).sum()))
        by_index = idx[:n].sort()
        total = float(run[n - 1])
        at = int((w[:n][by_index.indices].cumsum(0) > float(s["u"][i]) * total).int().argmax())
        token.append(by_index.values[at])
        logp.append(e[by_index.indices[at]] - math.log(total / UNIT))
    return {"token": torch.stack(token), "logp": torch.stack(logp)}
