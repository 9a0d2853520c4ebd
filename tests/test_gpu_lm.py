"""GPU parity of the language-model operators against the fp64 oracle (oracle/lm.py).

Tolerances (relative Frobenius error of a tensor unless said otherwise), derived from the
arithmetic:
  fp32 storage      1e-5: sums of at most a few hundred products, each within 2^-24, exponentials
                    within 2^-22
  bf16 storage      8e-3 on bf16 outputs: the output's rounding and one rounding of each of the
                    two operands that carry intermediate values, 2^-9 of a value each at most,
                    and room for sums smaller than their terms
                    2e-5 on fp32 states and dg: operands split in two bf16 parts, 2^-17 of a
                    value each at most, and room as above
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from conftest import rel_fro  # noqa: E402
from oracle import lm as olm  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16_OUT, BF16_STATE = 1e-5, 8e-3, 2e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


def np64(x):
    return x.detach().double().cpu().numpy()


def lin_inputs(B, T, H, Hk, Dk, Dv, bf16, s0, decay="gate", docs=0, seed=0, fused=False):
    """Inputs on the device; fused: q, k and v are column slices of one projection."""
    gen = torch.Generator().manual_seed(1000 + seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    xt = torch.bfloat16 if bf16 else torch.float32
    wq, wv = Hk * Dk, H * Dv
    proj = torch.cat([n(B, T, wq), n(B, T, wq) / Dk ** 0.5, n(B, T, wv)], -1).to(xt).cuda()
    parts = [proj[..., :wq], proj[..., wq:2 * wq], proj[..., 2 * wq:]]
    if not fused:
        parts = [p.contiguous() for p in parts]
    q, k, v = parts[0].unflatten(-1, (Hk, Dk)), parts[1].unflatten(-1, (Hk, Dk)), parts[2].unflatten(-1, (H, Dv))
    g = torch.log(torch.sigmoid(n(B, T, H) + 3))
    if decay == "strong":
        g = g * 100
    elif decay == "none":
        g = torch.zeros(B, T, H)
    elif decay == "mixed":
        g = torch.where(torch.rand(B, T, H, generator=gen) < 0.1, -80 * torch.rand(B, T, H, generator=gen), g)
    if docs:
        g = torch.where((torch.rand(B, T, 1, generator=gen) < 1 / docs), float("-inf"), g)
    x = dict(q=q, k=k, v=v, g=g.float().cuda(), s0=n(B, H, Dk, Dv).cuda() if s0 else None)
    x["go"] = n(B, T, H, Dv).to(xt).cuda()
    x["ds1"] = n(B, H, Dk, Dv).cuda() if s0 else None
    return x


def lin_check(B, T, H, Hk, Dk, Dv, bf16, s0=True, backward=True, **kw):
    from adjoint_gradients_long_gb300 import lm
    x = lin_inputs(B, T, H, Hk, Dk, Dv, bf16, s0, **kw)
    a = lm.LinAttn(B, T, H, Dk, Dv, Hk=Hk, x_bf16=bf16, scale=Dk ** -0.5, backward=backward)
    h = {n: None if y is None else np64(y) for n, y in x.items()}
    o, s1 = a.forward(x["q"], x["k"], x["v"], x["g"], x["s0"])
    ro, rs = olm.lin_forward(h["q"], h["k"], h["v"], h["g"], Dk ** -0.5, h["s0"])
    out, st = (BF16_OUT, BF16_STATE) if bf16 else (F32, F32)
    errs = {"o": (rel_fro(np64(o), ro), out), "s1": (rel_fro(np64(s1), rs), st)}
    if backward:
        got = a.backward(x["q"], x["k"], x["v"], x["g"], x["go"], x["s0"], x["ds1"])
        ref = olm.lin_backward(h["q"], h["k"], h["v"], h["g"], Dk ** -0.5, h["go"], h["s0"], h["ds1"])
        for nm, y, r, tol in zip(("dq", "dk", "dv", "dg", "ds0"), got, ref, (out, out, out, st, st)):
            errs[nm] = (rel_fro(np64(y), r), tol)
    torch.cuda.synchronize()
    assert a.status() == 0
    print(f"lin B={B} T={T} H={H}/{Hk} D={Dk}/{Dv} bf16={bf16} {kw}: " + " ".join(f"{n}={e:.1e}" for n, (e, _) in errs.items()))
    bad = {n: f"{e:.2e}" for n, (e, tol) in errs.items() if not e <= tol}
    assert not bad, bad
    return a, x


SIZES = [
    (1, 1, 1, 1, 8, 8), (2, 2, 3, 1, 16, 24), (1, 63, 2, 2, 64, 64), (1, 64, 2, 1, 128, 128), (2, 65, 2, 2, 72, 40),
    (1, 127, 2, 2, 128, 64), (1, 128, 1, 1, 128, 128), (3, 129, 4, 2, 40, 128), (1, 300, 6, 3, 96, 64),
    (2, 257, 2, 1, 64, 120),
]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,T,H,Hk,Dk,Dv", SIZES)
def test_lin_sizes(B, T, H, Hk, Dk, Dv, bf16):
    lin_check(B, T, H, Hk, Dk, Dv, bf16, seed=T)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kw", [dict(s0=False), dict(decay="strong"), dict(decay="none"), dict(decay="mixed"),
                                dict(docs=40), dict(docs=1, s0=False), dict(fused=True), dict(docs=3, fused=True)])
def test_lin_decays_and_layouts(kw, bf16):
    lin_check(2, 200, 4, 2, 64, 64, bf16, seed=3, **kw)


@pytest.mark.parametrize("bf16", [False, True])
def test_lin_long(bf16):
    """Many chunks: several segments a head, states carried over all of them."""
    lin_check(1, 3001, 2, 1, 64, 128, bf16, seed=9)


@pytest.mark.parametrize("low", [float("-inf"), -3.4028234663852886e38, -105.0])
def test_lin_new_start(low):
    """A decay of zero cuts every trace of what came before, whatever it held, and its own
    gradient is zero."""
    from adjoint_gradients_long_gb300 import lm
    for bf16 in (False, True):
        x = lin_inputs(1, 150, 2, 2, 64, 64, bf16, True, seed=4)
        x["g"][:, 70] = low
        a = lm.LinAttn(1, 150, 2, 64, 64, x_bf16=bf16, backward=True)
        o, s1 = (y.clone() for y in a.forward(x["q"], x["k"], x["v"], x["g"], x["s0"]))
        dg = a.backward(x["q"], x["k"], x["v"], x["g"], x["go"], x["s0"], x["ds1"])[3]
        assert (dg[:, 70] == 0).all() and torch.isfinite(dg).all()
        b = lm.LinAttn(1, 80, 2, 64, 64, x_bf16=bf16)
        o2, s2 = b.forward(*(x[n][:, 70:].contiguous() for n in "qkv"), x["g"][:, 70:].contiguous())
        assert rel_fro(np64(o[:, 70:]), np64(o2)) <= (BF16_OUT if bf16 else F32)
        assert rel_fro(np64(s1), np64(s2)) <= (BF16_STATE if bf16 else F32)


def test_lin_empty_and_zero_length():
    from adjoint_gradients_long_gb300 import lm
    for bf16 in (False, True):
        x = lin_inputs(2, 0, 2, 2, 16, 16, bf16, True)
        a = lm.LinAttn(2, 0, 2, 16, 16, x_bf16=bf16, backward=True)
        assert (a.forward(x["q"], x["k"], x["v"], x["g"], x["s0"])[1] == x["s0"]).all()
        assert (a.forward(x["q"], x["k"], x["v"], x["g"])[1] == 0).all()
        assert (a.backward(x["q"], x["k"], x["v"], x["g"], x["go"], x["s0"], x["ds1"])[4] == x["ds1"]).all()
        x = lin_inputs(0, 5, 2, 2, 16, 16, bf16, False)
        a = lm.LinAttn(0, 5, 2, 16, 16, x_bf16=bf16, backward=True)
        a.forward(x["q"], x["k"], x["v"], x["g"])
        a.backward(x["q"], x["k"], x["v"], x["g"], x["go"])


def test_lin_not_finite_reaches_onwards():
    """A NaN at token t reaches every later output that reads it and none of an earlier chunk."""
    from adjoint_gradients_long_gb300 import lm
    for bf16 in (False, True):
        x = lin_inputs(1, 400, 1, 1, 64, 64, bf16, False)
        x["v"][0, 200, 0, 3] = float("nan")
        a = lm.LinAttn(1, 400, 1, 64, 64, x_bf16=bf16)
        o, s1 = a.forward(x["q"], x["k"], x["v"], x["g"])
        assert torch.isnan(o[0, 200:, 0, 3]).all() and torch.isnan(s1[0, 0, :, 3]).all()
        assert torch.isfinite(o[0, :128]).all() and torch.isfinite(o[..., :3]).all()


def test_lin_same_bits_and_streams_and_graph():
    """The same inputs give the same bits: again, on another stream, from a captured graph."""
    from adjoint_gradients_long_gb300 import lm
    x = lin_inputs(2, 333, 4, 2, 64, 64, True, True)
    a = lm.LinAttn(2, 333, 4, 64, 64, Hk=2, backward=True)
    args = (x["q"], x["k"], x["v"], x["g"])

    def run():
        return [*a.forward(*args, x["s0"]), *a.backward(*args, x["go"], x["s0"], x["ds1"])]
    first = [y.clone() for y in run()]
    torch.cuda.synchronize()
    for y, z in zip(run(), first):
        assert torch.equal(y, z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for y in run():
            y_ = y.clone()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    for y in outs:
        y.zero_()
    g.replay()
    torch.cuda.synchronize()
    for y, z in zip(outs, first):
        assert torch.equal(y, z)
    del y_


# ---------------------------------------------------------------- the step
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,H,Hk,Dk,Dv", [(1, 1, 1, 8, 8), (1, 16, 16, 128, 128), (5, 6, 2, 72, 40), (40, 8, 1, 64, 104),
                                          (3, 2, 2, 128, 8), (2, 2, 1, 16, 72)])
def test_step(B, H, Hk, Dk, Dv, bf16):
    """Three tokens, one by one, against the recurrence; the pool is permuted, one row is padding
    and the other slots stay as they are.  A step's fp32 state is within 3 roundings: 1e-6."""
    from adjoint_gradients_long_gb300 import lm
    gen = torch.Generator().manual_seed(B * 7 + H)
    n_slots = B + 3
    pool = torch.randn(n_slots, H, Dk, Dv, generator=gen).cuda()
    slots = torch.randperm(n_slots, generator=gen)[:B].int()
    pad = B - 1 if B > 1 else None
    if pad is not None:
        slots[pad] = [-1, n_slots, 2 ** 31 - 1][B % 3]
    live = [b for b in range(B) if b != pad]
    S = np64(pool)
    before = pool.clone()
    st = lm.LinStep(B, H, Dk, Dv, Hk=Hk, x_bf16=bf16, scale=0.3)
    for t in range(3):
        x = lin_inputs(B, 1, H, Hk, Dk, Dv, bf16, False, seed=t, docs=4 if t == 2 else 0, fused=t == 1)
        q, k, v, g = (x[n][:, 0] for n in ("q", "k", "v", "g"))
        o = st.step(q, k, v, g.contiguous(), pool, slots.cuda())
        idx = slots[live].long().numpy()
        ro, s1 = olm.lin_forward(*(np64(x[n])[live] for n in "qkvg"), 0.3, S[idx])
        S[idx] = s1
        assert rel_fro(np64(o)[live], ro[:, 0]) <= (BF16_OUT if bf16 else F32)
        assert rel_fro(np64(pool), S) <= 1e-6
        if pad is not None:
            assert (o[pad] == 0).all()
    rest = [i for i in range(n_slots) if i not in idx]
    assert torch.equal(pool[rest], before[rest])


def test_step_agrees_with_chunks():
    from adjoint_gradients_long_gb300 import lm
    x = lin_inputs(2, 20, 4, 2, 64, 64, True, True)
    o, s1 = lm.LinAttn(2, 20, 4, 64, 64, Hk=2).forward(x["q"], x["k"], x["v"], x["g"], x["s0"])
    st, pool, outs = lm.LinStep(2, 4, 64, 64, Hk=2), x["s0"].clone(), []
    for t in range(20):
        outs.append(st.step(*(x[n][:, t].contiguous() for n in "qkvg"), pool).clone())
    assert rel_fro(np64(torch.stack(outs, 1)), np64(o)) <= 2 * BF16_OUT
    assert rel_fro(np64(pool), np64(s1)) <= BF16_STATE


def test_step_offsets_past_32_bits():
    """A pool of over 2^31 values: a slot at its end."""
    from adjoint_gradients_long_gb300 import lm
    n = 2 ** 31 // (16 * 128 * 128) + 3
    pool = torch.empty(n, 16, 128, 128, device="cuda")
    x = lin_inputs(1, 1, 16, 16, 128, 128, True, True)
    pool[n - 1] = x["s0"][0]
    pool[0] = 0
    st = lm.LinStep(1, 16, 128, 128)
    o = st.step(*(x[m][:, 0].contiguous() for m in "qkvg"), pool, torch.tensor([n - 1], dtype=torch.int32, device="cuda"))
    ro, rs = olm.lin_forward(*(np64(x[m]) for m in "qkvg"), 1.0, np64(x["s0"]))
    assert rel_fro(np64(o), ro[:, 0]) <= BF16_OUT and rel_fro(np64(pool[n - 1]), rs[0]) <= 1e-6
    assert (pool[0] == 0).all()


# ---------------------------------------------------------------- log probabilities
def logp_check(x, y, top, bf16, glp=None, gent=None, inplace=False):
    from adjoint_gradients_long_gb300 import lm
    N, V = x.shape
    p = lm.TokenLogProbs(N, V, x_bf16=bf16, top=top)
    h, yh = np64(x), y.cpu().numpy()
    if glp is None:
        r = p.forward(x, y)
    else:
        r = p.gradient(x, y, glp, gent, dlogits=x if inplace else None)
    logp, ent, lse, ids, tops = olm.logprob(h, yh, top)
    # fp32 sums of at most 2^17 terms by 512 threads, and the rounding of values near the
    # largest logit: 1e-5 of the tensor's scale
    for nm, got, want in (("logp", r.logp, logp), ("entropy", r.entropy, ent), ("lse", r.lse, lse)):
        got = np64(got)
        assert np.array_equal(np.isfinite(got), np.isfinite(want)), nm
        f = np.isfinite(want)
        assert np.array_equal(got[~f], want[~f], equal_nan=True), nm
        assert np.abs(got[f] - want[f]).max(initial=0) <= 1e-5 * max(1, np.abs(want[f]).max(initial=0)), nm
    if top:
        assert np.array_equal(r.top_id.cpu().numpy(), ids)
        with np.errstate(over="ignore"):
            tops = tops.astype(np.float32)               # past its range: minus infinity
        f = np.isfinite(tops)
        assert np.allclose(np64(r.top_logp)[f], tops[f], rtol=1e-5, atol=1e-5)
    if glp is not None:
        d = olm.logprob_grad(h, yh, np64(glp), np.zeros(N) if gent is None else np64(gent))
        assert rel_fro(np64(r.dlogits), d) <= (5e-3 if bf16 else F32)
        if inplace:
            assert r.dlogits.data_ptr() == x.data_ptr()
    return r


def logits(N, V, bf16, seed=0, mask=0, pitch=None, shift=0):
    """[N,V] logits; pitch and shift: a view with rows that far apart that starts off alignment."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(N, V, generator=gen) * 3
    if mask:
        x[:, torch.randperm(V, generator=gen)[:mask]] = float("-inf")
    xt = torch.bfloat16 if bf16 else torch.float32
    if pitch is None:
        out = x.to(xt).cuda()
    else:
        flat = torch.full((N * pitch + shift,), 1e4, dtype=xt, device="cuda")
        out = flat[shift:shift + N * pitch].view(N, pitch)[:, :V]
        out.copy_(x.to(xt))
    y = torch.randint(-1, V, (N,), generator=gen)
    return out, y.cuda()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N,V,top,kw", [
    (1, 1, 1, {}), (3, 2, 2, {}), (2, 7, 7, {}), (4, 33, 32, {}), (5, 1000, 5, dict(mask=300)), (1, 32000, 8, {}),
    (9, 5003, 3, {}), (3, 4097, 16, dict(pitch=4103, shift=3)), (2, 131072, 32, {}), (2, 300001, 4, dict(mask=7)),
    (700, 999, 2, {}), (2, 800, 32, dict(mask=790)),
])
def test_logprob(N, V, top, kw, bf16):
    x, y = logits(N, V, bf16, seed=V, **kw)
    logp_check(x, y, top, bf16)
    gen = torch.Generator().manual_seed(1)
    glp, gent = torch.randn(N, generator=gen).cuda(), torch.randn(N, generator=gen).cuda()
    logp_check(x, y, top, bf16, glp, gent)
    logp_check(x, y, 0, bf16, glp)
    logp_check(x.clone(), y, top, bf16, glp, gent, inplace=True)


@pytest.mark.parametrize("bf16", [False, True])
def test_logprob_ties_and_masks(bf16):
    """Equal values (all of a row, and many at the boundary of the list), a row masked
    altogether, one value left, targets out of range and masked."""
    xt = torch.bfloat16 if bf16 else torch.float32
    V = 6000
    x = torch.zeros(7, V, dtype=xt, device="cuda")
    x[1, ::2] = 1
    x[2] = float("-inf")
    x[3] = float("-inf")
    x[3, 4321] = -7
    x[4, 17:29] = 3
    x[5] = torch.arange(V, device="cuda").to(xt) / 100
    x[6, ::3] = -0.0
    y = torch.tensor([5, V, 3, 4321, 20, -5, 2], device="cuda")
    glp, gent = torch.ones(7, device="cuda"), torch.full((7,), 0.5, device="cuda")
    r = logp_check(x, y, 32, bf16, glp, gent)
    assert (r.dlogits[2] == 0).all() and r.logp[2].item() == float("-inf") and r.entropy[2].item() == 0
    assert r.logp[1].item() == 0 and r.logp[5].item() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_logprob_not_finite(bad, bf16):
    """A NaN or +inf makes its own row NaN and no other; NaN leads the top list."""
    from adjoint_gradients_long_gb300 import lm
    x, y = logits(3, 3000, bf16, seed=2)
    x[1, 100] = bad
    y[:] = 5
    p = lm.TokenLogProbs(3, 3000, x_bf16=bf16, top=4)
    r = p.gradient(x, y, torch.ones(3, device="cuda"))
    assert torch.isnan(r.logp[1]) and torch.isnan(r.dlogits[1]).all()
    assert torch.isfinite(r.logp[[0, 2]]).all() and torch.isfinite(r.dlogits[[0, 2]]).all()
    assert r.top_id[1, 0].item() == 100
    _, _, _, ids, _ = olm.logprob(np64(x), y.cpu().numpy(), 4)
    assert np.array_equal(r.top_id.cpu().numpy(), ids)


def test_logprob_extremes():
    """Logits at the ends of the range of fp32: no overflow, exact limits."""
    x = torch.tensor([[3e38, -3e38, 0.0, 1.0], [-3e38, -3e38, -3e38, -3e38], [80.0, -80.0, 0.0, 80.0]], device="cuda")
    y = torch.tensor([0, 1, 2], device="cuda")
    logp_check(x, y, 4, False, torch.ones(3, device="cuda"), torch.ones(3, device="cuda"))


def test_logprob_offsets_past_32_bits():
    from adjoint_gradients_long_gb300 import lm
    N, V = 16400, 131072
    x = torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
    x[N - 1], y1 = logits(1, V, True, seed=8)[0][0], 77
    y = torch.zeros(N, dtype=torch.int64, device="cuda")
    y[N - 1] = y1
    p = lm.TokenLogProbs(N, V, top=3)
    r = p.gradient(x, y, torch.ones(N, device="cuda"), dlogits=x.clone())
    logp, _, _, ids, _ = olm.logprob(np64(x[N - 1:]), np.array([y1]), 3)
    assert abs(r.logp[N - 1].item() - logp[0]) <= 1e-4 and np.array_equal(r.top_id[N - 1].cpu().numpy(), ids[0])
    d = olm.logprob_grad(np64(x[N - 1:]), np.array([y1]), np.ones(1), np.zeros(1))
    assert rel_fro(np64(r.dlogits[N - 1:]), d) <= 5e-3


# ---------------------------------------------------------------- clipping
def clip_tensors(sizes, seed=0, shift=0, scale=0.1):
    """Alternating types; shift: views that start that many values off alignment."""
    gen = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.empty(n + shift, dtype=torch.bfloat16 if i % 2 else torch.float32, device="cuda")[shift:]
        t.copy_(torch.randn(n, generator=gen) * scale)
        out.append(t)
    return out


@pytest.mark.parametrize("sizes,shift", [([1], 0), ([0, 3, 0], 1), ([5, 1000, 77777], 0), ([5, 1000, 77777, 8], 3),
                                         ([17] * 64, 1), ([33] * 65, 0), ([10] * 2500, 0), ([3000001, 999999], 5),
                                         ([30000000], 0), ([], 0)])
@pytest.mark.parametrize("inplace", [False, True])
def test_clip(sizes, shift, inplace):
    from adjoint_gradients_long_gb300 import lm
    x = clip_tensors(sizes, seed=len(sizes), shift=shift)
    ref = [np64(t) for t in x]
    outs = None if inplace else [torch.full_like(t, 9.0) for t in x]
    # the norm: fp32 partial sums of squares, 1e-6; the coefficient and its product with a
    # value: three roundings of fp32, or one of bf16
    for max_norm in (0.5, 1e6):
        c = lm.GradClip(x, outs)
        norm, coef = c.clip(max_norm)
        rn, rc, ry = olm.grad_clip(ref, max_norm)
        assert abs(norm.item() - rn) <= 1e-6 * rn and abs(coef.item() - rc) <= 2e-6
        for t, y, r in zip(x, x if inplace else outs, ry):
            if r.size:
                assert rel_fro(np64(y), r) <= (4e-3 if t.dtype == torch.bfloat16 else 3e-6)
        if inplace:
            ref = [np64(t) for t in x]


def test_clip_not_finite():
    from adjoint_gradients_long_gb300 import lm
    x = clip_tensors([1000, 1000])
    x[0][3] = float("inf")
    norm, coef = lm.GradClip(x, [torch.empty_like(t) for t in x]).clip(1.0)
    assert norm.item() == float("inf") and coef.item() == 0
    x[0][3] = float("nan")
    norm, coef = lm.GradClip(x).clip(1.0)
    assert torch.isnan(norm) and torch.isnan(coef) and torch.isnan(x[1]).all()


def test_clip_same_bits_and_graph():
    from adjoint_gradients_long_gb300 import lm
    x = clip_tensors([12345, 777777, 5])
    outs = [torch.empty_like(t) for t in x]
    c = lm.GradClip(x, outs)
    c.clip(0.7)
    first = [t.clone() for t in outs] + [c.result.clone()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.clip(0.7)
    for _ in range(3):
        for t in outs:
            t.zero_()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(first, outs + [c.result]))
