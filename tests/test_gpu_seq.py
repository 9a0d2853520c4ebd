"""GPU parity of the short convolution and the selective scan against the fp64 recurrences
(oracle/seq.py), through lm.py.

Tolerances (relative Frobenius error), from the arithmetic:
  HALF     a value rounded once to bf16: half a step, 2^-8 of it at most, and what fp32 had before
  CONV     fp32 sums of at most 4 products and one sigmoid: 8 roundings of 2^-24 and two units of 2^-22
  SUMS     sums of those over up to 3000 tokens in parts: their own roundings add up to 2^-24 times a few
           tens of levels at most
  SCAN     a state adds up what its memory holds, up to 60 tokens in these inputs (d A is 1/60 at least on
           average): each decay is off by 2^-22 (the exponential) and 2^-24 (its exponent), 60 x 3e-7, and
           the steps and products by a few units: 2e-5
  SCAN_G   gradients: an adjoint state times a state, each off as above, and room for sums smaller
           than their terms: 6e-5
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from conftest import rel_fro  # noqa: E402
from oracle import seq as oseq  # noqa: E402

pytestmark = pytest.mark.gpu

HALF, CONV, SUMS, SCAN, SCAN_G = 2.0 ** -8, 2e-6, 1e-5, 2e-5, 6e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


def np64(x):
    return None if x is None else x.detach().double().cpu().numpy()


def same_bits(x, y):
    """Equal, NaN for NaN."""
    return x.shape == y.shape and bool(((x == y) | ((x != x) & (y != y))).all())


class Maker:
    """Seeded inputs on the device; `wide`: token arrays as column slices of wider ones."""

    def __init__(self, seed, bf16, wide):
        self.gen, self.xt, self.wide = torch.Generator().manual_seed(seed), torch.bfloat16 if bf16 else torch.float32, wide

    def normal(self, *s):
        return torch.randn(*s, generator=self.gen)

    def tokens(self, *s):
        x = self.normal(*s).to(self.xt).cuda()
        if self.wide:
            w = torch.full((*s[:-1], s[-1] + 24), float("nan"), dtype=self.xt, device="cuda")
            w[..., 8:8 + s[-1]] = x
            x = w[..., 8:8 + s[-1]]
        return x

    def f32(self, *s):
        return self.normal(*s).cuda()


def offsets_of(lengths, before=0):
    return torch.tensor(np.concatenate([[before], before + np.cumsum(lengths)]), dtype=torch.int64, device="cuda")


def rows(x, width):
    return np64(x).reshape(-1, width)


# ---------------------------------------------------------------- convolution
def conv_case(seed, B, T, P, W, bf16, state=True, bias=True, lengths=None, before=0, wide=False):
    mk = Maker(seed, bf16, wide)
    lead = (T,) if lengths is not None else (B, T)
    x = dict(x=mk.tokens(*lead, P), go=mk.tokens(*lead, P).contiguous(), w=mk.f32(P, W) / W ** 0.5,
             bias=mk.f32(P) if bias else None, s0=mk.f32(B, W - 1, P).to(mk.xt) if state else None,
             ds1=mk.f32(B, W - 1, P).to(mk.xt) if state else None,
             offsets=None if lengths is None else offsets_of(lengths, before))
    return x, oseq.sequences(B, T, x["offsets"])


def conv_check(seed, B, T, P, W, bf16, act=True, lengths=None, **kw):
    from adjoint_gradients_long_gb300 import lm
    x, seqs = conv_case(seed, B, T, P, W, bf16, lengths=lengths, **kw)
    c = lm.ShortConv(B, T, P, W, x_bf16=bf16, act=act, packed=lengths is not None, backward=True)
    y, s1 = c.forward(x["x"], x["w"], x["bias"], x["s0"], x["offsets"])
    dx, dw, db, ds0 = c.backward(x["x"], x["w"], x["go"], x["bias"], x["s0"], x["ds1"], x["offsets"])
    h = rows(x["x"], P), np64(x["w"]), np64(x["bias"]), np64(x["s0"]), seqs
    ry, rs = oseq.conv_forward(*h, act=act)
    r = oseq.conv_backward(*h, rows(x["go"], P), np64(x["ds1"]), act=act)
    val = HALF if bf16 else CONV
    assert rel_fro(rows(y, P), ry) <= val
    assert (np64(s1) == rs).all()                          # inputs, copied
    for nm, got, ref, tol in (("dx", rows(dx, P), r[0], val), ("dw", np64(dw), r[1], SUMS), ("db", np64(db), r[2], SUMS),
                              ("ds0", np64(ds0), r[3], val)):
        assert rel_fro(got, ref) <= tol, nm
    return c, x


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,T,P", [(1, 1, 8), (3, 2, 16), (2, 3, 264), (1, 65, 8), (2, 131, 40), (1, 300, 520), (5, 7, 2048)])
def test_conv_sizes(B, T, P, W, bf16):
    conv_check(T * W, B, T, P, W, bf16)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kw", [dict(state=False), dict(bias=False), dict(act=False), dict(wide=True),
                                dict(lengths=[5, 0, 1, 60, 2, 0, 3, 90], wide=True), dict(lengths=[0, 0, 161]),
                                dict(lengths=[161, 0]), dict(lengths=[1] * 40, state=False), dict(lengths=[64, 64])])
def test_conv_forms(kw, bf16):
    kw = dict(kw)
    B = len(kw["lengths"]) if "lengths" in kw else 2
    conv_check(9, B, sum(kw["lengths"]) if "lengths" in kw else 161, 72, 4, bf16, **kw)


@pytest.mark.parametrize("before", [1, 20, 37])
def test_conv_sequences_within_the_tokens(before):
    for W in (2, 3, 4):
        conv_check(13, 3, 200, 72, W, True, lengths=[50, 0, 77], before=before)
        conv_check(14, 2, 700, 40, W, False, lengths=[1, 633], before=before)


def test_conv_long():
    conv_check(4, 1, 3000, 64, 4, True)


def test_conv_rows_of_no_sequence_stay():
    from adjoint_gradients_long_gb300 import lm
    for bf16 in (False, True):
        x, seqs = conv_case(2, 3, 200, 48, 4, bf16, lengths=[40, 0, 77], before=20)
        c = lm.ShortConv(3, 200, 48, 4, x_bf16=bf16, packed=True, backward=True)
        for n in ("x", "go"):                              # nothing is read there
            x[n][:20], x[n][137:] = float("nan"), float("inf")
        c.y.fill_(7.0)
        dx = c._like("x", x["x"])
        dx.fill_(7.0)
        y, _ = c.forward(x["x"], x["w"], x["bias"], x["s0"], x["offsets"])
        dx, dw, db, _ = c.backward(x["x"], x["w"], x["go"], x["bias"], x["s0"], x["ds1"], x["offsets"])
        for o in (y, dx):
            assert (o[:20] == 7).all() and (o[137:] == 7).all() and torch.isfinite(o).all() and (o[20:137] != 7).any()
        assert torch.isfinite(dw).all() and torch.isfinite(db).all()


def test_conv_steps_follow_the_prompt():
    """A prompt in one call and token by token: the same values to their rounding, the states equal."""
    from adjoint_gradients_long_gb300 import lm
    for bf16 in (False, True):
        for W in (2, 3, 4):
            x, _ = conv_case(3, 3, 9, 40, W, bf16)
            y, s1 = lm.ShortConv(3, 9, 40, W, x_bf16=bf16).forward(x["x"], x["w"], x["bias"], x["s0"])
            pool = torch.full((7, W - 1, 40), 5.0, dtype=x["s0"].dtype, device="cuda")
            slots = torch.tensor([6, 0, 3], dtype=torch.int32, device="cuda")
            pool[slots.long()] = x["s0"]
            st = lm.ShortConvStep(3, 40, W, x_bf16=bf16)
            for t in range(9):
                got = st.step(x["x"][:, t], x["w"], pool, x["bias"], slots)
                assert rel_fro(np64(got), np64(y[:, t])) <= (HALF if bf16 else CONV)
            assert (pool[slots.long()] == s1).all() and (pool[[1, 2, 4, 5]] == 5).all()


# ---------------------------------------------------------------- scan
def scan_case(seed, B, T, P, N, bf16, state=True, gate=True, skip=True, bias=True, lengths=None, before=0, wide=False, scale=1.0):
    mk = Maker(seed, bf16, wide)
    lead = (T,) if lengths is not None else (B, T)
    x = dict(x=mk.tokens(*lead, P), dt=mk.tokens(*lead, P), Bm=mk.tokens(*lead, N), Cm=mk.tokens(*lead, N),
             z=mk.tokens(*lead, P) if gate else None, go=mk.tokens(*lead, P).contiguous(),
             A=-(torch.rand(P, N, generator=mk.gen) + 0.1).cuda() * scale, D=mk.f32(P) if skip else None,
             dt_bias=mk.f32(P) - 1 if bias else None, s0=mk.f32(B, P, N) if state else None, ds1=mk.f32(B, P, N) if state else None,
             offsets=None if lengths is None else offsets_of(lengths, before))
    return x, oseq.sequences(B, T, x["offsets"])


FWD = ("x", "dt", "A", "Bm", "Cm")


def scan_run(s, x):
    y, s1 = s.forward(*(x[n] for n in FWD), x["D"], x["z"], x["dt_bias"], x["s0"], x["offsets"])
    r = s.backward(*(x[n] for n in FWD), x["go"], x["D"], x["z"], x["dt_bias"], x["s0"], x["ds1"], x["offsets"])
    return y, s1, r


def scan_check(seed, B, T, P, N, bf16, lengths=None, **kw):
    from adjoint_gradients_long_gb300 import lm
    x, seqs = scan_case(seed, B, T, P, N, bf16, lengths=lengths, **kw)
    s = lm.SelScan(B, T, P, N, x_bf16=bf16, packed=lengths is not None, backward=True)
    y, s1, r = scan_run(s, x)
    z = None if x["z"] is None else rows(x["z"], P)
    h = (rows(x["x"], P), rows(x["dt"], P), np64(x["A"]), rows(x["Bm"], N), rows(x["Cm"], N), np64(x["D"]), z, np64(x["dt_bias"]),
         np64(x["s0"]), seqs)
    ry, rs, _ = oseq.scan_forward(*h)
    g = oseq.scan_backward(*h, rows(x["go"], P), np64(x["ds1"]))
    half = HALF if bf16 else 0.0
    errs = {"y": (rel_fro(rows(y, P), ry), half + SCAN), "s1": (rel_fro(np64(s1), rs), SCAN)}
    for nm, got, ref, w in (("dx", r.dx, g[0], P), ("ddt", r.ddt, g[1], P), ("dA", r.dA, g[2], 0), ("dB", r.dB, g[3], N),
                            ("dC", r.dC, g[4], N), ("dD", r.dD, g[5], 0), ("dz", r.dz, g[6], P), ("dbias", r.ddt_bias, g[7], 0),
                            ("ds0", r.ds0, g[8], 0)):
        if got is not None:
            errs[nm] = (rel_fro(rows(got, w) if w else np64(got), ref), (half if w else 0.0) + SCAN_G)
    assert (r.dz is None) == (x["z"] is None)
    print(f"scan B={B} T={T} P={P} N={N} bf16={bf16} {kw}: " + " ".join(f"{n}={e:.1e}" for n, (e, _) in errs.items()))
    bad = {n: f"{e:.2e}" for n, (e, tol) in errs.items() if not e <= tol}
    assert not bad, bad
    return s, x


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("B,T,P", [(1, 1, 8), (2, 2, 136), (1, 17, 40), (3, 33, 64), (2, 150, 24)])
def test_scan_sizes(B, T, P, N, bf16):
    scan_check(T + N, B, T, P, N, bf16)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kw", [dict(state=False), dict(gate=False), dict(skip=False, bias=False), dict(wide=True), dict(scale=30.0),
                                dict(lengths=[5, 0, 1, 60, 2, 0, 3, 90], wide=True), dict(lengths=[0, 0, 161]),
                                dict(lengths=[161, 0]), dict(lengths=[1] * 40, state=False), dict(lengths=[64, 64]),
                                dict(lengths=[15, 1, 16, 17, 31, 33, 32, 1], gate=False)])
@pytest.mark.parametrize("N", [8, 16])
def test_scan_forms(kw, N, bf16):
    kw = dict(kw)
    B = len(kw["lengths"]) if "lengths" in kw else 2
    scan_check(9, B, sum(kw["lengths"]) if "lengths" in kw else 161, 72, N, bf16, **kw)


@pytest.mark.parametrize("N,P", [(8, 264), (16, 136), (32, 72), (64, 40)])
def test_scan_long(N, P):
    """Many segments, states carried over all of them, and sequences that begin inside them."""
    scan_check(5, 1, 2500, P, N, True)
    scan_check(6, 4, 2500, P, N, False, lengths=[700, 1, 0, 1799])


def test_scan_wide():
    """More channels than one turn of the machine takes: one segment."""
    scan_check(7, 1, 40, 16400, 8, True)


def test_scan_rows_of_no_sequence_stay():
    from adjoint_gradients_long_gb300 import lm
    for bf16 in (False, True):
        x, _ = scan_case(2, 3, 300, 40, 16, bf16, lengths=[40, 0, 77], before=20)
        s = lm.SelScan(3, 300, 40, 16, x_bf16=bf16, packed=True, backward=True)
        for n in ("x", "dt", "Bm", "Cm", "z", "go"):
            x[n][:20], x[n][137:] = float("nan"), float("inf")
        grads = [s._like(n, x[n]) for n in ("x", "dt", "Bm", "Cm", "z")]
        for o in (s.y, *grads):
            o.fill_(7.0)
        y, s1, r = scan_run(s, x)
        assert all(g is h for g, h in zip(grads, (r.dx, r.ddt, r.dB, r.dC, r.dz)))
        for o in (y, *grads):
            assert (o[:20] == 7).all() and (o[137:] == 7).all() and torch.isfinite(o).all() and (o[20:137] != 7).any()
        assert all(torch.isfinite(o).all() for o in (s1, r.dA, r.dD, r.ddt_bias, r.ds0))


@pytest.mark.parametrize("before", [1, 3, 20, 37])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_scan_sequences_within_the_tokens(N, before):
    """Tokens of no sequence on both sides, at places inside a tile."""
    for T, lengths in ((200, [50, 0, 77]), (700, [5, 300, 301])):
        for bf16 in (False, True):
            scan_check(N + before, 3, T, 40, N, bf16, lengths=lengths, before=before)


def test_scan_values_that_are_not_finite_stay_in_their_sequence():
    from adjoint_gradients_long_gb300 import lm
    for N in (8, 16):
        lengths = [70, 130, 90, 30]
        x, _ = scan_case(3, 4, 320, 40, N, True, lengths=lengths)
        s = lm.SelScan(4, 320, 40, N, packed=True, backward=True)
        clean = [o.clone() if o is not None else None for o in (*scan_run(s, x)[:2], *s.backward(
            *(x[n] for n in FWD), x["go"], x["D"], x["z"], x["dt_bias"], x["s0"], x["ds1"], x["offsets"]))]
        for n, v in (("x", "nan"), ("dt", "nan"), ("Bm", "inf"), ("go", "nan"), ("Cm", "inf"), ("z", "nan")):
            dirty = dict(x)
            dirty[n] = x[n].clone()
            dirty[n][100:103] = float(v)
            y, s1, r = scan_run(s, dirty)
            got = (y, s1, *r)
            for i in (0, 2, 3, 5, 6, 8):                   # arrays over tokens
                assert same_bits(got[i][:70], clean[i][:70]) and same_bits(got[i][200:], clean[i][200:]), (n, i)
            for i in (1, 10):
                assert all(same_bits(got[i][b], clean[i][b]) for b in (0, 2, 3)), (n, i)


def test_scan_a_channel_that_is_not_finite_stays_alone():
    """In all that belongs to one channel the others keep their bits (B and C are read by all)."""
    from adjoint_gradients_long_gb300 import lm
    for N in (8, 16, 32, 64):
        for bad in (0, 5, 39):
            x, _ = scan_case(4, 2, 700, 40, N, True)
            s = lm.SelScan(2, 700, 40, N, backward=True)
            keep = [c for c in range(40) if c != bad]
            clean = [o.clone() for o in (lambda y, s1, r: (y, s1, *r))(*scan_run(s, x))]
            for n in ("x", "dt", "z", "go"):
                dirty = dict(x)
                dirty[n] = x[n].clone()
                dirty[n][0, 20, bad] = float("nan")
                y, s1, r = scan_run(s, dirty)
                got = (y, s1, *r)
                for i in (0, 2, 3, 8):                      # y, dx, ddt, dz
                    assert same_bits(got[i][..., keep], clean[i][..., keep]), (N, bad, n, i)
                for i in (1, 10):                           # s1, ds0
                    assert same_bits(got[i][:, keep], clean[i][:, keep]), (N, bad, n, i)
                for i in (4, 7, 9):                         # dA, dD, ddt_bias
                    assert same_bits(got[i][keep], clean[i][keep]), (N, bad, n, i)


def test_scan_step_of_zero_keeps_the_state():
    """dt of minus infinity: the decay is one and nothing comes in, bit for bit."""
    from adjoint_gradients_long_gb300 import lm
    for bf16 in (False, True):
        x, _ = scan_case(1, 2, 200, 40, 16, bf16)
        x["dt"].fill_(float("-inf"))
        y, s1 = lm.SelScan(2, 200, 40, 16, x_bf16=bf16).forward(*(x[n] for n in FWD), None, None, x["dt_bias"], x["s0"])
        assert torch.equal(s1, x["s0"])
        ref = np.einsum("bpn,btn->btp", np64(x["s0"]), np64(x["Cm"]))
        assert rel_fro(np64(y), ref) <= (HALF if bf16 else 0.0) + CONV


def test_scan_steps_follow_the_prompt():
    from adjoint_gradients_long_gb300 import lm
    for bf16 in (False, True):
        for N in (8, 16, 32, 64):
            x, _ = scan_case(3, 3, 9, 40, N, bf16)
            y, s1 = lm.SelScan(3, 9, 40, N, x_bf16=bf16).forward(*(x[n] for n in FWD), x["D"], x["z"], x["dt_bias"], x["s0"])
            pool = torch.full((7, 40, N), 5.0, device="cuda")
            slots = torch.tensor([6, 0, 3], dtype=torch.int32, device="cuda")
            pool[slots.long()] = x["s0"]
            st = lm.SelScanStep(3, 40, N, x_bf16=bf16)
            for t in range(9):
                got = st.step(x["x"][:, t], x["dt"][:, t], x["A"], x["Bm"][:, t], x["Cm"][:, t], pool, x["D"], x["z"][:, t],
                              x["dt_bias"], slots)
                assert rel_fro(np64(got), np64(y[:, t])) <= (HALF if bf16 else 0.0) + SCAN
            assert rel_fro(np64(pool[slots.long()]), np64(s1)) <= SCAN and (pool[[1, 2, 4, 5]] == 5).all()


def test_steps_pad():
    """Slots outside the pool: rows of zeros, and the pool as it was."""
    from adjoint_gradients_long_gb300 import lm
    slots = torch.tensor([-1, 2, 4, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    mk = Maker(1, True, False)
    st, pool = lm.ShortConvStep(5, 24), mk.f32(4, 3, 24).bfloat16()
    keep = pool.clone()
    y = st.step(mk.tokens(5, 24), mk.f32(24, 4), pool, None, slots)
    assert (y[[0, 2, 3, 4]] == 0).all() and (y[1] != 0).any() and torch.equal(pool[[0, 1, 3]], keep[[0, 1, 3]])
    st, pool = lm.SelScanStep(5, 24, 16), mk.f32(4, 24, 16)
    keep = pool.clone()
    y = st.step(mk.tokens(5, 24), mk.tokens(5, 24), -mk.f32(24, 16).abs(), mk.tokens(5, 16), mk.tokens(5, 16), pool, mk.f32(24), None,
                None, slots)
    assert (y[[0, 2, 3, 4]] == 0).all() and (y[1] != 0).any() and torch.equal(pool[[0, 1, 3]], keep[[0, 1, 3]])


def test_empty():
    from adjoint_gradients_long_gb300 import lm
    for packed in (False, True):
        x, _ = scan_case(1, 3, 0, 16, 8, False, lengths=[0, 0, 0] if packed else None)
        s = lm.SelScan(3, 0, 16, 8, x_bf16=False, packed=packed, backward=True)
        _, s1, r = scan_run(s, x)
        assert torch.equal(s1, x["s0"]) and torch.equal(r.ds0, x["ds1"]) and (r.dA == 0).all() and (r.dD == 0).all()
        x, _ = conv_case(1, 3, 0, 16, 4, False, lengths=[0, 0, 0] if packed else None)
        c = lm.ShortConv(3, 0, 16, 4, x_bf16=False, packed=packed, backward=True)
        assert torch.equal(c.forward(x["x"], x["w"], x["bias"], x["s0"], x["offsets"])[1], x["s0"])
        _, dw, _, ds0 = c.backward(x["x"], x["w"], x["go"], x["bias"], x["s0"], x["ds1"], x["offsets"])
        assert torch.equal(ds0, x["ds1"]) and (dw == 0).all()
    x, _ = scan_case(1, 0, 5, 16, 8, False, state=False)
    s = lm.SelScan(0, 5, 16, 8, x_bf16=False, backward=True)
    assert (scan_run(s, x)[2].dA == 0).all()
    torch.cuda.synchronize()


def test_broken_offsets_stay_in_bounds():
    """Offsets that break their rule: unspecified values, but every access is inside the arrays (each
    kernel holds what it reads to them; checked by reading), and the next call is right."""
    from adjoint_gradients_long_gb300 import lm
    x, _ = scan_case(4, 3, 200, 40, 16, True, lengths=[40, 80, 80])
    s = lm.SelScan(3, 200, 40, 16, packed=True, backward=True)
    good = [o.clone() for o in scan_run(s, x)[:2]]
    c, cx = lm.ShortConv(3, 200, 40, packed=True, backward=True), conv_case(4, 3, 200, 40, 4, True, lengths=[40, 80, 80])[0]
    for bad in ([0, 150, 50, 200], [-5, 40, 10 ** 15, 200], [200, 100, 50, 0], [60, 60, 60, 60]):
        y = dict(x, offsets=torch.tensor(bad, dtype=torch.int64, device="cuda"))
        scan_run(s, y)
        c.forward(cx["x"], cx["w"], cx["bias"], cx["s0"], y["offsets"])
        c.backward(cx["x"], cx["w"], cx["go"], cx["bias"], cx["s0"], cx["ds1"], y["offsets"])
    assert all(torch.equal(o, g) for o, g in zip(scan_run(s, x)[:2], good))


def test_same_bits_and_graph():
    """A call gives the same bits every time, replayed from a CUDA graph too, on another stream."""
    from adjoint_gradients_long_gb300 import lm
    x, _ = scan_case(8, 2, 700, 136, 16, True)
    s = lm.SelScan(2, 700, 136, 16, backward=True)
    cx, _ = conv_case(8, 2, 700, 136, 4, True)
    c = lm.ShortConv(2, 700, 136, backward=True)

    def outs():
        y, s1, r = scan_run(s, x)
        yc, sc = c.forward(cx["x"], cx["w"], cx["bias"], cx["s0"])
        return [y, s1, *r, yc, sc, *c.backward(cx["x"], cx["w"], cx["go"], cx["bias"], cx["s0"], cx["ds1"])]
    first = [o.clone() for o in outs()]
    assert all(torch.equal(a, b) for a, b in zip(outs(), first))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        outs()
        with torch.cuda.graph(graph, stream=side):
            kept = outs()
    for o in kept:
        o.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, first))


def test_carried_on_with_the_objects_own_states():
    """A long prompt in pieces through one object, its s1 given back as s0, and the gradients from the last
    piece to the first, ds0 given back as ds1: as in one call."""
    from adjoint_gradients_long_gb300 import lm
    n, k = 96, 3                                           # whole tiles, so that states are summed up alike
    x, _ = scan_case(6, 2, n * k, 40, 16, False)
    s, whole = (lm.SelScan(2, t, 40, 16, x_bf16=False, backward=True) for t in (n, n * k))
    y, s1, r = scan_run(whole, x)
    piece = lambda i: {m: v[:, i * n:(i + 1) * n].contiguous() if v is not None and v.dim() == 3 and v.shape[1] == n * k else v  # noqa: E731
                       for m, v in x.items()}
    st, states, ys = x["s0"], [], []
    for i in range(k):
        p = piece(i)
        states.append(st.clone())
        got, st = s.forward(*(p[m] for m in FWD), p["D"], p["z"], p["dt_bias"], st)
        ys.append(got.clone())
    assert rel_fro(np64(torch.cat(ys, 1)), np64(y)) <= SCAN and rel_fro(np64(st), np64(s1)) <= SCAN
    ds, dxs = x["ds1"], []
    for i in reversed(range(k)):
        p = piece(i)
        g = s.backward(*(p[m] for m in FWD), p["go"], p["D"], p["z"], p["dt_bias"], states[i], ds)
        ds = g.ds0
        dxs.append(g.dx.clone())
    assert rel_fro(np64(torch.cat(dxs[::-1], 1)), np64(r.dx)) <= SCAN_G and rel_fro(np64(ds), np64(r.ds0)) <= SCAN_G
    cx, _ = conv_case(6, 2, 40 * 3, 48, 4, True)
    c, whole = (lm.ShortConv(2, t, 48, 4, backward=True) for t in (40, 120))
    y, s1 = (o.clone() for o in whole.forward(cx["x"], cx["w"], cx["bias"], cx["s0"]))
    dx, _, _, ds0 = whole.backward(cx["x"], cx["w"], cx["go"], cx["bias"], cx["s0"], cx["ds1"])
    st, states, ys, dxs, ds = cx["s0"], [], [], [], cx["ds1"]
    for i in range(3):
        states.append(st.clone())
        got, st = c.forward(cx["x"][:, 40 * i:40 * i + 40].contiguous(), cx["w"], cx["bias"], st)
        ys.append(got.clone())
    for i in reversed(range(3)):
        at = slice(40 * i, 40 * i + 40)
        g, _, _, ds = c.backward(cx["x"][:, at].contiguous(), cx["w"], cx["go"][:, at].contiguous(), cx["bias"], states[i], ds)
        dxs.append(g.clone())
    assert torch.equal(torch.cat(ys, 1), y) and torch.equal(st, s1)
    assert rel_fro(np64(torch.cat(dxs[::-1], 1)), np64(dx)) <= 2 * HALF     # ds0 between two pieces is rounded
    assert rel_fro(np64(ds), np64(ds0)) <= 2 * HALF


@pytest.mark.parametrize("bf16", [False, True])
def test_more_sequences_than_a_block_reads_together(bf16):
    lengths = [1, 0, 3, 9] * 65
    conv_check(10, 260, sum(lengths), 40, 4, bf16, lengths=lengths)
    scan_check(11, 260, sum(lengths), 24, 16, bf16, lengths=lengths)


def test_outputs_given_as_inputs_are_refused():
    from adjoint_gradients_long_gb300 import lib, lm
    x, _ = scan_case(6, 1, 32, 16, 16, True)
    s = lm.SelScan(1, 32, 16, 16, backward=True)
    y, _ = s.forward(*(x[m] for m in FWD))
    with pytest.raises(lib.AdjError):
        s.forward(y, *(x[m] for m in FWD[1:]))
    with pytest.raises(lib.AdjError):
        s.forward(*(x[m] for m in FWD), None, y)
    dx = s.backward(*(x[m] for m in FWD), x["go"]).dx
    with pytest.raises(lib.AdjError):
        s.backward(*(x[m] for m in FWD), dx)
    c = lm.ShortConv(1, 32, 16, backward=True)
    w = torch.zeros(16, 4, device="cuda")
    y, _ = c.forward(x["x"], w)
    with pytest.raises(lib.AdjError):
        c.forward(y, w)
    with pytest.raises(lib.AdjError):
        c.backward(x["x"], w, c.backward(x["x"], w, x["go"])[0])


def test_addresses_past_32_bits():
    """Rows and slots behind the first 2^31 elements give what dense copies of them give."""
    from adjoint_gradients_long_gb300 import lm
    T, P, N, ld = 1100, 16, 8, 1 << 21
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)                    # noqa: E731
    base = torch.empty(T, ld, dtype=torch.bfloat16, device="cuda")
    cols = [base[:, -c - 64:][:, :n] for c, n in ((0, P), (128, P), (256, P), (384, N), (512, N))]
    for c in cols:
        c.copy_(rand(*c.shape))
    w, b, A, D = rand(P, 4), rand(P), -rand(P, N).abs(), rand(P)
    go, off = rand(T, P).bfloat16(), torch.tensor([0, 500, T], device="cuda")
    assert T * ld > 2 ** 31
    got = []
    for x, dt, z, Bm, Cm in (cols, [c.contiguous() for c in cols]):
        conv, scan = (k(2, T, P, n, packed=True, backward=True) for k, n in ((lm.ShortConv, 4), (lm.SelScan, N)))
        got.append((*conv.forward(x, w, b, None, off), *conv.backward(x, w, go, b, None, None, off),
                    *scan.forward(x, dt, A, Bm, Cm, D, z, b, None, off), *scan.backward(x, dt, A, Bm, Cm, go, D, z, b, None, None, off)))
        del conv, scan
    assert all(same_bits(a, c) for a, c in zip(*got))
    del base, cols, got
    slots = torch.tensor([5, 0], dtype=torch.int32, device="cuda")
    for dtype, entry in ((torch.bfloat16, (3, 8192)), (torch.float32, (8192, 64))):
        n = 2 ** 31 // (entry[0] * entry[1]) + 8
        pool, small = torch.empty(n, *entry, dtype=dtype, device="cuda"), rand(8, *entry).to(dtype)
        pool[n - 8:] = small
        x = rand(2, 8192).bfloat16()
        ys = []
        for at, s in ((pool, slots + (n - 8)), (small, slots)):
            if dtype is torch.bfloat16:
                ys.append(lm.ShortConvStep(2, 8192).step(x, b.new_ones(8192, 4), at, None, s))
            else:
                m = x[:, :64].contiguous()
                ys.append(lm.SelScanStep(2, 8192, 64).step(x, x, -b.new_ones(entry), m, m, at, None, x, None, s))
        assert same_bits(*ys) and same_bits(pool[n - 8:], small)
        del pool


def test_graph_takes_new_offsets():
    """Offsets are read on the device: a captured call follows what they hold when it is replayed."""
    from adjoint_gradients_long_gb300 import lm
    x, _ = scan_case(12, 3, 160, 24, 8, True, lengths=[50, 60, 50])
    s = lm.SelScan(3, 160, 24, 8, packed=True, backward=True)
    scan_run(s, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s1, r = scan_run(s, x)
    for lengths in ([1, 0, 159], [100, 30, 30]):
        x["offsets"].copy_(offsets_of(lengths))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in (y, s1, *r)]
        fresh = lm.SelScan(3, 160, 24, 8, packed=True, backward=True)
        a, b, g = scan_run(fresh, x)
        assert all(torch.equal(o, p) for o, p in zip(got, (a, b, *g)))
