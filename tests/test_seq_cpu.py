"""The short convolution, the selective scan and sampling without a GPU: the fp64 oracle against
differences, and the refusals of the C ABI and of the Python objects (nothing is launched)."""
import ctypes
import math

import numpy as np
import pytest

from adjoint_gradients_long_gb300 import build as adj_build, lib
from oracle import seq as oseq


@pytest.fixture(scope="module")
def L():
    adj_build.build()
    return lib.load()


FAKE, BIG = 1 << 40, 1 << 50          # an aligned address that validation never dereferences
SEQS = [(0, 4), (4, 4), (4, 9), (9, 10)]


# ---------------------------------------------------------------- the oracle
def derivative(f, args, name, u):
    """The complex-step derivative of f(**args) in direction u of one argument (exact to rounding)."""
    return f(**{n: (x + 1e-30j * u if n == name else x) for n, x in args.items()}).imag / 1e-30


def test_scan_gradient_is_the_derivative():
    r = np.random.default_rng(1)
    P, N, R, B = 3, 2, 10, len(SEQS)
    args = dict(x=r.normal(size=(R, P)), dt=r.normal(size=(R, P)), A=-r.random((P, N)), Bm=r.normal(size=(R, N)),
                Cm=r.normal(size=(R, N)), D=r.normal(size=P), z=r.normal(size=(R, P)), bias=r.normal(size=P), s0=r.normal(size=(B, P, N)))
    go, ds1 = r.normal(size=(R, P)), r.normal(size=(B, P, N))
    grads = dict(zip(args, oseq.scan_backward(*args.values(), SEQS, go, ds1)))

    def f(**a):
        y, s1, _ = oseq.scan_forward(*(a[n] for n in args), SEQS)
        return np.sum(y * go) + np.sum(s1 * ds1)
    for n in args:
        u = r.normal(size=args[n].shape)
        want, got = derivative(f, args, n, u), np.sum(grads[n] * u)
        assert abs(got - want) <= 1e-10 * abs(want) + 1e-12, n


def test_conv_gradient_is_the_derivative():
    r = np.random.default_rng(2)
    P, R, B = 3, 10, len(SEQS)
    for W in (2, 3, 4):
        args = dict(x=r.normal(size=(R, P)), w=r.normal(size=(P, W)), bias=r.normal(size=P), s0=r.normal(size=(B, W - 1, P)))
        go, ds1 = r.normal(size=(R, P)), r.normal(size=(B, W - 1, P))
        for act in (True, False):
            grads = dict(zip(args, oseq.conv_backward(*args.values(), SEQS, go, ds1, act)))

            def f(**a):
                y, s1 = oseq.conv_forward(*(a[n] for n in args), SEQS, act)
                return np.sum(y * go) + np.sum(s1 * ds1)
            for n in args:
                u = r.normal(size=args[n].shape)
                want, got = derivative(f, args, n, u), np.sum(grads[n] * u)
                assert abs(got - want) <= 1e-10 * abs(want) + 1e-12, (W, act, n)


def test_states_carry_over():
    """Two halves with the state between them are the whole."""
    r = np.random.default_rng(3)
    P, N, R = 2, 3, 9
    x, dt, A, B, C = r.normal(size=(R, P)), r.normal(size=(R, P)), -r.random((P, N)), r.normal(size=(R, N)), r.normal(size=(R, N))
    y, s, _ = oseq.scan_forward(x, dt, A, B, C, None, None, None, None, [(0, R)])
    y1, s1, _ = oseq.scan_forward(x[:4], dt[:4], A, B[:4], C[:4], None, None, None, None, [(0, 4)])
    y2, s2, _ = oseq.scan_forward(x[4:], dt[4:], A, B[4:], C[4:], None, None, None, s1, [(0, 5)])
    assert np.allclose(np.concatenate([y1, y2]), y, rtol=1e-13) and np.allclose(s2, s, rtol=1e-13)
    w = r.normal(size=(P, 4))
    y, s = oseq.conv_forward(x, w, None, None, [(0, R)])
    y1, s1 = oseq.conv_forward(x[:2], w, None, None, [(0, 2)])
    y2, s2 = oseq.conv_forward(x[2:], w, None, s1, [(0, 7)])
    assert np.allclose(np.concatenate([y1, y2]), y, rtol=1e-13) and (s2 == s).all()


def test_sampling_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    draw = lambda u, **kw: oseq.sample(x, u, **kw)[0]  # noqa: E731
    assert [draw(u) for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.999)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [draw(u, top_k=2) for u in (0.0, 0.57, 0.58)] == [1, 1, 3]
    assert {draw(u / 50, top_p=0.65) for u in range(50)} == {1, 3}
    assert {draw(u / 50, min_p=0.45) for u in range(50)} == {1, 2, 3}
    assert draw(0.9, temperature=0.0) == 1 and draw(0.9, top_p=0.0) == 1 and draw(0.9, min_p=5.0) == 1
    assert abs(oseq.sample(x, 0.1, top_k=2)[1] - math.log(0.4 / 0.7)) < 1e-9
    assert oseq.sample(np.full(3, -np.inf), 0.5) == (-1, -math.inf)
    assert oseq.sample(np.array([0.0, np.nan]), 0.5)[0] == -1 and oseq.sample(x, 0.5, temperature=-1.0)[0] == -1
    assert oseq.sample(np.zeros(5), 0.5, top_k=2)[0] == 1                  # equal values: the lower indices stay


# ---------------------------------------------------------------- refusals of the C ABI
def conv(B=2, T=16, P=16, W=4, dt=lib.BF16, packed=0, act=1, **kw):
    d = lib.conv_dims(B, T, P, W, dt, packed, act)
    for n, x in kw.items():
        setattr(d, n, x)
    return ctypes.byref(d)


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), 2), (dict(T=-1), 2), (dict(P=12), 2), (dict(P=0), 2), (dict(P=1 << 21), 2), (dict(W=1), 2), (dict(W=5), 2),
    (dict(dt=2), 4), (dict(packed=2), 1), (dict(act=3), 1), (dict(reserved=1), 1), (dict(ldx=8), 2), (dict(ldx=20), 3),
    (dict(ldy=20), 3), (dict(ldx=1 << 31), 2), (dict(B=1 << 20, T=1 << 20), 2), (dict(B=1 << 31), 2),
])
def test_conv_dims_refused(L, bad, status):
    assert L.adj_conv_fwd(conv(**bad), FAKE, FAKE, None, None, FAKE if bad.get("packed") else None, FAKE, None, None) == status
    assert L.adj_conv_workspace_bytes(conv(**bad)) == 0


A1, A2 = FAKE + (1 << 20), FAKE + (2 << 20)


def test_conv_pointers_refused(L):
    args = dict(x=FAKE, w=FAKE, bias=None, s0=None, off=None, y=A1, s1=None)

    def fwd(d=None, **kw):
        return L.adj_conv_fwd(d or conv(), *{**args, **kw}.values(), None)
    for n in ("x", "w", "y"):
        assert fwd(**{n: None}) == 1 and fwd(**{n: FAKE + 8}) == 3
    for n in ("bias", "s0", "s1"):
        assert fwd(**{n: FAKE + 8}) == 3
    assert fwd(off=FAKE) == 1 and fwd(conv(packed=1)) == 1                 # offsets and packed together
    assert fwd(y=FAKE) == 1 and fwd(s0=A2, s1=A2) == 1                      # an output that is an input
    assert fwd(conv(packed=1), off=FAKE + 4) == 3
    assert fwd(conv(B=0)) == 0
    need = L.adj_conv_workspace_bytes(conv())
    back = dict(x=FAKE, w=FAKE, bias=None, s0=None, off=None, go=FAKE, ds1=None, dx=A1, dw=A1, dbias=None, ds0=None, ws=FAKE)

    def bwd(ws_bytes=BIG, **kw):
        return L.adj_conv_bwd(conv(), *{**back, **kw}.values(), ws_bytes, None)
    for n in ("x", "w", "go", "dx", "dw", "ws"):
        assert bwd(**{n: None}) == 1, n
    for n in ("ds1", "dbias", "ds0", "dw"):
        assert bwd(**{n: FAKE + 8}) == 3, n
    assert bwd(ws=FAKE + 64) == 3 and bwd(ws_bytes=need - 1) == 5
    assert bwd(dx=FAKE) == 1 and bwd(ds1=A2, ds0=A2) == 1 and bwd(s0=A2, ds0=A2) == 1

    def step(d=None, x=FAKE, state=FAKE, n=4, slots=FAKE):
        return L.adj_conv_step(d or conv(), x, FAKE, None, state, n, slots, FAKE, None)
    assert step(x=None) == 1 and step(state=None) == 1 and step(state=FAKE + 8) == 3 and step(slots=FAKE + 2) == 3
    assert step(n=1, slots=None) == 2 and step(n=-1) == 2 and step(conv(B=0)) == 0


def ssm(B=2, T=16, P=16, N=16, dt=lib.BF16, packed=0, **kw):
    d = lib.ssm_dims(B, T, P, N, dt, packed)
    for n, x in kw.items():
        setattr(d, n, x)
    return ctypes.byref(d)


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), 2), (dict(T=-1), 2), (dict(P=4), 2), (dict(N=4), 2), (dict(N=24), 2), (dict(N=128), 2), (dict(dt=7), 4),
    (dict(packed=-1), 1), (dict(lddt=8), 2), (dict(ldz=12), 2), (dict(ldB=18), 3), (dict(ldC=15), 2), (dict(ldy=20), 3),
    (dict(B=1 << 16, T=1 << 16), 2), (dict(T=1 << 31), 2),
])
def test_scan_dims_refused(L, bad, status):
    assert L.adj_ssm_fwd(ssm(**bad), *[FAKE] * 5, None, None, None, None, FAKE if bad.get("packed") else None, FAKE, None, FAKE, BIG,
                         None) == status
    assert L.adj_ssm_workspace_bytes(ssm(**bad), lib.OP_SSM_FWD) == 0


def test_scan_pointers_refused(L):
    args = dict(x=FAKE, dt=FAKE, A=FAKE, Bm=FAKE, Cm=FAKE, D=None, z=None, bias=None, s0=None, off=None, y=A1, s1=None, ws=FAKE)

    def fwd(d=None, ws_bytes=BIG, **kw):
        return L.adj_ssm_fwd(d or ssm(), *{**args, **kw}.values(), ws_bytes, None)
    for n in ("x", "dt", "A", "Bm", "Cm", "y", "ws"):
        assert fwd(**{n: None}) == 1 and fwd(**{n: FAKE + 8}) == 3, n
    for n in ("D", "z", "bias", "s0", "s1"):
        assert fwd(**{n: FAKE + 8}) == 3, n
    assert fwd(off=FAKE) == 1 and fwd(ssm(packed=1)) == 1 and fwd(ssm(B=0)) == 0
    assert fwd(y=FAKE) == 1 and fwd(z=A1) == 1 and fwd(s0=A2, s1=A2) == 1
    need = L.adj_ssm_workspace_bytes(ssm(), lib.OP_SSM_FWD)
    assert fwd(ws_bytes=need - 1) == 5
    assert L.adj_ssm_workspace_bytes(ssm(), lib.OP_SSM_BWD) > need and L.adj_ssm_workspace_bytes(ssm(), lib.OP_FWD) == 0
    back = dict(x=FAKE, dt=FAKE, A=FAKE, Bm=FAKE, Cm=FAKE, D=None, z=None, bias=None, s0=None, off=None, go=FAKE, ds1=None, dx=A1,
                ddt=A1, dA=A1, dB=A1, dC=A1, dD=None, dz=None, dbias=None, ds0=None, ws=FAKE)

    def bwd(ws_bytes=BIG, **kw):
        return L.adj_ssm_bwd(ssm(), *{**back, **kw}.values(), ws_bytes, None)
    for n in ("x", "dt", "A", "Bm", "Cm", "go", "dx", "ddt", "dA", "dB", "dC", "ws"):
        assert bwd(**{n: None}) == 1, n
    for n in ("ds1", "dD", "dbias", "ds0"):
        assert bwd(**{n: FAKE + 8}) == 3, n
    assert bwd(z=FAKE) == 1 and bwd(dz=A1) == 1                            # z and dz together
    assert bwd(dx=FAKE) == 1 and bwd(dB=FAKE) == 1 and bwd(ds1=A2, ds0=A2) == 1
    assert bwd(ws_bytes=L.adj_ssm_workspace_bytes(ssm(), lib.OP_SSM_BWD) - 1) == 5

    def step(d=None, x=FAKE, state=FAKE, n=4, slots=FAKE):
        return L.adj_ssm_step(d or ssm(), x, FAKE, FAKE, FAKE, FAKE, None, None, None, state, n, slots, FAKE, None)
    assert step(x=None) == 1 and step(state=None) == 1 and step(state=FAKE + 8) == 3 and step(slots=FAKE + 2) == 3
    assert step(n=1, slots=None) == 2 and step(n=-1) == 2 and step(ssm(B=0)) == 0


def test_steps_outputs_apart(L):
    """A step's y is none of what it reads, and neither is its pool."""
    def conv_step(x=FAKE, w=FAKE, bias=None, state=A1, slots=None, y=A2):
        return L.adj_conv_step(conv(), x, w, bias, state, 4, slots, y, None)

    def scan_step(x=FAKE, dt=FAKE, A=FAKE, Bm=FAKE, Cm=FAKE, D=None, z=None, bias=None, state=A1, slots=None, y=A2):
        return L.adj_ssm_step(ssm(), x, dt, A, Bm, Cm, D, z, bias, state, 4, slots, y, None)
    for step, names in ((conv_step, "x w bias slots"), (scan_step, "x dt A Bm Cm D z bias slots")):
        for n in names.split():
            assert step(**{n: A1}) == 1 and step(**{n: A2}) == 1, n
        assert step(state=A2) == 1


def test_scan_workspace_is_bounded(L):
    """Backwards: a state for every tile of tokens, the segments', and partial sums of dB and dC."""
    for P, N, T in ((1024, 16, 65536), (2048, 16, 16384), (8, 64, 100000), (4096, 8, 777)):
        fwd, bwd = (L.adj_ssm_workspace_bytes(ssm(1, T, P, N), op) for op in (lib.OP_SSM_FWD, lib.OP_SSM_BWD))
        tiles, segs = -(-T // (8 if N == 8 else 16)), 152 * 6 + 2
        cols = -(-P // (4 * 512 // N))
        state = 4 * P * N
        assert fwd <= 2 ** 16 + (152 * 3 + 2) * (state + 4 * P + 512)
        assert bwd <= 2 ** 16 + tiles * (state + 4 * P) + segs * (3 * state + 12 * P + 1024) + cols * T * 8 * N


def test_sample_refused(L):
    def call(N=4, V=100, ld=100, dt=lib.BF16, logits=FAKE, u=FAKE, temperature=None, k=None, p=None, q=None, token=FAKE, logp=None, reserved=0):
        d = lib.SampleDims(N, V, ld, dt, reserved)
        return L.adj_sample(ctypes.byref(d), logits, u, temperature, k, p, q, token, logp, None)
    assert call(N=-1) == 2 and call(V=0) == 2 and call(V=lib.SAMPLE_MAX_V + 1, ld=1 << 20) == 2 and call(ld=99) == 2 and call(dt=2) == 4
    assert call(reserved=1) == 1 and call(N=1 << 28) == 2
    assert call(logits=None) == 1 and call(u=None) == 1 and call(token=None) == 1
    assert call(logits=FAKE + 1) == 3 and call(token=FAKE + 4) == 3
    for n in ("u", "temperature", "k", "p", "q", "logp"):
        assert call(**{n: FAKE + 2}) == 3, n
    assert call(N=0) == 0


# ---------------------------------------------------------------- refusals of the Python objects
def test_objects_refuse(L):
    torch = pytest.importorskip("torch")
    from adjoint_gradients_long_gb300 import lm
    z, off = torch.zeros, torch.tensor([0, 3, 8])
    for bad in (dict(P=12), dict(W=5), dict(W=1)):
        with pytest.raises(ValueError):
            lm.ShortConv(**{**dict(B=1, T=8, P=16, W=4), **bad}, device="cpu")
    for bad in (dict(P=12), dict(N=12)):
        with pytest.raises(ValueError):
            lm.SelScan(**{**dict(B=1, T=8, P=16, N=16), **bad}, device="cpu")
        with pytest.raises(ValueError):
            lm.SelScanStep(**{**dict(B=1, P=16, N=16), **bad}, device="cpu")
    for V in (0, lib.SAMPLE_MAX_V + 1):
        with pytest.raises(ValueError):
            lm.Sampler(4, V, device="cpu")
    c = lm.ShortConv(2, 8, 16, x_bf16=False, device="cpu")
    x, w = z(2, 8, 16), z(16, 4)
    for bad in ((z(2, 8, 24), w), (x.bfloat16(), w), (x, z(16, 3)), (x, w.double()), (z(2, 8, 16, 2)[..., 0], w),
                (z(16, 8, 2).permute(2, 1, 0), w), (z(1, 8, 16).expand(2, 8, 16), w), (x, z(4, 16).T), (x, w, z(8)), (x, w, None, z(2, 4, 16)),
                (x, w, None, None, off)):
        with pytest.raises(ValueError):
            c.forward(*bad)
    with pytest.raises(ValueError):
        c.backward(x, w, x)                                                # made without backward
    p = lm.ShortConv(2, 8, 16, x_bf16=False, packed=True, device="cpu")
    for bad in ((z(8, 16), w), (z(8, 16), w, None, None, off.int()), (z(8, 16), w, None, None, off[:2]), (x, w, None, None, off)):
        with pytest.raises(ValueError):
            p.forward(*bad)
    s = lm.SelScan(2, 8, 16, 8, x_bf16=False, device="cpu")
    m, A = z(2, 8, 8), z(16, 8)
    for bad in ((x, x, A, m, z(2, 8, 16)), (x, x, z(8, 16), m, m), (x, x.bfloat16(), A, m, m), (x, x, A, m, m, z(8)), (x, x, A, m, m, None, m),
                (x, x, A, m, m, None, None, None, z(2, 8, 16))):
        with pytest.raises(ValueError):
            s.forward(*bad)
    with pytest.raises(ValueError):
        s.backward(x, x, A, m, m, x)
    st = lm.SelScanStep(2, 16, 8, x_bf16=False, device="cpu")
    x1, m1 = z(2, 16), z(2, 8)
    for bad in (dict(state=z(1, 16, 8)), dict(state=z(3, 8, 16)), dict(state=z(3, 16, 8), slots=z(2, dtype=torch.int64)),
                dict(state=z(3, 16, 8).bfloat16())):
        with pytest.raises(ValueError):
            st.step(x1, x1, A, m1, m1, **bad)
    with pytest.raises(ValueError):
        lm.ShortConvStep(2, 16, x_bf16=False, device="cpu").step(x1, w, z(1, 3, 16))
    t = lm.Sampler(4, 100, x_bf16=False, device="cpu")
    u, lg = z(4), z(4, 100)
    for bad in ((lg.bfloat16(), u), (z(4, 99), u), (z(100, 4).T, u), (z(1, 100).expand(4, 100), u), (lg, z(3)), (lg, u.double()),
                (lg, u, z(3)), (lg, u, None, z(4)), (lg, u, None, None, z(4, dtype=torch.int32))):
        with pytest.raises(ValueError):
            t.sample(*bad)


def test_host_tensors_are_refused(L):
    """Valid calls on host tensors: refused before the library gets a host address."""
    torch = pytest.importorskip("torch")
    from adjoint_gradients_long_gb300 import lm
    z, before = torch.zeros, lib.launch_count()
    x, w, m, A = z(1, 8, 16), z(16, 4), z(1, 8, 8), z(16, 8)
    c = lm.ShortConv(1, 8, 16, x_bf16=False, backward=True, device="cpu")
    s = lm.SelScan(1, 8, 16, 8, x_bf16=False, backward=True, device="cpu")
    t = lm.Sampler(4, 100, x_bf16=False, device="cpu")
    for call in (lambda: c.forward(x, w), lambda: c.backward(x, w, x), lambda: s.forward(x, x, A, m, m),
                 lambda: s.backward(x, x, A, m, m, x), lambda: t.sample(z(4, 100), z(4)),
                 lambda: lm.ShortConvStep(1, 16, x_bf16=False, device="cpu").step(x[:, 0], w, z(1, 3, 16)),
                 lambda: lm.SelScanStep(1, 16, 8, x_bf16=False, device="cpu").step(x[:, 0], x[:, 0], A, m[:, 0], m[:, 0], z(1, 16, 8))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    assert lib.launch_count() == before
