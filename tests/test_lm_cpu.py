"""The language-model operators without a GPU: the fp64 oracle against differences, and the
refusals of the C ABI and of the Python objects (nothing is launched)."""
import ctypes

import numpy as np
import pytest

from adjoint_gradients_long_gb300 import build as adj_build, lib
from oracle import lm as olm


@pytest.fixture(scope="module")
def L():
    adj_build.build()
    return lib.load()


FAKE, BIG = 1 << 40, 1 << 50          # an aligned address that validation never dereferences


# ---------------------------------------------------------------- the oracle
def _lin_inputs(seed, B=2, T=7, H=4, Hk=2, Dk=3, Dv=5):
    r = np.random.default_rng(seed)
    q, k, v = r.normal(size=(B, T, Hk, Dk)), r.normal(size=(B, T, Hk, Dk)), r.normal(size=(B, T, H, Dv))
    g = np.log(1 / (1 + np.exp(-r.normal(size=(B, T, H)) - 1)))
    return dict(q=q, k=k, v=v, g=g, s0=r.normal(size=(B, H, Dk, Dv))), r.normal(size=(B, T, H, Dv)), r.normal(size=(B, H, Dk, Dv))


def test_lin_gradient_is_the_derivative():
    """Complex-step derivatives (exact to rounding) of <o, go> + <s1, ds1> in a random direction
    of every input, against the reverse recurrence: relative 1e-10, far above rounding."""
    x, go, ds1 = _lin_inputs(1)
    grads = dict(zip(("q", "k", "v", "g", "s0"), olm.lin_backward(x["q"], x["k"], x["v"], x["g"], 0.7, go, x["s0"], ds1)))
    r = np.random.default_rng(2)
    for name in x:
        u = r.normal(size=x[name].shape)
        y = {n: (a + 1e-30j * u if n == name else a) for n, a in x.items()}
        o, s1 = olm.lin_forward(y["q"], y["k"], y["v"], y["g"], 0.7, y["s0"])
        want = (np.sum(o * go) + np.sum(s1 * ds1)).imag / 1e-30
        got = np.sum(grads[name] * u)
        assert abs(got - want) <= 1e-10 * abs(want) + 1e-12, name


def test_lin_reset_forgets():
    x, _, _ = _lin_inputs(3)
    x["g"][:, 4] = -np.inf
    o, s1 = olm.lin_forward(x["q"], x["k"], x["v"], x["g"], 1.0, x["s0"])
    tail = {n: x[n][:, 4:] for n in "qkvg"}
    o2, s2 = olm.lin_forward(tail["q"], tail["k"], tail["v"], tail["g"], 1.0, None)
    assert np.allclose(o[:, 4:], o2, rtol=1e-13) and np.allclose(s1, s2, rtol=1e-13)


def test_logprob_gradient_is_the_derivative():
    """Fourth-order central differences of sum glp logp + gent entropy, step 1e-3: truncation
    1e-12 and rounding 1e-12 relative to values of order one, tolerance 1e-9."""
    r = np.random.default_rng(5)
    x, y = r.normal(size=(3, 9)) * 2, np.array([4, -1, 8])
    glp, gent = r.normal(size=3), r.normal(size=3)
    x[1, 2] = -np.inf
    d = olm.logprob_grad(x, y, glp, gent)
    f = lambda z: float(np.sum(glp * olm.logprob(z, y)[0]) + np.sum(gent * olm.logprob(z, y)[1]))  # noqa: E731
    for n in range(3):
        for j in range(9):
            if x[n, j] == -np.inf:
                assert d[n, j] == 0
                continue
            def at(h):
                z = x.copy()
                z[n, j] += h
                return f(z)
            h = 1e-3
            want = (8 * (at(h) - at(-h)) - (at(2 * h) - at(-2 * h))) / (12 * h)
            assert abs(d[n, j] - want) <= 1e-9


def test_top_order():
    x = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0, 3.0]])
    assert olm.logprob(x, np.array([0]), 5)[3].tolist() == [[1, 2, 5, 4, 0]]


# ---------------------------------------------------------------- refusals of the C ABI
def lin(B=1, T=16, H=4, Hk=4, Dk=16, Dv=16, dt=lib.BF16, **kw):
    d = lib.lin_dims(B, T, H, Hk, Dk, Dv, dt)
    for n, x in kw.items():
        setattr(d, n, x)
    return d


def fwd(d, q=FAKE, o=FAKE, s0=None, ws=FAKE, ws_bytes=BIG):
    return lib.load().adj_lin_fwd(ctypes.byref(d), q, FAKE, FAKE, FAKE, s0, o, FAKE, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), 2), (dict(T=-1), 2), (dict(Hk=3), 2), (dict(Hk=0), 2), (dict(Dk=12), 2), (dict(Dk=136), 2),
    (dict(Dv=0), 2), (dict(B=65536), 2), (dict(dt=2), 4), (dict(ldq=56), 2), (dict(ldv=68), 3),
    (dict(scale=float("nan")), 1),
])
def test_lin_dims_refused(L, bad, status):
    d = lin(**bad)
    assert fwd(d) == status
    assert lib.lin_workspace_bytes(d, lib.OP_LIN_FWD) == 0


def test_lin_pointers_refused(L):
    d = lin()
    assert fwd(d, q=None) == 1 and fwd(d, o=None) == 1 and fwd(d, ws=None) == 1
    assert fwd(d, q=FAKE + 8) == 3 and fwd(d, s0=FAKE + 4) == 3 and fwd(d, ws=FAKE + 128) == 3
    need = lib.lin_workspace_bytes(d, lib.OP_LIN_FWD)
    assert fwd(d, ws_bytes=need - 1) == 5
    assert lib.lin_workspace_bytes(d, lib.OP_LIN_BWD) > need
    assert lib.lin_workspace_bytes(d, lib.OP_FWD) == 0
    assert fwd(lin(B=0)) == 0                                          # nothing to do
    args = [FAKE] * 14

    def bwd(at=None, value=None, ws_bytes=BIG):
        x = list(args[:13])
        if at is not None:
            x[at] = value
        return L.adj_lin_bwd(ctypes.byref(d), *x, ws_bytes, None)
    for i in (0, 1, 2, 3, 5, 7, 8, 9, 10, 12):
        assert bwd(i, None) == 1, i
    assert bwd(6, FAKE + 4) == 3                                       # ds1
    assert bwd(ws_bytes=256) == 5

    def step(state=FAKE, n=4, slots=FAKE, B=4):
        return L.adj_lin_step(ctypes.byref(lin(B=B)), FAKE, FAKE, FAKE, FAKE, state, n, slots, FAKE, None)
    assert step(state=None) == 1 and step(state=FAKE + 4) == 3 and step(slots=FAKE + 2) == 3
    assert step(n=3, slots=None) == 2                                  # fewer slots than sequences
    assert step(n=-1) == 2 and step(B=0) == 0


def test_logprob_refused(L):
    def call(N=4, V=100, ld=100, ldd=100, dt=lib.BF16, top=0, logits=FAKE, targets=FAKE, logp=FAKE, ids=None, tlp=None,
             glp=None, gent=None, dl=None):
        d = lib.logprob_dims(N, V, ld, ldd, dt, top)
        return L.adj_logprob(ctypes.byref(d), logits, targets, logp, FAKE, FAKE, ids, tlp, glp, gent, dl, None)
    assert call(N=-1) == 2 and call(V=0) == 2 and call(ld=99) == 2 and call(dt=5) == 4
    assert call(top=33, ids=FAKE, tlp=FAKE) == 2 and call(V=4, top=5, ids=FAKE, tlp=FAKE) == 2
    assert call(logits=None) == 1 and call(targets=None) == 1
    assert call(top=2) == 1 and call(top=2, ids=FAKE) == 1 and call(ids=FAKE, tlp=FAKE) == 1
    assert call(glp=FAKE) == 1 and call(dl=FAKE) == 1                  # cotangents and gradient together
    assert call(glp=FAKE, dl=FAKE, ldd=99) == 2
    assert call(glp=FAKE, dl=FAKE, ld=101) == 1                        # in place needs one pitch
    assert call(logits=FAKE + 1) == 3 and call(logits=FAKE + 2, dt=lib.F32) == 3 and call(logp=FAKE + 2) == 3
    assert call(N=0) == 0


def test_clip_refused(L):
    def call(seg=(FAKE, FAKE, 10, lib.F32, 0), n=1, max_norm=1.0, out=FAKE, ws=FAKE, ws_bytes=BIG):
        segs = (lib.GradSeg * 1)(lib.GradSeg(*seg))
        return L.adj_grad_clip(segs, n, max_norm, out, ws, ws_bytes, None)
    assert call(n=-1) == 2 and call(out=None) == 1 and call(ws=None) == 1 and call(ws=FAKE + 16) == 3
    assert call(max_norm=-1.0) == 1 and call(max_norm=float("nan")) == 1
    assert call(ws_bytes=lib.clip_workspace_bytes() - 1) == 5
    assert call(seg=(None, FAKE, 10, lib.F32, 0)) == 1 and call(seg=(FAKE, FAKE, -1, lib.F32, 0)) == 2
    assert call(seg=(FAKE, FAKE, 10, 7, 0)) == 4 and call(seg=(FAKE + 2, FAKE, 10, lib.F32, 0)) == 3
    assert L.adj_grad_clip(None, 1, 1.0, FAKE, FAKE, BIG, None) == 1


# ---------------------------------------------------------------- refusals of the Python objects
def test_objects_refuse(L):
    torch = pytest.importorskip("torch")
    from adjoint_gradients_long_gb300 import lm
    z = torch.zeros
    with pytest.raises(ValueError):
        lm.LinAttn(1, 8, 4, 12, 16, device="cpu")
    a = lm.LinAttn(1, 8, 4, 16, 16, Hk=2, x_bf16=False, device="cpu")
    q, v, g = z(1, 8, 2, 16), z(1, 8, 4, 16), z(1, 8, 4)
    for bad in ((z(1, 8, 4, 16), q, v, g), (q.bfloat16(), q, v, g), (q, z(1, 8, 2, 16, 2)[..., 0], v, g),
                (q, q, v, z(1, 8, 5)), (q, q, v, g.double()), (q, q, z(1, 4, 8, 16).transpose(1, 2), g)):
        with pytest.raises(ValueError):
            a.forward(*bad)
    with pytest.raises(ValueError):
        a.forward(q, q, v, g, z(1, 4, 16, 8))
    with pytest.raises(ValueError):
        a.backward(q, q, v, g, v)                                      # made without backward
    s = lm.LinStep(2, 4, 16, 16, x_bf16=False, device="cpu")
    x = z(2, 4, 16)
    with pytest.raises(ValueError):
        s.step(x, x, x, z(2, 4), z(1, 4, 16, 16))                      # one slot for two sequences
    with pytest.raises(ValueError):
        s.step(x, x, x, z(2, 4), z(3, 4, 16, 16), z(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        lm.TokenLogProbs(4, 100, top=33, device="cpu")
    t = lm.TokenLogProbs(4, 100, x_bf16=False, device="cpu")
    y = z(4, dtype=torch.int64)
    for bad in ((z(4, 101), y), (z(4, 100).bfloat16(), y), (z(1, 100).expand(4, 100), y), (z(100, 4).T, y),
                (z(4, 100), y.int())):
        with pytest.raises(ValueError):
            t.forward(*bad)
    with pytest.raises(ValueError):
        t.gradient(z(4, 100), y, z(3))
    with pytest.raises(ValueError):
        lm.GradClip([z(4).double()])
    with pytest.raises(ValueError):
        lm.GradClip([z(4)], [z(5)])
    with pytest.raises(ValueError):
        lm.GradClip([z(4, 4).T])
