"""GPU sampling against the definition with Python's whole numbers (oracle/seq.py).

Tokens are equal: the kernel's weights are off by one unit of 2^-40 at most, so a draw differs where u lies
that close to a border, which for the seeded rows here has a chance below 1e-6.  logp: the distance and a
logarithm, each to 2^-23 of values up to 30, and the total's 2^-24: 1e-5.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import seq as oseq  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


def check(x, u, **kw):
    """x [N,V] on the device, u and settings as lists; returns the tokens."""
    from adjoint_gradients_long_gb300 import lm
    N, V = x.shape
    s = lm.Sampler(N, V, x_bf16=x.dtype is torch.bfloat16)
    dev = {n: None if v is None else torch.tensor(v, dtype=torch.int32 if n == "top_k" else torch.float32, device="cuda")
           for n, v in kw.items()}
    token, logp = s.sample(x, torch.tensor(u, dtype=torch.float32, device="cuda"), **dev)
    token, logp = token.tolist(), logp.tolist()
    h = x.double().cpu().numpy()
    for i in range(N):
        one = {n: np.float32(v[i]).item() if n != "top_k" else v[i] for n, v in kw.items() if v is not None}
        want, lp = oseq.sample(h[i], np.float32(u[i]).item(), **one)
        assert token[i] == want, (i, u[i], one)
        assert (math.isnan(lp) and math.isnan(logp[i])) or logp[i] == lp or abs(logp[i] - lp) <= 1e-5 * max(1.0, abs(lp)), (i, logp[i], lp)
    return token


def logits(N, V, bf16, seed, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, V, generator=g) * scale
    return (x.bfloat16() if bf16 else x).cuda(), torch.rand(N, generator=g).tolist()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N,V", [(1, 1), (3, 2), (2, 7), (5, 33), (4, 511), (3, 4097), (1, 32000), (2, 50001), (1, 131072), (160, 300)])
def test_settings(N, V, bf16):
    """Each limit alone, then together, a value a row."""
    x, u = logits(N, V, bf16, V)
    r = np.random.default_rng(V)
    pick = lambda *v: [v[i] for i in r.integers(0, len(v), N)]  # noqa: E731
    check(x, u)
    check(x, u, temperature=pick(0.3, 0.9, 1.7, 0.0))
    check(x, u, top_k=pick(1, 2, 5, 40, V, V + 1, 0, -3))
    check(x, u, top_p=pick(0.1, 0.5, 0.9, 0.999, 1.0))
    check(x, u, min_p=pick(0.0, 0.01, 0.2, 1.0))
    check(x, u, temperature=pick(0.7, 1.0, 2.5), top_k=pick(3, 50, 0), top_p=pick(0.6, 0.95), min_p=pick(0.0, 0.05))


@pytest.mark.parametrize("bf16", [False, True])
def test_every_place_of_the_draw(bf16):
    """u over its whole range on one row: every kept token is met, in order of its index."""
    x, _ = logits(1, 12, bf16, 3, scale=1.0)
    u = [i / 400 for i in range(400)] + [0.0, 1 - 2.0 ** -24]
    kw = dict(top_k=[7] * 402, top_p=[0.97] * 402, temperature=[1.3] * 402)
    got = check(x.expand(402, 12).contiguous(), u, **kw)
    assert got[:400] == sorted(got[:400]) and len(set(got)) >= 5


@pytest.mark.parametrize("bf16", [False, True])
def test_equal_logits(bf16):
    """Rows of equal values, or of two: limits fall inside them, the lower indices stay."""
    xt = torch.bfloat16 if bf16 else torch.float32
    for V in (5, 1000, 40000):
        x = torch.zeros(6, V, dtype=xt, device="cuda")
        x[1, ::3] = 1.0
        x[2, V // 2:] = -1.0
        x[3] = -0.0
        x[4, 1::2] = 0.0078125
        u = [0.0, 0.3, 0.9999, 0.5, 0.77, 0.1]
        check(x, u, top_k=[3, 4, V // 2 + 1, 2, V - 1, V // 3 + 1])
        check(x, u, top_p=[0.5, 0.25, 0.9, 0.01, 0.6, 1.0])
        check(x, u, top_k=[4, 2, 0, 3, V // 2, V], top_p=[0.5, 0.5, 0.99, 0.7, 0.5, 0.3])
        check(x, u, temperature=[0.0] * 6)


@pytest.mark.parametrize("bf16", [False, True])
def test_masks_and_extremes(bf16):
    xt = torch.bfloat16 if bf16 else torch.float32
    low, big = torch.finfo(xt).min, torch.finfo(xt).max
    V, inf, nan = 300, math.inf, math.nan
    x, u = logits(12, V, bf16, 5)
    x[0] = -inf                                             # nothing left
    x[1, 1:] = -inf                                         # one token
    x[2, 7] = nan
    x[3, 299] = inf
    x[4, :290] = -inf
    x[5] = low                                              # the lowest finite values are values
    x[6, :200] = low
    x[7, 3] = big
    x[8, 3:5] = big
    x[8, 5:] = low
    x[9] = low
    x[9, 250] = big
    x[10, ::2] = -inf
    for kw in (dict(), dict(top_k=[5] * 12), dict(top_p=[0.9] * 12), dict(min_p=[0.3] * 12), dict(temperature=[0.0] * 12),
               dict(temperature=[0.01] * 12, top_p=[0.5] * 12), dict(temperature=[50.0] * 12, top_k=[200] * 12, top_p=[0.9] * 12)):
        check(x, u, **kw)


def test_settings_at_their_ends():
    x, u = logits(10, 500, False, 6)
    nan = math.nan
    check(x, u, temperature=[nan, -1.0, 0.0, 1e-30, 1e-40, 1e30, 1e-5, 1.0, 3e38, 0.1])
    check(x, u, top_p=[nan, -1.0, 0.0, 1e-9, 1.0, 2.0, 0.99999994, 0.5, 1e-40, 1.0], top_k=[3] * 10)
    check(x, u, min_p=[nan, -1.0, 0.0, 1e-9, 1.0, 2.0, 0.99999994, 0.5, 1e-40, 1e-13])
    check(x, [0.0, 1.0, -1.0, 2.0, nan, 1 - 2.0 ** -24, 0.5, 1e-40, math.inf, -math.inf], top_p=[0.9] * 10)


@pytest.mark.parametrize("bf16", [False, True])
def test_temperature_of_either_zero(bf16):
    for V in (3, 500, 20000):
        x, u = logits(2, V, bf16, 8)
        want = check(x, u, temperature=[0.0] * 2)
        assert check(x, u, temperature=[-0.0] * 2) == want == x.argmax(1).tolist()
        check(x, u, temperature=[-0.0] * 2, top_k=[2] * 2, top_p=[0.5] * 2, min_p=[0.1] * 2)


def test_rows_strided_and_ragged():
    """Rows at every alignment, and a row alone or in a batch: the same token."""
    from adjoint_gradients_long_gb300 import lm
    for bf16 in (False, True):
        wide, u = logits(6, 3001, bf16, 7)
        for a, V in ((1, 2990), (3, 777), (8, 64), (5, 1)):
            check(wide[:, a:a + V], u, top_k=[20] * 6, top_p=[0.9] * 6)
        x, u = logits(300, 9000, bf16, 8)
        t = lambda v, dt=torch.float32: torch.tensor(v, dtype=dt, device="cuda")  # noqa: E731
        kw = [("top_k", t([50] * 300, torch.int32)), ("top_p", t([0.9] * 300))]
        all_rows = lm.Sampler(300, 9000, x_bf16=bf16).sample(x, t(u), **dict(kw))[0].tolist()
        one = lm.Sampler(1, 9000, x_bf16=bf16)
        for i in (0, 17, 299):
            assert one.sample(x[i:i + 1], t(u[i:i + 1]), **{n: v[i:i + 1] for n, v in kw})[0].item() == all_rows[i]


def test_rows_past_32_bits():
    from adjoint_gradients_long_gb300 import lm
    N, V, ld = 1100, 50, 1 << 21
    wide = torch.empty(N, ld, dtype=torch.bfloat16, device="cuda")[:, ld - 99:][:, :V]
    x, u = logits(N, V, True, 9)
    wide.copy_(x)
    assert (N - 1) * ld > 2 ** 31
    s, p, u = lm.Sampler(N, V), torch.full((N,), 0.9, device="cuda"), torch.tensor(u, dtype=torch.float32, device="cuda")
    token, logp = (o.clone() for o in s.sample(x, u, top_p=p))
    again, logp2 = s.sample(wide, u, top_p=p)
    assert torch.equal(token, again) and torch.equal(logp, logp2)


def test_graph_takes_new_numbers():
    from adjoint_gradients_long_gb300 import lm
    x, u = logits(4, 8000, True, 9)
    s, ut = lm.Sampler(4, 8000), torch.tensor(u, device="cuda")
    s.sample(x, ut)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.sample(x, ut)
    for seed in (1, 2):
        y, v = logits(4, 8000, True, seed)
        x.copy_(y)
        ut.copy_(torch.tensor(v))
        graph.replay()
        got = s.token.tolist()
        assert got == check(y, v)
