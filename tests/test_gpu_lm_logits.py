"""Log probabilities over logits far from zero (GPU, against the fp64 oracle): large finite values
that stand for masked tokens, rows with nothing else, large maxima, large cotangents of the entropy.

Tolerances, row by row:
  lse       3e-7 of it (one rounding of a sum with the largest logit, 2^-24, and one of its storage)
            and 1e-5 for the logarithm of a sum of up to 2^17 terms
  logp, entropy, top list   1e-5 of a value, at least 1e-5: differences x - max are exact to 2^-24
  dlogits   the error of ln p and of the entropy, at most 1e-5 of one, times the cotangents and p;
            and the storage type's rounding of the value, 2^-8 or 1e-5
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import lm as olm  # noqa: E402

pytestmark = pytest.mark.gpu

LOWEST = {True: torch.finfo(torch.bfloat16).min, False: torch.finfo(torch.float32).min}
SHAPES = [(6, 700), (6, 4099), (6, 12001), (6, 70007)]         # one block a row, then clusters of 2 to 8


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


def np64(x):
    return x.detach().double().cpu().numpy()


def close(name, got, want, rel, least):
    with np.errstate(over="ignore"):
        want = want.astype(np.float32).astype(np.float64)      # past its range: infinite
    got = np64(got)
    f = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), f) and np.array_equal(got[~f], want[~f]), (name, got, want)
    err = np.abs(got - want)[f] - rel * np.abs(want[f])
    assert (err <= least).all(), (name, got, want)


def check(x, y, bf16, glp, gent, top=8):
    from adjoint_gradients_long_gb300 import lm
    N, V = x.shape
    p = lm.TokenLogProbs(N, V, x_bf16=bf16, top=top)
    logp, ent, lse, ids, tops = olm.logprob(np64(x), y.cpu().numpy(), top)
    for r in (p.forward(x, y), p.gradient(x, y, glp, gent)):
        close("lse", r.lse, lse, 3e-7, 1e-5)
        close("logp", r.logp, logp, 1e-5, 1e-5)
        close("entropy", r.entropy, ent, 1e-5, 1e-5)
        assert np.array_equal(r.top_id.cpu().numpy(), ids)
        close("top_logp", r.top_logp, tops, 1e-5, 1e-5)
    d = olm.logprob_grad(np64(x), y.cpu().numpy(), np64(glp), np64(gent))
    got = np64(r.dlogits)
    c = (np.abs(np64(glp)) + np.abs(np64(gent)))[:, None]
    assert np.isfinite(got).all()
    assert (np.abs(got - d) <= 1e-5 * c + (2.0 ** -8 if bf16 else 1e-5) * np.abs(d)).all(), np.abs(got - d).max(1)
    return r


def logits(N, V, bf16, seed):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, V, generator=gen) * 3).to(torch.bfloat16 if bf16 else torch.float32).cuda()
    y = torch.randint(-1, V, (N,), generator=gen).cuda()
    return x, y, torch.randn(N, generator=gen).cuda(), torch.randn(N, generator=gen).cuda(), gen


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N,V", SHAPES)
@pytest.mark.parametrize("fill", [-1e4, -65504.0, -1e9, -5e9, -1e10, -1e12, -1e15, -1e20, -1e30, "lowest"])
def test_finite_masks(fill, N, V, bf16):
    """A fill in place of minus infinity: at the head of the row, in all of it, in most of it at
    random, around one value left, at the tail, and in the target."""
    fill = LOWEST[bf16] if fill == "lowest" else fill
    x, y, glp, gent, gen = logits(N, V, bf16, V)
    x[0, :V * 6 // 10] = fill
    x[1] = fill
    x[2][(torch.rand(V, generator=gen) < 0.95).cuda()] = fill
    x[3] = fill
    x[3, V // 3] = 1.5
    x[4, -V // 4:] = fill
    x[5, ::2] = fill
    y[5] = 2 * (V // 5)
    check(x, y, bf16, glp, gent)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N,V", SHAPES)
@pytest.mark.parametrize("big", [1e4, 3e4, 65536.0, 1e6, 5e9, 1e10, 1e20, 1e38])
def test_large_maxima(big, N, V, bf16):
    """Rows whose largest value is far from zero, or whose values all are, of either sign."""
    x, y, glp, gent, gen = logits(N, V, bf16, V + 1)
    x[0, V // 2] = big
    x[1, ::3] = big
    x[2] = -big
    x[3] = big
    x[4] = ((torch.rand(V, generator=gen) - 0.5) * 2 * big).to(x.dtype).cuda()
    x[5] = (big * (1 + torch.rand(V, generator=gen) / 64)).to(x.dtype).cuda()
    check(x, y, bf16, glp, gent)


@pytest.mark.parametrize("bf16", [False, True])
def test_maxima_around_one_scale(bf16):
    """Parts of one row whose maxima lie on both sides of a power of two, for every power: the
    parts' sums are measured from different references."""
    V = 20000
    for e in range(8, 40, 2):
        x = torch.full((4, V), -3e38, device="cuda")
        m = 2.0 ** e
        gen = torch.Generator().manual_seed(e)
        near = m + m * 2.0 ** -20 * torch.randn(V, generator=gen) if not bf16 else m * (1 + torch.randint(-2, 3, (V,), generator=gen) / 128)
        x[0] = near.cuda()
        x[1] = -near.cuda()
        x[2, : V // 2], x[2, V // 2:] = near[: V // 2].cuda(), 0.5
        x[3, ::2] = -near[::2].cuda()
        x = x.to(torch.bfloat16 if bf16 else torch.float32)
        y = torch.tensor([5, V - 2, 17, 4], device="cuda")
        check(x, y, bf16, torch.ones(4, device="cuda"), torch.full((4,), 0.5, device="cuda"))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("gent", [4.0, -8.0, 1e4, -1e4, 1e20])
@pytest.mark.parametrize("N,V", [(6, 700), (6, 12001)])
def test_large_entropy_cotangent(N, V, gent, bf16):
    """Masked tokens of a confident row get no gradient, whatever the cotangent."""
    x, y, glp, ge, _ = logits(N, V, bf16, V + 2)
    x[:3, 5] = 40
    ge[:] = gent
    for n, low in enumerate((float("-inf"), LOWEST[bf16], -1e30)):
        x[n, V // 2:] = low
        x[3 + n, 1::2] = low
    y[:] = torch.tensor([5, 7, -1, 0, 2, 4], device="cuda")
    r = check(x, y, bf16, glp, ge)
    for n in range(3):
        assert (r.dlogits[n, V // 2:] == 0).all() and (r.dlogits[3 + n, 1::2] == 0).all()
