"""Sampling where its definition's words end: a temperature without end, min-p above one, distances beyond fp32."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_sample import check, logits  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [7, 3000, 40000])
def test_infinite_temperature(V, bf16):
    """All finite logits weigh the same; minus infinity stays masked."""
    x, u = logits(4, V, bf16, V)
    x[1, ::2] = -math.inf
    x[2, 1:] = -math.inf
    for kw in (dict(), dict(top_k=[3] * 4), dict(top_p=[0.5] * 4), dict(min_p=[0.5] * 4), dict(top_k=[V // 2 + 1] * 4, top_p=[0.25] * 4)):
        check(x, u, temperature=[math.inf] * 4, **kw)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [7, 3000, 40000])
def test_min_p_above_one_is_one(V, bf16):
    x, _ = logits(1, V, bf16, V)
    x[0, [1, V // 2, V - 1]] = 30.0                         # three of the largest: none is dropped
    u = [0.0, 0.2, 0.4, 0.6, 0.8, 0.9999]
    got = check(x.expand(6, V).contiguous(), u, min_p=[1.0, 1.5, 2.0, 1e30, math.inf, 1.0])
    assert got == [1, 1, V // 2, V // 2, V - 1, V - 1]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T", [1.0, 1e37, 3e38])
def test_distances_beyond_fp32_are_masked(T, bf16):
    """The largest and the lowest value lie further apart than fp32 holds: nothing is left of the lowest at any temperature."""
    from adjoint_gradients_long_gb300 import lm
    xt = torch.bfloat16 if bf16 else torch.float32
    f = lambda v, dt=torch.float32: torch.full((2,), v, dtype=dt, device="cuda")  # noqa: E731
    for V in (5, 9000):
        x = torch.full((2, V), torch.finfo(xt).min, dtype=xt, device="cuda")
        x[0, 3] = x[1, V - 1] = torch.finfo(xt).max
        s = lm.Sampler(2, V, x_bf16=bf16)
        for kw in (dict(), dict(top_k=f(4, torch.int32)), dict(top_p=f(0.999))):
            for u in (0.0, 1 - 2.0 ** -24):
                token, logp = s.sample(x, f(u), temperature=f(T), **kw)
                assert token.tolist() == [3, V - 1] and (logp == 0).all()
