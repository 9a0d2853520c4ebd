"""How far linear attention of bf16 layers is from the fp64 oracle (GPU): as far as the storage of its
results and sums in 32 bits make it, and no further.

Bounds (relative, Frobenius):
  s1        2.5e-7: the tensor cores' accumulator drops what is below its last bit.  A sum over a chunk
            grows over 8 steps of 16 tokens, each of which loses half of a last bit of what is there on
            average, half of 8.5e-8 of it; the smaller parts of the keys add up before.  And the fp32
            roundings of the state.
  ds0       6.5e-7: the same with a chunk in two halves, whose smaller parts also meet the larger one
            of the half before: 16 steps
  o dq dk dv  2.0e-3: one rounding to bf16 of a normal value is 1.66e-3, two are 2.35e-3
  dg        1e-6: sums of products of two such accumulators each, 2 x 2.4e-7 and 2.4e-7 + 4.5e-7 in the
            terms with a state; the states themselves to 2^-24
"""
import pytest

torch = pytest.importorskip("torch")

from conftest import rel_fro  # noqa: E402
from oracle import lm as olm  # noqa: E402
from test_gpu_lm_decays import inputs, np64  # noqa: E402

pytestmark = pytest.mark.gpu

STATE, ADJOINT, ONE_ROUNDING, DECAY = 2.5e-7, 6.5e-7, 2.0e-3, 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


def errors(B, T, H, Hk, Dk, Dv, seed, mean=3.0):
    """mean: of the gates' arguments (3: decays around 0.95 a token; 12: hardly any)."""
    from adjoint_gradients_long_gb300 import lm
    x = inputs(B, T, H, Hk, Dk, Dv, True, seed, lambda gen, s: torch.log(torch.sigmoid(torch.randn(s, generator=gen) + mean)))
    a = lm.LinAttn(B, T, H, Dk, Dv, Hk=Hk, scale=Dk ** -0.5, backward=True)
    got = [y.clone() for y in a.forward(x["q"], x["k"], x["v"], x["g"], x["s0"])]
    got += a.backward(x["q"], x["k"], x["v"], x["g"], x["go"], x["s0"], x["ds1"])
    h = {m: np64(y) for m, y in x.items()}
    ref = [*olm.lin_forward(h["q"], h["k"], h["v"], h["g"], Dk ** -0.5, h["s0"]),
           *olm.lin_backward(h["q"], h["k"], h["v"], h["g"], Dk ** -0.5, h["go"], h["s0"], h["ds1"])]
    e = {m: rel_fro(np64(y), r) for m, y, r in zip(("o", "s1", "dq", "dk", "dv", "dg", "ds0"), got, ref)}
    print(f"{B}x{T}, {H}/{Hk} heads of {Dk} and {Dv}: " + " ".join(f"{m}={v:.2e}" for m, v in e.items()))
    return e


SIZES = [(1, 77, 4, 4, 64, 64), (2, 128, 4, 4, 128, 128), (1, 300, 4, 2, 64, 64), (2, 500, 8, 2, 96, 64), (1, 1100, 2, 1, 64, 128)]


@pytest.mark.parametrize("size", SIZES)
def test_states(size):
    e = errors(*size, seed=size[1])
    assert e["s1"] <= STATE and e["ds0"] <= ADJOINT, e


@pytest.mark.parametrize("size", SIZES + [(2, 7, 4, 4, 128, 128), (1, 40, 4, 2, 72, 104), (2, 300, 2, 2, 128, 128)])
def test_outputs(size):
    e = errors(*size, seed=size[1] + 5)
    assert e["o"] <= ONE_ROUNDING, e


@pytest.mark.parametrize("size", SIZES)
def test_gradients_of_tokens(size):
    e = errors(*size, seed=size[1] + 1)
    assert max(e["dq"], e["dk"], e["dv"]) <= ONE_ROUNDING, e


@pytest.mark.parametrize("size", SIZES)
def test_gradients_of_decays(size):
    e = errors(*size, seed=size[1] + 2)
    assert e["dg"] <= DECAY, e


@pytest.mark.parametrize("size", [(2, 2, 3, 1, 16, 24), (4, 1, 8, 4, 64, 64), (2, 7, 4, 4, 128, 128), (1, 40, 4, 2, 72, 104)])
def test_gradients_of_decays_where_the_state_counts(size):
    """Few tokens between a state and its cotangent: dg is little else than their product."""
    e = errors(*size, seed=size[1] + 3)
    assert e["dg"] <= DECAY, e


@pytest.mark.parametrize("size", [(2, 200, 4, 2, 64, 64), (1, 1000, 2, 2, 128, 128)])
def test_gradients_of_weak_decays(size):
    """States that cross whole chunks."""
    e = errors(*size, seed=size[1] + 4, mean=12.0)
    assert e["dg"] <= DECAY, e
