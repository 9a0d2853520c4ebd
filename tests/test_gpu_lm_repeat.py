"""The small language model's gradients have the same bits on every run (GPU)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


def test_gradients_repeat():
    """Tokens that occur hundreds of times: the sums of their rows are taken in one order."""
    from adjoint_gradients_long_gb300.lm_train import TinyLm, cycle_tokens
    m = TinyLm(200, 4, 512, H=2, D=64)
    tok = cycle_tokens(4, 512, 5, 200)
    m.loss_and_grads(tok)
    first = [g.clone() for g in m.grads]
    for _ in range(10):
        m.loss_and_grads(tok)
        assert all(torch.equal(g, f) for g, f in zip(m.grads, first))
