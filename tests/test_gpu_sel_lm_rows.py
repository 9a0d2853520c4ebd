"""The selective language model with batches that shrink: rows behind (or before) the documents of a step hold
what an older call left in the operators' outputs, and reach no gradient."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


T, DOCS = 448, 5


def model():
    from adjoint_gradients_long_gb300.lm_train import SelLm
    return SelLm(200, DOCS, T, P=64)


def batch(lengths, before, seed):
    gen = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, 200, (T,), generator=gen)
    targets = torch.full((T,), -1, dtype=torch.int64)
    targets[before:before + sum(lengths)] = torch.randint(0, 200, (sum(lengths),), generator=gen)
    offsets = torch.tensor([before, *lengths]).cumsum(0)
    return tokens.cuda(), targets.cuda(), offsets.cuda()


LONG = [100, 90, 128, 60, 70]


@pytest.mark.parametrize("lengths,before", [([30, 0, 61, 2, 1], 0), ([130, 0, 61, 0, 1], 37), ([0, 0, 0, 0, 3], 0), ([1, 0, 0, 0, 0], T - 1)])
def test_a_shorter_batch_after_a_longer_one(lengths, before):
    """The loss and all gradients are those of a model that has seen no other batch, bit for bit."""
    assert sum(LONG) == T
    short = batch(lengths, before, 2)
    fresh = model()
    want = [fresh.loss_and_grads(*short), *fresh.grads]
    m = model()
    m.loss_and_grads(*batch(LONG, 0, 1))
    assert all(torch.equal(a, b) for a, b in zip([m.loss_and_grads(*short), *m.grads], want))


def test_values_that_are_not_finite_in_rows_of_no_document():
    """What an older call left may be anything."""
    short = batch([30, 0, 61, 2, 1], 5, 2)
    fresh = model()
    want = [fresh.loss_and_grads(*short), *fresh.grads]
    assert all(torch.isfinite(w).all() for w in want)
    for bad in (float("nan"), float("inf")):
        m = model()
        m.loss_and_grads(*short)                            # makes the gradients of every layout
        for o in (m.conv.y, m.scan.y, *m.conv._strided.values(), *m.scan._strided.values()):
            o.fill_(bad)
        assert all(torch.equal(a, b) for a, b in zip([m.loss_and_grads(*short), *m.grads], want))
