"""Clipping whose blocks do not meet (GPU): the limit of the wait, what the call leaves, and the
next call."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


@pytest.mark.parametrize("inplace", [False, True])
def test_blocks_that_do_not_meet(inplace):
    """The ticket of the last block is spoilt, so that no block takes itself for the last one and every
    wait runs into its limit (a few seconds): no value is scaled, the result is NaN, the status says
    so, and the object works again afterwards."""
    from adjoint_gradients_long_gb300 import lib, lm
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = [torch.randn(n, device="cuda", generator=gen) for n in (5, 1000, 77777)]
    outs = x if inplace else [torch.full_like(t, 9.0) for t in x]
    before = [t.clone() for t in outs]
    want = sum(t.double().square().sum() for t in x).sqrt().item()
    c = lm.GradClip(x, None if inplace else outs)
    c.ws[2] = 1 << 20                            # the ticket: past every block's
    norm, coef = c.clip(1.0)
    assert torch.isnan(norm) and torch.isnan(coef)
    assert all(torch.equal(t, b) for t, b in zip(outs, before))
    assert lib.STATUS[c.status()] == "ADJ_ETIMEOUT"
    assert c.status() == 0
    norm, coef = c.clip(1.0)
    assert abs(norm.item() - want) <= 1e-6 * want and abs(coef.item() - 1 / want) <= 2e-6
    for t, b, y in zip(x, before, outs):
        assert torch.allclose(y, (b if inplace else t) * coef, rtol=1e-6)
    assert c.status() == 0
