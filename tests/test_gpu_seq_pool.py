"""Single tokens with a pool of states that has no entries: every slot is padding."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


@pytest.mark.parametrize("bf16", [False, True])
def test_a_pool_without_entries(bf16):
    from adjoint_gradients_long_gb300 import lm
    xt = torch.bfloat16 if bf16 else torch.float32
    slots = torch.tensor([0, -1, 7], dtype=torch.int32, device="cuda")
    x, m = torch.ones(3, 24, dtype=xt, device="cuda"), torch.ones(3, 16, dtype=xt, device="cuda")
    conv = lm.ShortConvStep(3, 24, x_bf16=bf16)
    conv.y.fill_(7.0)
    y = conv.step(x, torch.ones(24, 4, device="cuda"), torch.empty(0, 3, 24, dtype=xt, device="cuda"), None, slots)
    assert (y == 0).all()
    scan = lm.SelScanStep(3, 24, 16, x_bf16=bf16)
    scan.y.fill_(7.0)
    y = scan.step(x, x, -torch.ones(24, 16, device="cuda"), m, m, torch.empty(0, 24, 16, device="cuda"), torch.ones(24, device="cuda"), x,
                  None, slots)
    assert (y == 0).all()
    with pytest.raises(ValueError):                         # without slots three entries are needed
        conv.step(x, torch.ones(24, 4, device="cuda"), torch.empty(0, 3, 24, dtype=xt, device="cuda"))
