"""The language-model objects launch on the current CUDA device alone (nothing is launched here)."""
import pytest

torch = pytest.importorskip("torch")

from adjoint_gradients_long_gb300 import build as adj_build, lib, lm  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    adj_build.build()


def test_host_tensors_are_refused():
    """Valid calls on host tensors: refused before the library gets a host address."""
    z = torch.zeros
    before = lib.launch_count()
    a = lm.LinAttn(1, 8, 4, 16, 16, Hk=2, x_bf16=False, backward=True, device="cpu")
    q, v, g = z(1, 8, 2, 16), z(1, 8, 4, 16), z(1, 8, 4)
    s, x = lm.LinStep(2, 4, 16, 16, x_bf16=False, device="cpu"), z(2, 4, 16)
    t = lm.TokenLogProbs(4, 100, x_bf16=False, device="cpu")
    y = z(4, dtype=torch.int64)
    c = lm.GradClip([z(4)])
    for call in (lambda: a.forward(q, q, v, g), lambda: a.backward(q, q, v, g, v),
                 lambda: s.step(x, x, x, z(2, 4), z(2, 4, 16, 16)), lambda: t.forward(z(4, 100), y),
                 lambda: t.gradient(z(4, 100), y, z(4)), lambda: c.clip(1.0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError):
        lm.TokenLogProbs(4, 100, x_bf16=False, device="cpu:0").forward(z(4, 100), y)
    assert lib.launch_count() == before


def test_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    assert lib.raw_stream(torch.device("cuda", 0)) == 0
    with pytest.raises(ValueError, match="cuda:1"):
        lib.raw_stream(torch.device("cuda", 1))


def test_clip_refuses_what_no_launch_can_cover():
    """A tensor of more chunks than a launch counts: refused by its size (nothing is launched)."""
    for n in (1 << 40, 1 << 42, (1 << 43) - 1):
        segs = (lib.GradSeg * 1)(lib.GradSeg(1 << 40, 1 << 40, n, lib.F32, 0))
        assert lib.load().adj_grad_clip(segs, 1, 1.0, 1 << 40, 1 << 40, 1 << 50, None) == 2


def test_backward_workspace_follows_the_heads():
    """Small heads keep small states: what the gradients need beyond the forward pass is the kept
    states of both directions, two dense parts and a third in pieces of 32 columns."""
    def need(Dk, Dv, op, T=131072, H=64):
        return lib.lin_workspace_bytes(lib.lin_dims(1, T, H, H, Dk, Dv), op)
    for Dk, Dv in ((8, 8), (64, 64), (128, 128), (72, 40), (8, 128)):
        parts = 2 * Dk * Dv + Dk * ((Dv + 31) // 32 * 32)          # values of a state, both directions alike
        growth = need(Dk, Dv, lib.OP_LIN_BWD) - need(Dk, Dv, lib.OP_LIN_FWD)
        assert growth <= 1.2 * 2 * 2 * (131072 // 128) * 64 * parts + 2 ** 20, (Dk, Dv)
