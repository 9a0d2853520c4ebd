"""Linear attention gives the same bits on every run (GPU)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


def inputs(B, T, H, Hk, Dk, Dv, bf16, seed, g):
    gen = torch.Generator().manual_seed(seed)
    xt = torch.bfloat16 if bf16 else torch.float32
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = dict(q=n(B, T, Hk, Dk).to(xt), k=(n(B, T, Hk, Dk) / Dk ** 0.5).to(xt), v=n(B, T, H, Dv).to(xt),
             go=n(B, T, H, Dv).to(xt), s0=n(B, H, Dk, Dv), ds1=n(B, H, Dk, Dv), g=g(gen, (B, T, H)))
    return {m: y.cuda() for m, y in x.items()}


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,T,H,Hk,D", [(2, 333, 4, 2, 64), (1, 2500, 16, 16, 128), (3, 700, 40, 10, 96)])
def test_same_bits_again_and_on_another_stream(B, T, H, Hk, D, bf16):
    """The same inputs give the same bits, whatever the outputs held before, on the current stream
    and on another one."""
    from adjoint_gradients_long_gb300 import lm
    gate = lambda gen, s: torch.log(torch.sigmoid(torch.randn(s, generator=gen) + 3))  # noqa: E731
    x = inputs(B, T, H, Hk, D, D, bf16, T, gate)
    a = lm.LinAttn(B, T, H, D, D, Hk=Hk, x_bf16=bf16, backward=True)

    def run():
        for y in (a.o, a.s1, a.dq, a.dk, a.dv, a.dg, a.ds0):
            y.fill_(float("nan"))
        args = (x["q"], x["k"], x["v"], x["g"])
        return [y.clone() for y in (*a.forward(*args, x["s0"]), *a.backward(*args, x["go"], x["s0"], x["ds1"]))]
    first = run()
    for _ in range(10):
        for y, z in zip(run(), first):
            assert torch.equal(y, z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [run() for _ in range(10)]
    torch.cuda.current_stream().wait_stream(side)
    for outs in again:
        for y, z in zip(outs, first):
            assert torch.equal(y, z)
    assert a.status() == 0
