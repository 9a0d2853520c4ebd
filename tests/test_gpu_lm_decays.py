"""Linear attention where strong decays follow weak ones inside a block of tokens (GPU, against the
fp64 oracle), and the same bits on every run.

Tolerances as in test_gpu_lm.py: 2e-5 (relative, Frobenius) on fp32 states and gradients of bf16
layers, 8e-3 on bf16 outputs, 1e-5 on fp32 layers.  The decays themselves are differences of sums
that are exact to 2^-46, so that they add one rounding of an exponential, 2^-22.
"""
import pytest

torch = pytest.importorskip("torch")

from conftest import rel_fro  # noqa: E402
from oracle import lm as olm  # noqa: E402

pytestmark = pytest.mark.gpu

F32, BF16_OUT, BF16_STATE = 1e-5, 8e-3, 2e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


def np64(x):
    return x.detach().double().cpu().numpy()


def inputs(B, T, H, Hk, Dk, Dv, bf16, seed, g):
    gen = torch.Generator().manual_seed(seed)
    xt = torch.bfloat16 if bf16 else torch.float32
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = dict(q=n(B, T, Hk, Dk).to(xt), k=(n(B, T, Hk, Dk) / Dk ** 0.5).to(xt), v=n(B, T, H, Dv).to(xt),
             go=n(B, T, H, Dv).to(xt), s0=n(B, H, Dk, Dv), ds1=n(B, H, Dk, Dv), g=g(gen, (B, T, H)))
    return {m: y.cuda() for m, y in x.items()}


def strong_ends(weak, block, low, high):
    """Of every `block` tokens the first `weak` decay little, the others by e^low to e^high."""
    def g(gen, shape):
        gate = torch.log(torch.sigmoid(torch.randn(shape, generator=gen) + 3))
        hard = low + (high - low) * torch.rand(shape, generator=gen)
        t = torch.arange(shape[1])[None, :, None]
        return torch.where(t % block < weak, gate, hard).float()
    return g


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("weak,block,low,high", [(24, 32, -90, -20), (16, 32, -100, -50), (8, 32, -103, -90),
                                                 (100, 128, -100, -50), (4, 8, -60, -30), (1, 2, -103, -100)])
def test_weak_before_strong(weak, block, low, high, bf16):
    from adjoint_gradients_long_gb300 import lm
    B, T, H, Hk, Dk, Dv = 1, 300, 4, 2, 64, 64
    x = inputs(B, T, H, Hk, Dk, Dv, bf16, weak, strong_ends(weak, block, low, high))
    a = lm.LinAttn(B, T, H, Dk, Dv, Hk=Hk, x_bf16=bf16, scale=0.125, backward=True)
    h = {m: np64(y) for m, y in x.items()}
    got = [y.clone() for y in a.forward(x["q"], x["k"], x["v"], x["g"], x["s0"])]
    got += a.backward(x["q"], x["k"], x["v"], x["g"], x["go"], x["s0"], x["ds1"])
    ref = [*olm.lin_forward(h["q"], h["k"], h["v"], h["g"], 0.125, h["s0"]),
           *olm.lin_backward(h["q"], h["k"], h["v"], h["g"], 0.125, h["go"], h["s0"], h["ds1"])]
    out, st = (BF16_OUT, BF16_STATE) if bf16 else (F32, F32)
    errs = {m: (rel_fro(np64(y), r), tol) for m, y, r, tol in
            zip(("o", "s1", "dq", "dk", "dv", "dg", "ds0"), got, ref, (out, st, out, out, out, st, st))}
    print(f"weak {weak} of {block}, {low}..{high}, bf16={bf16}: " + " ".join(f"{m}={e:.1e}" for m, (e, _) in errs.items()))
    bad = {m: f"{e:.2e}" for m, (e, tol) in errs.items() if not e <= tol}
    assert not bad, bad


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


def test_graph_outlives_another_layout():
    """A captured backward pass replays into its own arrays after a call in another layout."""
    from adjoint_gradients_long_gb300 import lm
    B, T, H, D = 2, 200, 2, 64
    gate = lambda gen, s: torch.log(torch.sigmoid(torch.randn(s, generator=gen) + 3))  # noqa: E731
    x = inputs(B, T, H, H, D, D, True, 5, gate)
    wide = torch.cat([x[n].flatten(2) for n in "qkv"], -1)
    apart = [wide[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3)]
    a = lm.LinAttn(B, T, H, D, D, backward=True)
    first = [y.clone() for y in a.backward(x["q"], x["k"], x["v"], x["g"], x["go"])[:4]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.backward(x["q"], x["k"], x["v"], x["g"], x["go"])
    at = [a.dq.data_ptr(), a.dk.data_ptr(), a.dv.data_ptr()]
    outs = a.backward(*apart, x["g"], x["go"])[:4]
    assert [y.stride() for y in outs[:3]] == [y.stride() for y in apart]
    assert all(torch.equal(y, z) for y, z in zip(outs, first))
    g.replay()                                   # into the arrays that the object still holds
    again = a.backward(x["q"], x["k"], x["v"], x["g"], x["go"])
    assert [y.data_ptr() for y in again[:3]] == at
    assert all(torch.equal(y, z) for y, z in zip(again, first))
