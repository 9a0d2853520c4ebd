"""The small language model runs the operators together: its gradients against differences of
its own loss, training, and answers that agree with the prompt pass."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


def test_gradients_against_differences():
    """The loss along the gradient's own direction: fourth-order central differences at steps that
    move the loss by about half a percent and 1 percent (second-order ones are 8 percent off there
    for W_in, whose gradient is small against its curvature).  bf16 activations put noise of 2^-9
    on values whose mean is taken over 512 tokens; 5 percent of the derivative covers it."""
    from adjoint_gradients_long_gb300.lm_train import TinyLm, cycle_tokens
    m = TinyLm(200, 2, 256, H=2, D=64, Hk=1)
    tok = cycle_tokens(2, 256, 23, 200)
    loss = m.loss_and_grads(tok).item()
    grads = [g.clone() for g in m.grads]
    for i, g in enumerate(grads):
        n2 = g.double().square().sum().item()
        h = 0.005 * loss / n2
        keep = m.params[i].clone()

        def at(k):
            m.params[i].copy_(keep).add_(g, alpha=k * h)
            return m.loss_and_grads(tok).item()
        got = (8 * (at(1) - at(-1)) - (at(2) - at(-2))) / (12 * h)
        m.params[i].copy_(keep)
        assert abs(got - n2) <= 0.05 * n2, i


def test_trains_and_answers():
    from adjoint_gradients_long_gb300.lm_train import TinyLm, cycle_tokens
    B, T, vocab, period = 4, 256, 300, 19
    m = TinyLm(vocab, B, T)
    tok = cycle_tokens(B, T, period, vocab)
    losses = [m.step(tok)[0].item() for _ in range(60)]
    assert losses[-1] < 0.2 * losses[0]
    seq = tok[0]
    got = m.answer(seq[:80], 10)
    assert [t for t, _, _ in got] == seq[80:90].tolist()
    # the same positions through the prompt pass: the chunked form and the single steps agree
    from adjoint_gradients_long_gb300 import lm
    probs = lm.TokenLogProbs(1, vocab, top=4)
    for i in (0, 4, 9):
        logits, _ = m.prompt(seq[:80 + i])
        r = probs.forward(logits, seq[80 + i:81 + i])
        assert r.top_id[0, 0].item() == got[i][0]
        assert abs(r.logp[0].item() - got[i][1]) <= 0.05 * max(1.0, abs(got[i][1]))
