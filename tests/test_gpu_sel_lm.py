"""The selective language model runs the convolution, the scan and the sampler together: its gradients
against differences of its own loss, packed documents against each alone, and answers that agree
with the prompt pass."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


LENGTHS = [130, 0, 61, 200, 1]


def batch(model, lengths, seed=0):
    """Random tokens of documents behind one another; rows behind the last have no target."""
    gen = torch.Generator().manual_seed(seed)
    n = sum(lengths)
    tokens = torch.randint(0, model.V, (model.T,), generator=gen)
    targets = torch.full((model.T,), -1, dtype=torch.int64)
    targets[:n] = torch.randint(0, model.V, (n,), generator=gen)
    offsets = torch.tensor([0, *lengths]).cumsum(0)
    return tokens.cuda(), targets.cuda(), offsets.cuda()


def test_gradients_against_differences():
    """The loss along the gradient's own direction, fourth-order central differences: the steps move the
    loss by half a percent and one percent, bf16 activations put noise of 2^-8 on values of which the mean over
    392 tokens is taken; 5 percent of the derivative covers it.  Steps of the recurrence of about 0.7 (a
    dt_bias of zero): with the first ones, 0.001 to 0.1, A's gradient is 3e-8, far below that noise."""
    from adjoint_gradients_long_gb300.lm_train import SelLm
    m = SelLm(200, len(LENGTHS), 448, P=64)
    m.dt_bias.zero_()
    args = batch(m, LENGTHS)
    loss = m.loss_and_grads(*args).item()
    grads = [g.clone() for g in m.grads]
    for i, g in enumerate(grads):
        n2 = g.double().square().sum().item()
        h = 0.005 * loss / n2
        # a step that would change a parameter by more than a tenth of its size is no small one, and A stays negative
        # (an A of 30 grows as e^20 a token)
        h = min(h, 0.1 * (m.params[i].double().norm() + 0.1).item() / n2 ** 0.5)
        if m.params[i] is m.A:
            h = min(h, 0.4 * (m.A / g).abs().min().item())
        keep = m.params[i].clone()

        def at(k):
            m.params[i].copy_(keep).add_(g, alpha=k * h)
            return m.loss_and_grads(*args).item()
        got = (8 * (at(1) - at(-1)) - (at(2) - at(-2))) / (12 * h)
        m.params[i].copy_(keep)
        # noise of the loss itself: 2^-8 of logits of size one over 392 tokens, 2e-4, over a step of h
        assert abs(got - n2) <= 0.05 * n2 + 2e-4 / h, (i, got, n2)


def test_gradients_repeat_and_leave_the_rest():
    from adjoint_gradients_long_gb300.lm_train import SelLm
    m = SelLm(100, len(LENGTHS), 448, P=64)
    tokens, targets, offsets = batch(m, LENGTHS)
    m.loss_and_grads(tokens, targets, offsets)
    first = [g.clone() for g in m.grads]
    m.loss_and_grads(tokens, targets, offsets)
    assert all(torch.equal(g, f) for g, f in zip(m.grads, first))
    # the layer's own gradients do not see what stands behind the last document
    tokens[sum(LENGTHS):] = (tokens[sum(LENGTHS):] + 7) % m.V
    m.loss_and_grads(tokens, targets, offsets)
    assert all(torch.equal(m.grads[i], first[i]) for i in (4, 5, 6, 7, 8))


def test_trains_and_answers():
    """A packed prompt is each prompt alone, and the answers' steps are the prompt pass over one token more."""
    from adjoint_gradients_long_gb300.lm_train import SelLm
    m = SelLm(300, 5, 448, P=64)
    args = batch(m, LENGTHS)
    losses = [m.step(*args)[0].item() for _ in range(3)]
    assert all(x == x and x < 100 for x in losses)
    seqs = [args[0][:37], args[0][50:53], args[0][100:250]]
    offsets = torch.tensor([0, 37, 40, 190], device="cuda")
    logits, taps, state = (t.clone() for t in m.prompts(torch.cat(seqs), offsets))
    for i, s in enumerate(seqs):
        one = m.prompts(s, torch.tensor([0, len(s)], device="cuda"))
        assert torch.equal(one[1][0], taps[i])
        assert (one[2][0] - state[i]).norm() <= 1e-4 * state[i].norm()      # cut into other segments and tiles
        assert (one[0][0].float() - logits[i].float()).norm() <= 2.0 ** -6 * logits[i].float().norm()
    tokens, logps = m.answers(torch.cat(seqs), offsets, 6)
    for i, s in enumerate(seqs):
        for t in (0, 3, 5):
            so_far = torch.cat([s, tokens[i, :t]])
            again = m.prompts(so_far, torch.tensor([0, len(so_far)], device="cuda"))[0][0].float()
            # the likeliest token, or one whose logit is as large to the activations' rounding
            assert again.max() - again[tokens[i, t]] <= 0.05 * max(1.0, again.abs().max().item())
    assert (logps == 0).all()                                               # temperature zero: nothing else to draw
    drawn, lp = m.answers(torch.cat(seqs), offsets, 6, sampling=dict(temperature=0.9, top_k=40, top_p=0.9, min_p=0.01), seed=3)
    again, _ = m.answers(torch.cat(seqs), offsets, 6, sampling=dict(temperature=0.9, top_k=40, top_p=0.9, min_p=0.01), seed=3)
    assert torch.equal(drawn, again) and ((drawn >= 0) & (drawn < 300)).all() and (lp <= 0).all() and (lp > -4).all()


def test_linear_attention_model_draws():
    from adjoint_gradients_long_gb300.lm_train import TinyLm
    m = TinyLm(200, 1, 64, H=2, D=64)
    seq = torch.arange(50, device="cuda")
    greedy = m.answer(seq, 5)
    zero = m.answer(seq, 5, sampling=dict(temperature=0.0))
    assert [t for t, _, _ in greedy] == [t for t, _, _ in zero] and all(lp == 0 for _, lp, _ in zero)
    drawn = m.answer(seq, 5, sampling=dict(top_k=3), seed=1)
    assert all(t in [b for b, _ in best[:3]] for t, _, best in drawn)
