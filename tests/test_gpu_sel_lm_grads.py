"""The selective language model's loss and all nine gradients against the same model in 64 bits with torch's
autograd on the host, document by document.

The model there rounds its activations to bf16 where SelLm does (forwards only: the rounding's derivative is taken
as one), so forwards the two differ by fp32 rounding.  Backwards SelLm rounds five times at most between the loss
and a parameter (the logits' gradient, the scan's cotangent, its gradients, the convolution's cotangent, its
gradient), each by 2^-8 of a value at most.  A gradient is a sum over tokens and channels whose terms have either
sign, and so have their roundings, so the sum's relative error is not above the terms': 5 x 2^-8.
The loss: fp32 sums of 2^-24 each over rows of 200 logits, and now and then a logit that rounds the other way: 1e-4."""
import pytest

torch = pytest.importorskip("torch")

from conftest import rel_fro  # noqa: E402

pytestmark = pytest.mark.gpu

NAMES = ("E", "W_in", "W_x", "W_o", "w", "b", "A", "D", "dt_bias")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


def bf16(x):
    return x + (x.detach().bfloat16().double() - x.detach())


def silu(x):
    return x / (1 + torch.exp(-x))


def restated(params, tokens, targets, offsets, N, W):
    """The loss over documents, differentiable in params."""
    E, W_in, W_x, W_o, w, b, A, D, dt_bias = params
    P = E.shape[1]
    nll = []
    for t0, t1 in zip(offsets[:-1], offsets[1:]):
        if t0 == t1:
            continue
        x = E[tokens[t0:t1]]
        uz = bf16(x @ W_in)
        u, z = uz[:, :P], uz[:, P:]
        u = torch.cat([u.new_zeros(W - 1, P), u])
        c = bf16(silu(b + sum(w[:, j] * u[j:j + t1 - t0] for j in range(W))))
        h = bf16(c @ W_x)
        d = torch.nn.functional.softplus(h[:, :P] + dt_bias, threshold=1e9)
        Bm, Cm = h[:, P:P + N], h[:, P + N:]
        state, v = x.new_zeros(P, N), []
        for t in range(t1 - t0):
            state = torch.exp(d[t, :, None] * A) * state + (d[t] * c[t])[:, None] * Bm[t]
            v.append((state * Cm[t]).sum(-1) + D * c[t])
        s = bf16(torch.stack(v) * silu(z))
        logits = bf16((x + s @ W_o) @ E.T)
        nll.append(torch.logsumexp(logits, -1) - logits.gather(1, targets[t0:t1, None])[:, 0])
    return torch.cat(nll).mean()


@pytest.mark.parametrize("steps", ["first", "large"])
@pytest.mark.parametrize("lengths,before", [([130, 0, 61, 200, 1], 0), ([3, 90, 0, 0, 155], 21)])
def test_loss_and_gradients(lengths, before, steps):
    from adjoint_gradients_long_gb300.lm_train import SelLm
    T, V = 448, 200
    m = SelLm(V, len(lengths), T, P=64)
    if steps == "large":
        m.dt_bias.zero_()                                   # of about 0.7: states that forget within the documents
    gen = torch.Generator().manual_seed(7)
    n = sum(lengths)
    tokens = torch.randint(0, V, (T,), generator=gen)
    targets = torch.full((T,), -1, dtype=torch.int64)
    targets[before:before + n] = torch.randint(0, V, (n,), generator=gen)
    offsets = torch.tensor([before, *lengths]).cumsum(0)
    params = [p.detach().double().cpu().requires_grad_(True) for p in m.params]
    want = restated(params, tokens, targets, offsets.tolist(), m.N, m.W)
    want.backward()
    loss = m.loss_and_grads(tokens.cuda(), targets.cuda(), offsets.cuda())
    assert abs(loss.item() - want.item()) <= 1e-4
    errs = {name: rel_fro(g.double().cpu().numpy(), p.grad.numpy()) for name, g, p in zip(NAMES, m.grads, params)}
    print(" ".join(f"{k}={e:.1e}" for k, e in errs.items()))
    assert all(e <= 5 * 2.0 ** -8 for e in errs.values()), errs
