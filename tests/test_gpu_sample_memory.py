"""Sampling does not depend on what a kernel before left in shared memory."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


WORDS = [0, 1, 0x7FFFFFFF, -0x80000000, -1, 0x3FFFFFFF, 0x7F800001]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [5000, 20000, 40000, 131072])     # 1, 4, 8 and 8 blocks a row
def test_whatever_shared_memory_holds(bf16, V):
    """A row of 160 KB on every SM leaves one word all over its shared memory; then limits one token short of all
    of a row of equal values, and of two values: the last tokens, by index, are the ones left out."""
    from adjoint_gradients_long_gb300 import lm
    fill = lm.Sampler(608, 40000, x_bf16=False)
    words = torch.empty(608, 40000, dtype=torch.int32, device="cuda")
    fu = torch.zeros(608, device="cuda")
    s = lm.Sampler(1, V, x_bf16=bf16)
    x = torch.zeros(2, 1, V, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    x[1, 0, :V // 2] = 1.0
    u = torch.full((1,), 1 - 2.0 ** -24, device="cuda")     # the last kept token, by index
    for word in WORDS:
        words.fill_(word)
        for row in range(2):
            for short in (1, 2, 3):
                k = torch.full((1,), V - short, dtype=torch.int32, device="cuda")
                fill.sample(words.view(torch.float32), fu)
                token, _ = s.sample(x[row], u, top_k=k)
                assert token.item() == V - short - 1, (word, row, short)
