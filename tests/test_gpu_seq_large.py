"""The largest forms of the selective scan and of the sampler: channels that fill the machine with one segment of all
tokens, and the longest rows."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_sample import check  # noqa: E402
from test_gpu_seq import scan_check  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from adjoint_gradients_long_gb300 import build
    build.build()


@pytest.mark.parametrize("bf16,kw", [(True, dict(B=1, T=130)), (False, dict(B=3, T=130, lengths=[50, 0, 71], before=5))])
def test_scan_one_segment_of_many_channels(bf16, kw):
    """15000 channels of 64 states are 469 blocks of four warps, more than fit the machine at a time, and 1875
    warps, too many for the short prompts' form: the tokens (nine tiles) stay in one segment, forwards by the
    output pass alone."""
    scan_check(21, P=15000, N=64, bf16=bf16, **kw)


V = 393216


@pytest.mark.parametrize("bf16", [False, True])
def test_sampler_longest_rows(bf16):
    """A row fills eight blocks (fp32), or four where there are many rows (bf16), and begins anywhere."""
    from adjoint_gradients_long_gb300 import lib
    assert V == lib.SAMPLE_MAX_V
    g = torch.Generator().manual_seed(3)
    xt = torch.bfloat16 if bf16 else torch.float32
    for N, at in ((2, 0), (2, 1), (20, 5)):
        wide = (torch.randn(N, V + 9, generator=g) * 2).to(xt).cuda()
        x, u = wide[:, at:at + V], torch.rand(N, generator=g).tolist()
        r = np.random.default_rng(at)
        pick = lambda *v: [v[i] for i in r.integers(0, len(v), N)]  # noqa: E731
        check(x, u, top_k=pick(50, 1000, 300000), top_p=pick(0.9, 0.999))
        if N == 2:
            check(x, u)
            check(x, u, temperature=pick(0.7, 1.3), min_p=pick(0.01, 0.0), top_k=pick(7, 0))
            check(x, u, top_p=[0.5, 0.99])


@pytest.mark.parametrize("bf16", [False, True])
def test_sampler_longest_rows_of_equal_values(bf16):
    """The total of the weights passes 2^58; limits and draws fall at whole tokens."""
    x = torch.zeros(3, V, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    x[1, V // 2:] = -math.inf
    x[2, -1] = 1.0
    for u in ([0.0] * 3, [0.5] * 3, [0.75] * 3, [1 - 2.0 ** -24] * 3):
        check(x, u)
        check(x, u, top_k=[V - 1, V // 4, V // 2])
        check(x, u, top_p=[0.5, 0.25, 0.75])
