"""The sampler's weights, round(2^40 e^((x - m) / T)) as whole numbers from pairs of fp32, off by one unit at most: the
arithmetic of csrc/adj_sample.cu (Weigh) restated operation by operation and compared with extended precision."""
import numpy as np
import pytest

f, X = np.float32, np.longdouble
pytestmark = pytest.mark.skipif(np.finfo(X).nmant < 63, reason="needs an extended floating-point type")


def fma(a, b, c):
    """Rounded to 24 bits once but for ties of the extended type's own rounding."""
    return (np.asarray(a).astype(X) * np.asarray(b).astype(X) + np.asarray(c).astype(X)).astype(f)


def quotient(T):
    """log2 e / T as a pair of fp32."""
    H, L = f(1.44269502162933349609375), f(1.925963033500011079e-8)
    hi = f(H / T)
    return hi, f(f(fma(-hi, T, H) + L) / T)


def weights(m, x, T):
    hi, lo = quotient(T)
    steps = X(2) ** (-(np.arange(256) + 1) / X(256))
    s_hi = steps.astype(f)
    s_lo = (steps - s_hi.astype(X)).astype(f)
    magic = f(12582912)
    d = m - x
    t = d * hi
    b = d - m
    dl = (m - (d - b)) - (x + b)
    e = fma(d, hi, -t) + fma(d, lo, dl * hi)
    kf = fma(t, f(256), magic - f(1))
    kb = kf.view(np.uint32)
    r = fma(kf - (magic - f(1)), f(-1 / 256), t)
    L, LL = f(0.693147182464599609375), f(-1.904654323148236017e-9)
    ph = -r * L
    pl = fma(-r, L, -ph)
    rest = fma(-e, L, fma(-r, LL, pl))
    tail = fma(ph, fma(ph, fma(ph, f(1 / 6), f(0.5)), rest), rest)
    sx, sy = s_hi[kb & 255], s_lo[kb & 255]
    q = sx * ph
    low = fma(sx, ph, -q) + fma(sy, ph, fma(sx, tail, sy))
    total = q + low
    lost = low - (total - q)
    qa = fma(total, f(1048576), magic)
    qb = fma(fma(qa - magic, f(-1 / 1048576), total) + lost, f(2.0 ** 42), magic)
    u64, bits = np.uint64, 0x4B400000
    upper = ((sx.view(np.uint32) & 0x7FFFFF) | 0x800000).astype(u64) + (qa.view(np.uint32).astype(u64) << u64(4))
    upper = (upper - u64(bits << 4) - u64(bits >> 18)) & u64(0xFFFFFFFF)
    whole = (upper << u64(18)) + qb.view(np.uint32).astype(u64)
    w = ((whole >> (((kb >> 8) + 1) & 63).astype(u64)) + u64(1)) >> u64(1)
    return np.where(t < f(41.5), w, u64(0))


@pytest.mark.parametrize("T", [0.05, 0.8, 1.0, 1.7, 30.0])
def test_within_a_unit(T):
    r, T, m = np.random.default_rng(0), f(T), f(9.37)
    x = (m - np.abs(r.normal(size=200000) * 6 * float(T))).astype(f)
    x[:3] = m
    x[3:1000] = m - (np.arange(997) * 1e-5).astype(f)
    w = weights(m, x, T)
    exact = np.exp(-(X(m) - x.astype(X)) / X(T)) * X(2) ** 40
    err = np.abs(w.astype(X) - exact).max()
    assert (w[:3] == 1 << 40).all() and err <= 1, err
    assert err <= 0.76                                      # half a unit of the last rounding, and a quarter before it
