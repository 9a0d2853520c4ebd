"""The short convolution, the selective scan with states and sampling in fp64, step by step from
their definitions (test infrastructure; shares nothing with the library).

Sequences are given as a list of (begin, end) over rows of tokens; arrays are [rows, ...].
"""
import math

import numpy as np


def sequences(B, T, offsets=None):
    """(begin, end) of each of B sequences: of T tokens each, or between the offsets."""
    if offsets is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    o = [int(x) for x in offsets]
    return list(zip(o[:-1], o[1:]))


def _kind(*xs):
    return np.result_type(np.float64, *(x for x in xs if x is not None))


def conv_forward(x, w, bias, s0, seqs, act=True):
    """y [rows,P] (zeros outside the sequences), s1 [B,W-1,P]."""
    P, W = w.shape
    k = _kind(x, w, bias, s0)
    y, s1 = np.zeros(x.shape, k), np.zeros((len(seqs), W - 1, P), k)
    for b, (t0, t1) in enumerate(seqs):
        c = np.concatenate([np.zeros((W - 1, P)) if s0 is None else s0[b], x[t0:t1]])
        for t in range(t1 - t0):
            p = sum(w[:, j] * c[t + j] for j in range(W)) + (0 if bias is None else bias)
            y[t0 + t] = p / (1 + np.exp(-p)) if act else p
        s1[b] = c[t1 - t0:]
    return y, s1


def conv_backward(x, w, bias, s0, seqs, go, ds1=None, act=True):
    """dx, dw, dbias, ds0."""
    P, W = w.shape
    dx, dw, db, ds0 = np.zeros(x.shape), np.zeros((P, W)), np.zeros(P), np.zeros((len(seqs), W - 1, P))
    for b, (t0, t1) in enumerate(seqs):
        n = t1 - t0
        c = np.concatenate([np.zeros((W - 1, P)) if s0 is None else s0[b], x[t0:t1]])
        dc = np.zeros_like(c)
        if ds1 is not None:
            dc[n:] += ds1[b]
        for t in range(n):
            dp = go[t0 + t]
            if act:
                p = sum(w[:, j] * c[t + j] for j in range(W)) + (0 if bias is None else bias)
                s = 1 / (1 + np.exp(-p))
                dp = dp * s * (1 + p * (1 - s))
            db += dp
            for j in range(W):
                dc[t + j] += w[:, j] * dp
                dw[:, j] += c[t + j] * dp
        dx[t0:t1], ds0[b] = dc[W - 1:], dc[:W - 1]
    return dx, dw, db, ds0


def softplus(v):
    return np.where(v.real > 0, v, 0) + np.log1p(np.exp(np.where(v.real > 0, -v, v)))


def scan_forward(x, dt, A, Bm, Cm, D, z, bias, s0, seqs):
    """y [rows,P], s1 [B,P,N], and what the gradients use: v [rows,P], states before and after every token."""
    (P, N), rows = A.shape, x.shape[0]
    k = _kind(x, dt, A, Bm, Cm, D, z, bias, s0)
    d = softplus(dt + (0 if bias is None else bias))
    v, y, s1 = np.zeros((rows, P), k), np.zeros((rows, P), k), np.zeros((len(seqs), P, N), k)
    before, after = np.zeros((rows, P, N), k), np.zeros((rows, P, N), k)
    for b, (t0, t1) in enumerate(seqs):
        h = np.zeros((P, N), k) if s0 is None else s0[b].astype(k)
        for t in range(t0, t1):
            before[t] = h
            h = np.exp(d[t][:, None] * A) * h + (d[t] * x[t])[:, None] * Bm[t]
            after[t] = h
            v[t] = h @ Cm[t] + (0 if D is None else D * x[t])
            y[t] = v[t] if z is None else v[t] * z[t] / (1 + np.exp(-z[t]))
        s1[b] = h
    return y, s1, (v, before, after)


def scan_backward(x, dt, A, Bm, Cm, D, z, bias, s0, seqs, go, ds1=None):
    """dx, ddt, dA, dB, dC, dD, dz, dbias, ds0."""
    P, N = A.shape
    raw = dt + (0 if bias is None else bias)
    d, sig = softplus(raw), 1 / (1 + np.exp(-raw))
    v, before, after = scan_forward(x, dt, A, Bm, Cm, D, z, bias, s0, seqs)[2]
    dx, ddt, dz = np.zeros(x.shape), np.zeros(x.shape), np.zeros(x.shape)
    dB, dC, dA, dD, ds0 = np.zeros(Bm.shape), np.zeros(Cm.shape), np.zeros((P, N)), np.zeros(P), np.zeros((len(seqs), P, N))
    for b, (t0, t1) in enumerate(seqs):
        e = np.zeros((P, N)) if ds1 is None else np.array(ds1[b], np.float64)
        for t in reversed(range(t0, t1)):
            g = go[t]
            if z is not None:
                s = 1 / (1 + np.exp(-z[t]))
                dz[t] = g * v[t] * s * (1 + z[t] * (1 - s))
                g = g * z[t] * s
            m = g[:, None] * Cm[t] + e
            dC[t], dB[t] = g @ after[t], (d[t] * x[t]) @ m
            mB = m @ Bm[t]
            e = np.exp(d[t][:, None] * A) * m
            q = e * before[t]
            dA += q * d[t][:, None]
            dx[t] = d[t] * mB + (0 if D is None else D * g)
            dD += g * x[t]
            ddt[t] = (x[t] * mB + (q * A).sum(-1)) * sig[t]
        ds0[b] = e
    return dx, ddt, dA, dB, dC, dD, dz, ddt.sum(0), ds0


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logp) of one row."""
    x = np.asarray(x, np.float64)
    if not temperature >= 0 or math.isnan(top_p) or math.isnan(min_p) or np.isnan(x).any() or (x == np.inf).any():
        return -1, math.nan
    m = x.max()
    if m == -np.inf:
        return -1, -math.inf
    order = np.lexsort((np.arange(len(x)), -x))
    far = np.where(x == -np.inf, -np.inf, (x - m) / temperature if temperature else np.where(x == m, 0.0, -np.inf))
    w = [int(v) for v in np.rint(np.exp(far) * 2.0 ** 40)]
    kept = [i for i in order if w[i] >= max(1, min(min_p, 1.0) * 2.0 ** 40)]
    if top_k > 0:
        kept = kept[:top_k]
    if temperature == 0:
        kept = kept[:1]
    total, run, n = sum(w[i] for i in kept), 0, len(kept)
    if top_p < 1:
        for n, i in enumerate(kept, 1):
            run += w[i]
            if run >= top_p * total:
                break
    kept = sorted(kept[:n])
    total = sum(w[i] for i in kept)
    u = 0.0 if math.isnan(u) else min(max(float(u), 0.0), 1 - 2.0 ** -24)
    run = 0
    for i in kept:
        run += w[i]
        if run > u * total:
            return int(i), float(far[i]) - math.log(total / 2.0 ** 40)
