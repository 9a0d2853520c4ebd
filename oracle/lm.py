"""The language-model operators in fp64, step by step from their definitions (test
infrastructure; shares nothing with the library).

lin_forward, lin_backward   the recurrence S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale q_t S_t
                            token by token, and its reverse
logprob, logprob_grad       log probabilities, entropy, top list and the gradient, row by row
grad_clip                   the global norm and the clipped tensors
"""
import numpy as np


def _heads(x, H):
    """[B,T,Hk,D] -> [B,T,H,D]: head h reads q and k of head h // (H // Hk)."""
    return np.repeat(x, H // x.shape[2], axis=2)


def lin_states(k, v, g, s0=None):
    """States [T+1, B, H, Dk, Dv]: before the first token and after each one."""
    B, T, H, Dv = v.shape
    k = _heads(np.asarray(k), H)
    S = np.zeros((T + 1, B, H, k.shape[3], Dv), dtype=np.result_type(k, v, g, *(() if s0 is None else (s0,)), np.float64))
    if s0 is not None:
        S[0] = s0
    for t in range(T):
        S[t + 1] = np.exp(g[:, t])[..., None, None] * S[t] + k[:, t, :, :, None] * v[:, t, :, None, :]
    return S


def lin_forward(q, k, v, g, scale, s0=None):
    S = lin_states(k, v, g, s0)
    o = scale * np.einsum("bthd,tbhde->bthe", _heads(np.asarray(q), v.shape[2]), S[1:])
    return o, S[-1]


def lin_backward(q, k, v, g, scale, go, s0=None, ds1=None):
    """dq, dk (summed over a group's heads), dv, dg, ds0."""
    B, T, H, Dv = v.shape
    Hk, Dk = q.shape[2:]
    S, qh, kh = lin_states(k, v, g, s0), _heads(q, H), _heads(k, H)
    Z = np.zeros((B, H, Dk, Dv)) if ds1 is None else np.array(ds1, np.float64)
    dq, dk, dv, dg = np.zeros((B, T, H, Dk)), np.zeros((B, T, H, Dk)), np.zeros((B, T, H, Dv)), np.zeros((B, T, H))
    for t in reversed(range(T)):
        w = scale * go[:, t]
        dq[:, t] = np.einsum("bhde,bhe->bhd", S[t + 1], w)
        Z = Z + qh[:, t, :, :, None] * w[:, :, None, :]
        dk[:, t] = np.einsum("bhde,bhe->bhd", Z, v[:, t])
        dv[:, t] = np.einsum("bhde,bhd->bhe", Z, kh[:, t])
        a = np.exp(g[:, t])
        dg[:, t] = a * np.einsum("bhde,bhde->bh", Z, S[t])
        Z = a[..., None, None] * Z
    share = lambda x: x.reshape(B, T, Hk, H // Hk, Dk).sum(3)  # noqa: E731
    return share(dq), share(dk), dv, dg, Z


def logprob(x, y, top=0):
    """(logp, entropy, lse, top_id, top_logp) of rows x [N,V] for targets y [N]."""
    N, V = x.shape
    x = np.asarray(x, np.float64)
    logp, ent, lse = np.zeros(N), np.zeros(N), np.zeros(N)
    ids, tops = np.zeros((N, top), np.int32), np.zeros((N, top))
    for n in range(N):
        m = x[n].max()
        if m == -np.inf:
            lse[n], lp = -np.inf, np.full(V, -np.inf)
        else:
            with np.errstate(invalid="ignore"):
                z = np.log(np.exp(x[n] - m).sum())
                lse[n] = m + z
                lp = x[n] - m - z
                p = np.exp(lp)
                ent[n] = -np.sum(p[~(p == 0)] * lp[~(p == 0)])
        if 0 <= y[n] < V:
            logp[n] = lp[y[n]]
        # NaN first, then descending, equal values by index
        order = np.lexsort((np.arange(V), -x[n], ~np.isnan(x[n])))[:top]
        ids[n], tops[n] = order, lp[order]
    return logp, ent, lse, ids, tops


def logprob_grad(x, y, glp, gent):
    """dlogits for the cotangents of logp and entropy."""
    N, V = x.shape
    x = np.asarray(x, np.float64)
    _, ent, lse, _, _ = logprob(x, y)
    d = np.zeros((N, V))
    for n in range(N):
        if lse[n] == -np.inf:
            continue
        lp = x[n] - x[n].max()
        lp = lp - np.log(np.exp(lp).sum())
        p = np.exp(lp)
        d[n] = -gent[n] * np.where(p > 0, p * (np.where(p > 0, lp, 0.0) + ent[n]), 0.0)
        if 0 <= y[n] < V:
            d[n] -= glp[n] * p
            d[n, y[n]] += glp[n]
    return d


def grad_clip(tensors, max_norm, eps=1e-6):
    norm = np.sqrt(sum(float(np.sum(np.asarray(t, np.float64) ** 2)) for t in tensors))
    coef = min(1.0, max_norm / (norm + eps))
    return norm, coef, [np.asarray(t, np.float64) * coef for t in tensors]
