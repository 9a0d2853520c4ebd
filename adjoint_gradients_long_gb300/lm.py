"""Operators of a language model built of recurrent layers, through libadj.so.

LinAttn, LinStep    linear attention with a decay for each head: chunked for prompts and
                    training (with gradients), recurrent for single tokens
TokenLogProbs       log probabilities of given tokens, entropy, top alternatives, gradient
GradClip            clipping gradients by their global norm

include/adj.h states each operator in full.  As the drivers of the layers do, an object holds
the sizes, the workspace and the outputs of one shape: a call overwrites the outputs of the
call before it, enqueues kernels on torch's current stream and synchronises nothing, and can
be captured into a CUDA graph.  Calls on one object belong to one stream at a time (they share
its buffers).  An object's device has to be the current one during a call.  Tensors are checked for
shape, type, device and layout (ValueError) before the library checks its own arguments
(lib.AdjError).
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

import torch

from . import lib
from .lib import raw_stream

LogProbs = namedtuple("LogProbs", "logp entropy lse top_id top_logp dlogits")


def _check(name, x, shape, dtype, device):
    if x.dtype is not dtype or x.shape != shape or x.device != device:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {device}, got {x.dtype} {tuple(x.shape)} on {x.device}")


def _dense(name, x, shape, dtype, device):
    """The address of a dense tensor."""
    _check(name, x, shape, dtype, device)
    if not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor, got strides {x.stride()}")
    return x.data_ptr()


def _device(device):
    """The device as tensors name it: CUDA ones with an index, any other without."""
    d = torch.device(device)
    if d.type != "cuda":
        return torch.device(d.type)
    return d if d.index is not None else torch.device("cuda", torch.cuda.current_device())


def _workspace(nbytes, device):
    ws = torch.empty((nbytes + 255) // 4, dtype=torch.int32, device=device)
    ws[:64].zero_()             # the header: status word and tickets
    return ws


class _Lin:
    """What LinAttn and LinStep share: sizes, and arrays [*lead, heads, width] whose heads lie
    densely in a token and whose tokens lie a common distance apart."""

    def __init__(self, lead, T, H, Dk, Dv, Hk, x_bf16, scale, device):
        Hk = H if Hk is None else Hk
        self.H, self.Hk, self.Dk, self.Dv = H, Hk, Dk, Dv
        self.device = _device(device)
        self.xt = torch.bfloat16 if x_bf16 else torch.float32
        self.lead = lead
        self.qk, self.vo, self.gates, self.states = (*lead, Hk, Dk), (*lead, H, Dv), (*lead, H), (lead[0], H, Dk, Dv)
        self.dims = lib.lin_dims(lead[0], T, H, Hk, Dk, Dv, lib.BF16 if x_bf16 else lib.F32, scale)
        self._pd = ctypes.byref(self.dims)

    def _pitch(self, name, x, shape):
        """The distance of two tokens in x."""
        _check(name, x, shape, self.xt, self.device)
        least = shape[-2] * shape[-1]
        if x.is_contiguous():
            return least
        s = x.stride()
        ld = s[-3]
        if s[-1] != 1 or s[-2] != shape[-1] or ld < least or (len(shape) == 4 and shape[0] > 1 and s[0] != shape[1] * ld):
            raise ValueError(f"{name}: heads must lie densely in a token and tokens evenly, got strides {s}")
        return ld

    def _inputs(self, q, k, v, g):
        d = self.dims
        d.ldq, d.ldk, d.ldv = self._pitch("q", q, self.qk), self._pitch("k", k, self.qk), self._pitch("v", v, self.vo)
        return q.data_ptr(), k.data_ptr(), v.data_ptr(), _dense("g", g, self.gates, torch.float32, self.device)

    def _state(self, name, s):
        return None if s is None else _dense(name, s, self.states, torch.float32, self.device)

    def _empty(self, shape, dtype=None):
        return torch.empty(shape, dtype=dtype or self.xt, device=self.device)


class LinAttn(_Lin):
    """Linear attention over B rows of T tokens: S_t = e^{g_t} S_{t-1} + k_t v_t^T,
    o_t = scale q_t S_t, q and k [B,T,Hk,Dk] shared by groups of H / Hk heads, v [B,T,H,Dv],
    g [B,T,H] fp32 (at most 0; minus infinity starts a new document).  backward: also hold what
    the gradients need."""

    def __init__(self, B, T, H, Dk, Dv, Hk=None, x_bf16=True, scale=1.0, backward=False, device="cuda"):
        super().__init__((B, T), T, H, Dk, Dv, Hk, x_bf16, scale, device)
        need = lib.lin_workspace_bytes(self.dims, lib.OP_LIN_FWD)
        if backward:
            need = max(need, lib.lin_workspace_bytes(self.dims, lib.OP_LIN_BWD))
        if need == 0:
            raise ValueError("unsupported linear-attention sizes")
        self.ws_bytes = int(need)
        self.ws = _workspace(self.ws_bytes, self.device)
        self.o = self._empty(self.vo)
        self.s1 = self._empty((B, H, Dk, Dv), torch.float32)
        self.has_backward = backward
        self._fwd, self._bwd = lib.bind("adj_lin_fwd", self._pd), lib.bind("adj_lin_bwd", self._pd)
        self._out = self.o.data_ptr(), self.s1.data_ptr(), self.ws.data_ptr(), self.ws_bytes
        if backward:
            self.dq, self.dk, self.dv = self._empty(self.qk), self._empty(self.qk), self._empty(self.vo)
            self._strided = {("q", None): self.dq, ("k", None): self.dk, ("v", None): self.dv}
            self.dg = self._empty((B, T, H), torch.float32)
            self.ds0 = self._empty((B, H, Dk, Dv), torch.float32)

    def forward(self, q, k, v, g, s0=None):
        """(o [B,T,H,Dv], s1 [B,H,Dk,Dv]): the outputs and the state after the last token."""
        self._fwd(*self._inputs(q, k, v, g), self._state("s0", s0), *self._out, raw_stream(self.device))
        return self.o, self.s1

    def _like(self, name, x):
        """The gradient of x, in x's layout: one array for each layout that has been met, kept with
        the object, as a captured graph goes on writing to the one that it was captured with."""
        at = name, None if x.is_contiguous() else x.stride()
        if at not in self._strided:
            self._strided[at] = (torch.empty(x.shape, dtype=x.dtype, device=x.device) if at[1] is None
                                 else torch.empty_strided(x.shape, at[1], dtype=x.dtype, device=x.device))
        return self._strided[at]

    def backward(self, q, k, v, g, go, s0=None, ds1=None):
        """(dq, dk, dv, dg, ds0) for the cotangents go of o and ds1 of s1; dq, dk and dv have the
        layout of q, k and v."""
        if not self.has_backward:
            raise ValueError("this LinAttn was made without backward=True")
        at = self._inputs(q, k, v, g)
        at += self._state("s0", s0), _dense("go", go, self.vo, self.xt, self.device), self._state("ds1", ds1)
        self.dq, self.dk, self.dv = self._like("q", q), self._like("k", k), self._like("v", v)
        self._bwd(*at, self.dq.data_ptr(), self.dk.data_ptr(), self.dv.data_ptr(), self.dg.data_ptr(), self.ds0.data_ptr(),
                  *self._out[2:], raw_stream(self.device))
        return self.dq, self.dk, self.dv, self.dg, self.ds0

    def status(self, stream=None) -> int:
        return lib.stream_status(self.ws, stream)


class LinStep(_Lin):
    """The same recurrence for one token of each of B sequences: q, k [B,Hk,Dk], v [B,H,Dv],
    g [B,H] fp32, and a pool of states [n_slots,H,Dk,Dv] fp32 that is updated in place."""

    def __init__(self, B, H, Dk, Dv, Hk=None, x_bf16=True, scale=1.0, device="cuda"):
        super().__init__((B,), 1, H, Dk, Dv, Hk, x_bf16, scale, device)
        if lib.lin_workspace_bytes(self.dims, lib.OP_LIN_FWD) == 0:
            raise ValueError("unsupported linear-attention sizes")
        self.o = self._empty(self.vo)
        self._step, self._out = lib.bind("adj_lin_step", self._pd), self.o.data_ptr()

    def step(self, q, k, v, g, state, slots=None):
        """o [B,H,Dv].  slots [B] int32: sequence b's state is state[slots[b]] (a slot outside
        the pool: padding, a row of zeros); None: state[b]."""
        n = state.shape[0]
        pool = _dense("state", state, (n, self.H, self.Dk, self.Dv), torch.float32, self.device)
        if slots is not None:
            slots = _dense("slots", slots, self.lead, torch.int32, self.device)
        elif n < self.lead[0]:
            raise ValueError(f"state: {n} slots for {self.lead[0]} sequences")
        self._step(*self._inputs(q, k, v, g), pool, n, slots, self._out, raw_stream(self.device))
        return self.o


class TokenLogProbs:
    """Log probabilities of given tokens over logits [N,V] (rows may be strided): targets [N]
    int64 (outside [0,V): not scored), the row's entropy, its `top` best tokens, and the
    gradient of both for the logits."""

    def __init__(self, N, V, x_bf16=True, top=0, device="cuda"):
        self.N, self.V, self.top = N, V, top
        self.rows, self.shape = (N,), (N, V)
        self.device = _device(device)
        self.xt = torch.bfloat16 if x_bf16 else torch.float32
        self.dims = lib.logprob_dims(N, V, V, V, lib.BF16 if x_bf16 else lib.F32, top)
        if not (0 <= top <= min(V, lib.LOGPROB_MAX_TOP)):
            raise ValueError(f"top: 0 to {min(V, lib.LOGPROB_MAX_TOP)}, got {top}")
        f = lambda *s: torch.empty(*s, dtype=torch.float32, device=self.device)  # noqa: E731
        self.logp, self.entropy, self.lse = f(N), f(N), f(N)
        self.top_id = torch.empty(N, top, dtype=torch.int32, device=self.device) if top else None
        self.top_logp = f(N, top) if top else None
        self.dlogits = None
        self._logprob = lib.bind("adj_logprob", ctypes.byref(self.dims))
        self._out = tuple(None if x is None else x.data_ptr()
                          for x in (self.logp, self.entropy, self.lse, self.top_id, self.top_logp))
        self._plain = LogProbs(self.logp, self.entropy, self.lse, self.top_id, self.top_logp, None)

    def _row(self, name, x):
        _check(name, x, self.shape, self.xt, self.device)
        if x.is_contiguous():
            return self.V
        if x.stride(1) != 1 and self.V > 1:
            raise ValueError(f"{name}: rows must be contiguous, got strides {x.stride()}")
        if self.N > 1 and x.stride(0) < self.V:
            raise ValueError(f"{name}: rows must not overlap, got strides {x.stride()}")
        return x.stride(0) if self.N > 1 else self.V

    def forward(self, logits, targets):
        """LogProbs without a gradient."""
        self.dims.ld = self._row("logits", logits)
        y = _dense("targets", targets, self.rows, torch.int64, self.device)
        self._logprob(logits.data_ptr(), y, *self._out, None, None, None, raw_stream(self.device))
        return self._plain

    def gradient(self, logits, targets, glp, gent=None, dlogits=None):
        """LogProbs with dlogits for the cotangents glp of logp and gent of the entropy, [N] fp32.
        dlogits: the array to write, which may be the logits themselves; None: one of this
        object's."""
        self.dims.ld = self._row("logits", logits)
        y = _dense("targets", targets, self.rows, torch.int64, self.device)
        cot = (_dense("glp", glp, self.rows, torch.float32, self.device),
               None if gent is None else _dense("gent", gent, self.rows, torch.float32, self.device))
        if dlogits is None:
            if self.dlogits is None:
                self.dlogits = torch.empty(self.N, self.V, dtype=self.xt, device=self.device)
            dlogits = self.dlogits
        self.dims.ldd = self._row("dlogits", dlogits)
        self._logprob(logits.data_ptr(), y, *self._out, *cot, dlogits.data_ptr(), raw_stream(self.device))
        return self._plain._replace(dlogits=dlogits)


class GradClip:
    """Clipping a fixed list of gradient tensors (fp32 or bf16, contiguous) by their global norm:
    outs[i] = min(1, max_norm / (norm + 1e-6)) grads[i]; outs None clips in place.  The object keeps
    these tensors and clips them at every call: a program that frees its gradients and makes
    others needs another object for those."""

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.outs) != len(self.grads):
            raise ValueError(f"{len(self.outs)} outputs for {len(self.grads)} gradients")
        self.device = _device(self.grads[0].device if self.grads else "cuda")
        kinds = {torch.float32: lib.F32, torch.bfloat16: lib.BF16}
        self.segs = (lib.GradSeg * max(1, len(self.grads)))()
        for i, (x, y) in enumerate(zip(self.grads, self.outs)):
            if x.dtype not in kinds:
                raise ValueError(f"gradient {i}: fp32 or bf16, got {x.dtype}")
            _dense(f"gradient {i}", x, tuple(x.shape), x.dtype, self.device)
            _dense(f"output {i}", y, tuple(x.shape), x.dtype, self.device)
            self.segs[i] = lib.GradSeg(x.data_ptr(), y.data_ptr(), x.numel(), kinds[x.dtype], 0)
        self.ws_bytes = lib.clip_workspace_bytes()
        self.ws = _workspace(self.ws_bytes, self.device)
        self.result = torch.empty(2, dtype=torch.float32, device=self.device)
        self.norm, self.coef = self.result[0], self.result[1]
        self._clip = lib.bind("adj_grad_clip", self.segs, len(self.grads))
        self._out = self.result.data_ptr(), self.ws.data_ptr(), self.ws_bytes

    def clip(self, max_norm):
        """(norm, coefficient) as device scalars; the outputs hold the clipped gradients."""
        self._clip(max_norm, *self._out, raw_stream(self.device))
        return self.norm, self.coef

    def status(self, stream=None) -> int:
        """Waits for `stream`: 0, or the status (lib.STATUS) of a call whose blocks did not meet in
        time.  Such a call leaves (NaN, NaN) and what it has not scaled as it was; the object is
        ready for the next call afterwards."""
        st = lib.stream_status(self.ws, stream)
        if st:
            self.ws[:64].zero_()
        return st
