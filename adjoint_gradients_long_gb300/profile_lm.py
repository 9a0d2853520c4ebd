"""Run one language-model operator a few times: the command that the ncu captures of these
kernels under profiles/ are taken with.

  python -m adjoint_gradients_long_gb300.profile_lm fwd|bwd|step|score|loss|clip|conv|conv_bwd|scan|scan_bwd|scan_step|sample
      [--runs N]

fwd, bwd   linear attention, 2 rows of 16384 tokens (bwd: 4096), 16 heads of 128, bf16
fwd32      the same in fp32, 2 rows of 2048 tokens, 8 heads of 128
step       256 sequences, 16 heads of 128
score      log probabilities and 5 alternatives, 912 rows of 50001 fp32 logits
loss       log probabilities and gradient, 2736 rows of 32768 bf16 logits
clip       120 tensors of 733333 bf16 values
conv       short convolution, 32768 tokens of 24 packed sequences, 2048 channels, 4 taps, bf16
conv_bwd   its gradients, 8 rows of 2048 tokens
scan       selective scan with gate, 16384 tokens, 1024 channels of 16 states, bf16
scan_bwd   its gradients, 4096 tokens, 2048 channels
scan_step  256 sequences, 2048 channels of 16 states
sample     top-p 0.9, 152 rows of 50001 fp32 logits
"""
from __future__ import annotations

import argparse

import torch

from . import build, lm


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("op", choices=("fwd", "bwd", "fwd32", "step", "score", "loss", "clip", "conv", "conv_bwd", "scan", "scan_bwd",
                                    "scan_step", "sample"))
    ap.add_argument("--runs", type=int, default=2)
    a = ap.parse_args(argv)
    build.build()
    gen = torch.Generator(device="cuda").manual_seed(0)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    if a.op in ("fwd", "bwd", "fwd32"):
        bf = a.op != "fwd32"
        B, T, H, D = 2, {"fwd": 16384, "bwd": 4096, "fwd32": 2048}[a.op], 16 if bf else 8, 128
        c = (lambda x: x.bfloat16()) if bf else (lambda x: x)
        q, k, v, go = c(n(B, T, H, D)), c(n(B, T, H, D) / D ** 0.5), c(n(B, T, H, D)), c(n(B, T, H, D))
        g = torch.nn.functional.logsigmoid(n(B, T, H) + 3)
        att = lm.LinAttn(B, T, H, D, D, x_bf16=bf, scale=D ** -0.5, backward=a.op == "bwd")
        run = (lambda: att.backward(q, k, v, g, go)) if a.op == "bwd" else (lambda: att.forward(q, k, v, g))
    elif a.op == "step":
        B, H, D = 256, 16, 128
        q, g, state = n(B, H, D).bfloat16(), -0.1 * torch.ones(B, H, device="cuda"), n(B, H, D, D)
        st = lm.LinStep(B, H, D, D)
        run = lambda: st.step(q, q, q, g, state)  # noqa: E731
    elif a.op in ("score", "loss"):
        N, V, bf = (912, 50001, False) if a.op == "score" else (2736, 32768, True)
        x = 2 * n(N, V)
        x = x.bfloat16() if bf else x
        y = torch.randint(0, V, (N,), device="cuda", generator=gen)
        p = lm.TokenLogProbs(N, V, x_bf16=bf, top=0 if bf else 5)
        glp = torch.full((N,), -1.0 / N, device="cuda")
        run = (lambda: p.gradient(x, y, glp, glp)) if a.op == "loss" else (lambda: p.forward(x, y))
    elif a.op in ("conv", "conv_bwd"):
        packed = a.op == "conv"
        P, T, B = 2048, 32768 if packed else 2048, 24 if packed else 8
        c = lm.ShortConv(B, T, P, packed=packed, backward=not packed)
        x, go = (n(*c.x).bfloat16() for _ in range(2))
        w, b = n(P, 4) / 2, n(P)
        off = torch.linspace(0, T, B + 1, device="cuda").long() if packed else None
        run = (lambda: c.forward(x, w, b, None, off)) if packed else (lambda: c.backward(x, w, go, b))
    elif a.op in ("scan", "scan_bwd", "scan_step"):
        B, T, P, N = {"scan": (1, 16384, 1024, 16), "scan_bwd": (1, 4096, 2048, 16), "scan_step": (256, 1, 2048, 16)}[a.op]
        lead = (B,) if a.op == "scan_step" else (B, T)
        x, dt, z, go = (n(*lead, P).bfloat16() for _ in range(4))
        Bm, Cm = (n(*lead, N).bfloat16() for _ in range(2))
        A, D, b = -(torch.arange(N, device="cuda") + 1.0).repeat(P, 1), torch.ones(P, device="cuda"), torch.full((P,), -4.0, device="cuda")
        if a.op == "scan_step":
            st, state = lm.SelScanStep(B, P, N), n(300, P, N)
            slots = torch.randperm(300, device="cuda", generator=gen)[:B].int()
            run = lambda: st.step(x, dt, A, Bm, Cm, state, D, z, b, slots)  # noqa: E731
        else:
            s = lm.SelScan(B, T, P, N, backward=a.op == "scan_bwd")
            run = (lambda: s.backward(x, dt, A, Bm, Cm, go, D, z, b)) if a.op == "scan_bwd" else (lambda: s.forward(x, dt, A, Bm, Cm, D, z, b))
    elif a.op == "sample":
        N, V = 152, 50001
        x, u = 2 * n(N, V), torch.rand(N, device="cuda", generator=gen)
        s, top_p = lm.Sampler(N, V, x_bf16=False), torch.full((N,), 0.9, device="cuda")
        run = lambda: s.sample(x, u, None, None, top_p)  # noqa: E731
    else:
        gs = [n(733333).bfloat16() for _ in range(120)]
        c = lm.GradClip(gs, [torch.empty_like(t) for t in gs])
        run = lambda: c.clip(1.0)  # noqa: E731
    for _ in range(a.runs):
        run()
    torch.cuda.synchronize()
    print(f"{a.op}: {a.runs} runs")


if __name__ == "__main__":
    main()
