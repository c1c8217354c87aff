"""The expert-layer operators together, as a model uses them: a sparse expert
layer whose weights are held in block-scaled FP8, for a decode step and a
prefill, and a dense layer's training step in the same format.

    python examples/expert_layer.py

Each result is compared with the same computation on the unquantised weights in
64 bits; what differs is the rounding to FP8 (a few percent).  The timed calls
are whole passes through the operators, on the device's clock.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_tensor_core_gemm_gb300 as tg  # noqa: E402


class ExpertLayer:
    """y_t = sum_j w_tj W2_e gelu(W1_e x_t) over the top_k experts e of token t."""

    def __init__(self, w1, w2, router, bias, top_k, groups=1, top_groups=1):
        # w1: (E, F, H), w2: (E, H, F), router: (H, E); quantised once
        self.router = router.to(torch.bfloat16)
        self.bias, self.top_k, self.groups, self.top_groups = bias, top_k, groups, top_groups
        q, s = tg.quantize_block(w1, "tile")
        self.w1, self.s1 = q.transpose(1, 2), s.transpose(1, 2)
        q, s = tg.quantize_block(w2, "tile")
        self.w2, self.s2 = q.transpose(1, 2), s.transpose(1, 2)

    def route(self, x):
        logits = tg.gemm(x, self.router)
        return tg.route(logits, self.top_k, score="sigmoid", bias=self.bias, groups=self.groups,
                        top_groups=self.top_groups, group_score="top2")

    def __call__(self, x):
        r = self.route(x)
        q, s = tg.quantize_block(x, "row", scatter=r.slots)              # to the experts' rows
        h = tg.gemm_experts(q, s, self.w1, self.s1, r.offsets, act="gelu", out="bf16")
        q, s = tg.quantize_block(h, "row")
        y = tg.gemm_experts(q, s, self.w2, self.s2, r.offsets, out="bf16")
        return tg.combine(y, r.slots, r.weights)


def dense_step(x, w, grad):
    """Y = X W^T and its gradients (dX, dW) from dY, all products in block-scaled FP8."""
    wq, ws = tg.quantize_block(w, "tile")
    xq, xs = tg.quantize_block(x, "row")
    y = tg.gemm_scaled(xq, xs, wq.t(), ws.t(), out="bf16")
    gq, gs = tg.quantize_block(grad, "row")
    dx = tg.gemm_scaled(gq, gs, wq, ws, out="bf16")
    xc, xcs = tg.quantize_block(x, "col")                                # along the tokens
    gc, gcs = tg.quantize_block(grad, "col")
    dw = tg.gemm_scaled(gc.t(), gcs.t(), xc, xcs)
    return y, dx, dw


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def exact_layer(layer, x, w1, w2):
    """The layer on the unquantised weights in 64 bits, with the layer's own routing."""
    r = layer.route(x)
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for e in range(w1.shape[0]):
        t, j = (r.indices == e).nonzero(as_tuple=True)
        if len(t):
            h = x[t].double() @ w1[e].double().t()
            out.index_add_(0, t, r.weights[t, j].double()[:, None] * ((h * torch.special.ndtr(h)) @ w2[e].double().t()))
    return out


def timed(fn, passes=20):
    for _ in range(3):
        fn()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(passes):
        fn()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / passes * 1e3


def main(hidden=2048, inner=1024, experts=64, top_k=8, tokens=(16, 2048)) -> dict:
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")       # noqa: E731
    w1, w2 = rand(experts, inner, hidden) * hidden ** -0.5, rand(experts, hidden, inner) * inner ** -0.5
    layer = ExpertLayer(w1, w2, rand(hidden, experts) * hidden ** -0.5, 0.05 * rand(experts), top_k,
                        groups=8 if experts % 8 == 0 else 1, top_groups=4 if experts % 8 == 0 else 1)
    found = {}
    for t in tokens:
        x = rand(t, hidden).to(torch.bfloat16)
        found[f"experts, {t} tokens"] = off(layer(x), exact_layer(layer, x, w1, w2))
        print(f"expert layer, {t} tokens of {hidden}, {experts} experts of {inner}: "
              f"{timed(lambda: layer(x)):.1f} us, off by {found[f'experts, {t} tokens']:.3f}")
    t = max(tokens)
    x, g = rand(t, hidden).to(torch.bfloat16), rand(t, inner).to(torch.bfloat16)
    w = w1[0]
    y, dx, dw = dense_step(x, w, g)
    found["Y"] = off(y, x.double() @ w.double().t())
    found["dX"] = off(dx, g.double() @ w.double())
    found["dW"] = off(dw, g.double().t() @ x.double())
    print(f"dense step, {t} x {hidden} -> {inner}: {timed(lambda: dense_step(x, w, g)):.1f} us, "
          f"Y off by {found['Y']:.3f}, dX by {found['dX']:.3f}, dW by {found['dW']:.3f}")
    status = tg.gemm_get_status(torch.cuda.current_stream().cuda_stream)
    if status != tg.GEMM_OK:
        raise RuntimeError(tg.gemm_last_error())
    return found


if __name__ == "__main__":
    main()
