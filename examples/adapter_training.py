"""Low-rank adapters and the projection's loss together, as a model uses them: a
training step of several adapters at once on frozen weights, and a decode step of
a batch whose requests each have an adapter of their own.

    python examples/adapter_training.py

The model is one block, h = x + gelu(x.W1 + adapter).W2 + adapter, and its
logits h.V^T.  The gradients are compared with the same computation in 64
bits; the timed calls are whole passes, on the device's clock.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_tensor_core_gemm_gb300 as tg  # noqa: E402


class Block:
    """x + up(x) through W2, W1 and W2 frozen, with a stack of adapters on each."""

    def __init__(self, dim, inner, vocab, rank, adapters, gen, dtype=torch.bfloat16):
        rand = lambda *s: torch.randn(s, generator=gen, device="cuda")          # noqa: E731
        self.w1, self.w2 = (rand(dim, inner) * dim ** -0.5).to(dtype), (rand(inner, dim) * inner ** -0.5).to(dtype)
        self.head = (rand(vocab, dim) * dim ** -0.5).to(dtype)
        self.a1, self.b1 = (rand(adapters, rank, dim) * dim ** -0.5).to(dtype), (0.1 * rand(adapters, rank, inner)).to(dtype)
        self.a2, self.b2 = (rand(adapters, rank, inner) * inner ** -0.5).to(dtype), (0.1 * rand(adapters, rank, dim)).to(dtype)
        self.scales = torch.full((adapters,), 2.0, device="cuda")

    def forward(self, x, plan):
        up = tg.gemm_adapters(x, self.w1, self.a1, self.b1, plan, self.scales)
        act = torch.nn.functional.gelu(up)
        return up, act, x + tg.gemm_adapters(act, self.w2, self.a2, self.b2, plan, self.scales)

    def step(self, x, ids, labels):
        """The losses and the adapters' gradients of their mean."""
        plan = tg.adapter_plan(ids, len(self.scales), backward=True)            # once, for both projections
        up, act, h = self.forward(x, plan)
        loss, lse = tg.project_loss(h, self.head, labels)
        mean = 1.0 / (labels >= 0).sum().clamp_min(1).float()
        dh, _ = tg.project_loss_backward(mean.expand(len(loss)), h, self.head, labels, lse, want_W=False)
        dact, da2, db2 = tg.gemm_adapters_backward(dh, act, self.w2, self.a2, self.b2, plan, self.scales)
        dup = torch.ops.aten.gelu_backward(dact, up)
        _, da1, db1 = tg.gemm_adapters_backward(dup, x, self.w1, self.a1, self.b1, plan, self.scales, want_X=False)
        return loss, (da1, db1, da2, db2)


def exact_step(block, x, ids, labels):
    """The same in 64 bits, gradients by differentiation."""
    a1, b1, a2, b2 = (t.double().requires_grad_() for t in (block.a1, block.b1, block.a2, block.b2))

    def project(v, w, a, b):
        y = v @ w.double()
        for i in range(len(a)):
            at = (ids == i).nonzero()[:, 0]
            y = y.index_add(0, at, block.scales[i].double() * ((v[at] @ a[i].t()) @ b[i]))
        return y
    x = x.double()
    h = x + project(torch.nn.functional.gelu(project(x, block.w1, a1, b1)), block.w2, a2, b2)
    loss = torch.nn.functional.cross_entropy(h @ block.head.double().t(), labels, ignore_index=-100, reduction="none")
    (loss.sum() / (labels >= 0).sum()).backward()
    return loss.detach(), [t.grad for t in (a1, b1, a2, b2)]


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def timed(fn, passes=10):
    for _ in range(3):
        fn()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(passes):
        fn()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / passes * 1e3


def main(tokens=4096, dim=2048, inner=4096, vocab=32000, rank=16, adapters=4, steps=3) -> dict:
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    block = Block(dim, inner, vocab, rank, adapters, gen)
    x = torch.randn((tokens, dim), generator=gen, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, adapters, (tokens,), generator=gen, device="cuda", dtype=torch.int32).sort().values
    labels = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    labels[::7] = -100                                                          # prompts and padding
    loss, grads = block.step(x, ids, labels)
    want, exact = exact_step(block, x, ids, labels)
    found = {"loss": off(loss, want)}
    found.update({name: off(g, e) for name, g, e in zip(("dA1", "dB1", "dA2", "dB2"), grads, exact)})
    for _ in range(steps):                                                      # plain descent on the adapters
        _, grads = block.step(x, ids, labels)
        for p, g in zip((block.a1, block.b1, block.a2, block.b2), grads):
            p.sub_(g, alpha=0.1)
    print(f"training step, {tokens} tokens of {dim}, {adapters} adapters of rank {rank}, vocabulary {vocab}: "
          f"{timed(lambda: block.step(x, ids, labels)):.0f} us; off by " +
          ", ".join(f"{k} {v:.4f}" for k, v in found.items()))
    few = min(32, tokens)
    plan = tg.adapter_plan(ids[:few].contiguous(), adapters)
    print(f"decode step of {few}: {timed(lambda: block.forward(x[:few], plan)):.0f} us")
    status = tg.gemm_get_status(torch.cuda.current_stream().cuda_stream)
    if status != tg.GEMM_OK:
        raise RuntimeError(tg.gemm_last_error())
    return found


if __name__ == "__main__":
    main()
