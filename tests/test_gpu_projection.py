"""The projection's loss and the low-rank adapters on the GPU, each against its
definition in 64 bits.

Bounds (stated before any run), u half a step of the 16-bit type (bf16 2^-8, fp16
2^-11), elementwise:

* A product's sum is within 1e-5 of the same sum over absolute values (the library's
  gate for FP32 accumulation of 16-bit inputs).
* A logit z is then off by at most e = 1e-5 D, D = max_v sum_k |h w|, capped or not
  (tanh has slope at most 1), plus for a cap c: 4 * 2^-24 c.  lse is off by no more than
  its logits, plus 2^-20 (exponentials within 2^-22, sums of up to 4 chains and joins
  within 2^-21 relative), plus 4 * 2^-24 |lse| for its own arithmetic; loss takes lse,
  1 - s logits and s mean logits: twice e + ..., and 2 a |lse| more for the z loss.
* d = grad (...) is off by u |d| (its rounding; FP16's is scaled into range: 2^-38 of the
  largest possible |d| besides) and by |grad| (1 + 2 a |lse|) p (2 e + 2^-19) for p;
  the cap's slope 1 - tanh^2 adds 2^-20 relative.  dH and dW are off by that against
  |W| or |H|, by 1e-5 of the sum of |d| |W| (|H|), and by u of themselves (fp16 outputs
  have a step of 2^-24 near zero: 2^-25).
* low = s (x . a) is off by 1e-5 |s| sum |x a| and u |low|; C, dX by that against the
  other factor, 1e-5 of the sums of magnitudes, times 1.13 (GELU's slope; its own
  4e-8 |x| is below), and by u of themselves; dA and dB by low's error against the
  activations, 1e-5 and u.
"""
import os
import subprocess
import sys

import pytest
import torch

import tiled_tensor_core_gemm_gb300 as tg
from tiled_tensor_core_gemm_gb300 import build as tgbuild

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {BF16: 0.0, F16: 2.0 ** -25, torch.float32: 0.0}
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def lib():
    tgbuild.build()
    return tg.load_library()


@pytest.fixture(autouse=True)
def options_and_status():
    yield
    for key in ("product_bn", "product_splits", "loss_columns"):
        tg.gemm_set_option(key, 0)
    s = torch.cuda.current_stream().cuda_stream
    assert tg.gemm_get_status(s) == tg.GEMM_OK, tg.gemm_last_error()


def randn(*shape, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def randint(lo, hi, n, seed=0, dtype=torch.int64):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(lo, hi, (n,), generator=g, device="cuda", dtype=dtype)


def padded(t, by=8):
    """t with rows that start on 16 bytes, NaN between them."""
    pitch = -(-t.shape[-1] // 8) * 8 + by
    held = torch.full((*t.shape[:-1], pitch), float("nan"), dtype=t.dtype, device=t.device)
    held[..., :t.shape[-1]] = t
    return held[..., :t.shape[-1]]


def within(got, want, bound, what):
    assert got.shape == want.shape
    got = got.double()
    assert bool(torch.isfinite(got).all()), what
    over = (got - want).abs() - bound
    assert float(over.max()) <= 0.0, f"{what}: {float(((got - want).abs() / bound.clamp_min(1e-300)).max()):.3g} of the bound"


# -------------------------------------------------------------------- loss ---
def made_loss(T, V, D, dtype, layout="vd", seed=1, ignored=0.2, spread=1.5):
    W = (randn(V, D, seed=seed) * spread * D ** -0.5).to(dtype)
    if layout == "dv":
        W = W.t().contiguous().t()
    elif layout == "padded":
        W = padded(W)
    y = randint(0, V, T, seed=seed + 1)
    H = (randn(T, D, seed=seed + 2) + 2.0 * W[y].float()).to(dtype)
    drop = torch.rand(T, generator=torch.Generator().manual_seed(seed)) < ignored
    y[drop.cuda()] = -100
    return H, W, y


def exact_loss(H, W, y, grad=None, softcap=0.0, smoothing=0.0, z_loss=0.0):
    """The definitions in 64 bits and the bounds above."""
    u, V = U[H.dtype], W.shape[0]
    h, w = H.double(), W.double()
    has = (y >= 0) & (y < V)
    h = torch.where(has[:, None], h, h.nan_to_num(0.0, 0.0, 0.0))
    z = h @ w.t()
    e = 1e-5 * (h.abs() @ w.abs().t()).amax(1) + 4 * 2.0 ** -24 * softcap
    t = torch.tanh(z / softcap) if softcap else torch.zeros_like(z)
    if softcap:
        z = softcap * t
    lse = torch.logsumexp(z, 1)
    hit = z.gather(1, y.clamp(0, V - 1)[:, None])[:, 0]
    loss = torch.where(has, lse - (1 - smoothing) * hit - smoothing / V * z.sum(1) + z_loss * lse ** 2, 0.0)
    e_lse = e + 2.0 ** -20 + 4 * 2.0 ** -24 * lse.abs()
    e_loss = e_lse * (1 + 2 * z_loss * lse.abs()) + e + 8 * 2.0 ** -24 * (lse.abs() + hit.abs() + z_loss * lse ** 2)
    out = dict(lse=(lse, e_lse), loss=(loss, torch.where(has, e_loss, 0.0)))
    if grad is not None:
        g = torch.where(has, grad.double(), 0.0)
        p = torch.exp(z - lse[:, None])
        top = g.abs() * (1 + 2 * z_loss * lse.abs())
        d = p * (1 + 2 * z_loss * lse)[:, None] - smoothing / V
        d[torch.arange(len(y), device=y.device), y.clamp(0, V - 1)] -= 1 - smoothing
        d = d * g[:, None] * (1 - t * t)
        e_d = u * d.abs() + top[:, None] * p * (2 * e[:, None] + 2.0 ** -19 + 4 * 2.0 ** -24 * lse.abs()[:, None])
        e_d += 2.0 ** -20 * top[:, None] * (p + smoothing / V) if softcap or smoothing else 0.0
        e_d += 2.0 ** -38 * top.max()
        e_d[torch.arange(len(y), device=y.device), y.clamp(0, V - 1)] += 2.0 ** -20 * top
        e_d = torch.where(has[:, None], e_d, 0.0)
        for name, a, b, eb in (("dH", d, w, e_d), ("dW", d.t(), h, e_d.t())):
            want = a @ b
            out[name] = (want, eb @ b.abs() + 1e-5 * (a.abs() @ b.abs()) + u * want.abs() * (1 + 2 * u) + TINY[H.dtype]
                         + u * (eb @ b.abs()))
    return out


def check_loss(H, W, y, grad=None, **how):
    loss, lse = tg.project_loss(H, W, y, **how)
    want = exact_loss(H, W, y, grad, **how)
    counts = (y >= 0) & (y < W.shape[0])
    within(lse[counts], want["lse"][0][counts], want["lse"][1][counts], "lse")
    within(loss, *want["loss"], "loss")
    assert bool((loss[~counts] == 0).all())
    if grad is not None:
        dH, dW = tg.project_loss_backward(grad, H, W, y, lse, **how)
        assert dH.dtype is H.dtype and dW.shape == W.shape
        within(dH, *want["dH"], "dH")
        within(dW, *want["dW"], "dW")
        assert bool((dH[~counts] == 0).all())
        return loss, lse, dH, dW
    return loss, lse


@pytest.mark.parametrize("dtype", (BF16, F16))
@pytest.mark.parametrize("layout", ("vd", "dv", "padded"))
@pytest.mark.parametrize("T,V,D", [(1, 1, 8), (1, 1000, 64), (1, 300, 77), (2, 129, 1), (17, 257, 72), (33, 1000, 77), (64, 64, 64),
                                   (127, 513, 130), (130, 255, 520), (300, 1111, 263), (257, 2049, 1032)])
def test_loss_and_its_gradients(T, V, D, layout, dtype):
    H, W, y = made_loss(T, V, D, dtype, layout, seed=T)
    check_loss(H, W, y, randn(T, seed=9).abs() + 0.1)


@pytest.mark.parametrize("bn", (128, 256))
@pytest.mark.parametrize("columns", (64, 256, 1024, 0))
@pytest.mark.parametrize("how", [dict(), dict(softcap=8.0, smoothing=0.1, z_loss=1e-2)])
def test_loss_in_pieces_of_the_vocabulary(columns, bn, how):
    H, W, y = made_loss(390, 2500, 200, BF16, seed=4)
    assert tg.gemm_set_option("loss_columns", columns) == 0 and tg.gemm_set_option("product_bn", bn) == 0
    check_loss(H, W, y, randn(390, seed=5), **how)


@pytest.mark.parametrize("columns", (0, 256))
@pytest.mark.parametrize("T,V,D", [(48, 6000, 64), (300, 20000, 130)])       # few tiles of dH over a long vocabulary
def test_loss_gradient_of_the_tokens_in_ranges(T, V, D, columns):
    tg.gemm_set_option("loss_columns", columns)
    H, W, y = made_loss(T, V, D, F16, seed=6)
    check_loss(H, W, y, randn(T, seed=5))


@pytest.mark.parametrize("dtype", (BF16, F16))
@pytest.mark.parametrize("how", [dict(softcap=3.0), dict(softcap=50.0), dict(smoothing=0.3), dict(z_loss=0.1),
                                 dict(softcap=1.0, smoothing=0.9, z_loss=1.0)])
def test_loss_variants(how, dtype):
    # logits up to several times the cap
    H, W, y = made_loss(200, 777, 256, dtype, seed=7, spread=4.0)
    check_loss(H, W, y, randn(200, seed=8), **how)


@pytest.mark.parametrize("layout", ("vd", "dv"))
@pytest.mark.parametrize("bn", (0, 128))
@pytest.mark.parametrize("T", (1, 3, 8, 16, 31, 32, 33, 200))       # few tokens: tiles of any width
def test_loss_of_few_tokens(T, bn, layout):
    tg.gemm_set_option("product_bn", bn)
    H, W, y = made_loss(T, 50021, 320, BF16, layout, seed=T)
    check_loss(H, W, y)


def test_loss_gradients_against_differences():
    H, W, y = made_loss(12, 50, 16, F16, seed=11, ignored=0.0)
    how = dict(softcap=5.0, smoothing=0.2, z_loss=0.05)
    _, lse = tg.project_loss(H, W, y, **how)
    dH, _ = tg.project_loss_backward(torch.ones(12, device="cuda"), H, W, y, lse, **how)
    # Central differences of step 2^-4, exact in the type: H is rounded to multiples of 2^-4 first.  The
    # loss is off by under 1e-5, a difference by 1e-5 / 2^-4 = 2e-4; the third derivative by under
    # h^2 |w|^3 / 6 < 2e-3 for |w| < 1.5; dH by 2^-10 of |dH| < 3.
    H = (H.float() * 16).round().div(16).to(F16)
    _, lse = tg.project_loss(H, W, y, **how)
    dH, _ = tg.project_loss_backward(torch.ones(12, device="cuda"), H, W, y, lse, **how)
    assert float(W.abs().max()) < 1.5 and float(dH.abs().max()) < 3
    for k in range(16):
        up, down = H.clone(), H.clone()
        up[:, k] += 2.0 ** -4
        down[:, k] -= 2.0 ** -4
        slope = (tg.project_loss(up, W, y, **how)[0] - tg.project_loss(down, W, y, **how)[0]) * 8
        assert float((slope - dH[:, k].float()).abs().max()) < 6e-3


def test_loss_of_tokens_that_do_not_count_whatever_they_hold():
    H, W, y = made_loss(150, 600, 96, BF16, seed=12)
    y[:4] = torch.tensor([-1, 600, 2 ** 40, -2 ** 40], device="cuda")
    drop = (y < 0) | (y >= 600)
    g = randn(150, seed=13)
    want = check_loss(H, W, y, g)
    H2, g2 = H.clone(), g.clone()
    H2[drop] = float("nan")
    H2[3] = float("inf")
    g2[drop] = float("nan")
    loss, lse = tg.project_loss(H2, W, y)
    dH, dW = tg.project_loss_backward(g2, H2, W, y, lse)
    assert torch.equal(loss, want[0]) and torch.equal(dH, want[2]) and torch.equal(dW, want[3])
    # nobody counts
    loss, lse = tg.project_loss(H2, W, torch.full_like(y, -100))
    dH, dW = tg.project_loss_backward(g2, H2, W, torch.full_like(y, -100), lse)
    assert not bool(loss.any()) and not bool(dH.any()) and not bool(dW.any())


def test_loss_of_a_token_that_is_not_finite_stays_in_its_row():
    H, W, y = made_loss(70, 300, 64, BF16, seed=14, ignored=0.0)
    want, lse = tg.project_loss(H, W, y)
    H[5] = float("nan")
    got, lse2 = tg.project_loss(H, W, y)
    keep = torch.arange(70, device="cuda") != 5
    assert bool(got[5].isnan()) and torch.equal(got[keep], want[keep]) and torch.equal(lse2[keep], lse[keep])


def test_loss_of_large_logits():
    # logits of +-3000: exponentials that would overflow; all but one column far below the largest
    H, W, y = made_loss(40, 200, 64, F16, seed=15, spread=1.0)
    H = (H.float() * 400).to(F16)
    check_loss(H, W, y, randn(40, seed=3))


@pytest.mark.parametrize("labels", (torch.int64, torch.int32))
def test_loss_strides_types_and_wanted_outputs(labels):
    H, W, y = made_loss(60, 500, 88, BF16, seed=16)
    y = y.to(labels)
    want = check_loss(H, W, y.long(), torch.full((60,), 0.25, device="cuda"))
    one = torch.full((1,), 0.25, device="cuda").expand(60)
    for h in (H, padded(H), padded(H, 3), torch.cat((H, H), 1)[:, 88:]):
        loss, lse = tg.project_loss(h, W, y)
        assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])
        dH, dW = tg.project_loss_backward(one, h, W, y, lse)
        assert torch.equal(dH, want[2]) and torch.equal(dW, want[3])
    dH, none = tg.project_loss_backward(one, H, W, y, lse, want_W=False)
    assert none is None and torch.equal(dH, want[2])
    none, dW = tg.project_loss_backward(one, H, W, y, lse, want_H=False)
    assert none is None and torch.equal(dW, want[3])


def test_loss_writes_its_outputs_only():
    T, V, D = 70, 333, 50
    H, W, y = made_loss(T, V, D, BF16, seed=17)
    lib, s = tg.load_library(), torch.cuda.current_stream().cuda_stream
    out = torch.full((2, T + 20), 7.0, device="cuda")
    rc = lib.gemm_project_loss(T, V, D, tg.GEMM_BF16, H.data_ptr(), D, W.data_ptr(), D, 0, y.data_ptr(), 8, None,
                               out[0, 10:].data_ptr(), out[1, 10:].data_ptr(), s)
    assert rc == 0, tg.gemm_last_error()
    want = exact_loss(H, W, y, torch.ones(T, device="cuda"))
    within(out[0, 10:10 + T], *want["loss"], "loss")
    assert bool((out[:, :10] == 7).all()) and bool((out[:, 10 + T:] == 7).all())
    for pitch in (D + 6, D + 7):                 # TMA stores and ordinary ones
        dH, dW = (torch.full((n + 2, pitch), 7.0, dtype=BF16, device="cuda") for n in (T, V))
        rc = lib.gemm_project_loss_backward(T, V, D, tg.GEMM_BF16, torch.ones(T, device="cuda").data_ptr(), 1, H.data_ptr(), D,
                                            W.data_ptr(), D, 0, y.data_ptr(), 8, None, out[1, 10:].data_ptr(),
                                            dH[1:].data_ptr(), pitch, dW[1:].data_ptr(), pitch, s)
        assert rc == 0, tg.gemm_last_error()
        for t, n, name in ((dH, T, "dH"), (dW, V, "dW")):
            within(t[1:-1, :D], *want[name], name)
            assert bool((t[0] == 7).all()) and bool((t[-1] == 7).all()) and bool((t[1:-1, D:] == 7).all())


def test_loss_of_nothing():
    H, W, y = made_loss(5, 40, 16, BF16, seed=18)
    loss, lse = tg.project_loss(H[:0], W, y[:0])
    assert loss.shape == lse.shape == (0,)
    dH, dW = tg.project_loss_backward(lse, H[:0], W, y[:0], lse)
    assert dH.shape == (0, 16) and not bool(dW.any())
    y[:] = 3
    loss, lse = tg.project_loss(H[:, :0], W[:, :0], y)             # every logit is 0
    # (within the bounds above at e = 0: 2^-20 and 4 * 2^-24 of log 40)
    assert float((lse - torch.log(torch.tensor(40.0))).abs().max()) < 2e-6 and torch.equal(loss, lse)


# ---------------------------------------------------------------- adapters ---
def made_adapters(T, K, N, r, L, dtype, order="mixed", w_major=0, seed=1):
    X = randn(T, K, seed=seed).to(dtype)
    W = padded((randn(K, N, seed=seed + 1) * K ** -0.5).to(dtype)) if not w_major else \
        padded((randn(N, K, seed=seed + 1) * K ** -0.5).to(dtype)).t()
    A, B = padded((randn(L, r, K, seed=seed + 2) * K ** -0.5).to(dtype)), padded((randn(L, r, N, seed=seed + 3) * r ** -0.5).to(dtype))
    ids = randint(-1, L, T, seed=seed + 4, dtype=torch.int32)
    if order == "sorted":
        ids = ids.sort().values
    elif order == "none":
        ids[:] = -1
    elif order == "one":
        ids[:] = L - 1
    scales = torch.linspace(0.5, 2.0, L, device="cuda")
    return X, W, A, B, ids, scales


def exact_adapters(X, W, A, B, ids, scales, dY=None, bias=None, act="none", out=None):
    dt, u = X.dtype, U[X.dtype]
    x, w, a, b, s = X.double(), W.double(), A.double(), B.double(), scales.double()
    y, e = x @ w, 1e-5 * (x.abs() @ w.abs())
    res = {}
    if dY is not None:
        g = dY.double()
        dX, e_x = g @ w.t(), 1e-5 * (g.abs() @ w.abs().t())
        dA, dB, e_a, e_b = (torch.zeros_like(t) for t in (a, b, a, b))
    for i in range(len(a)):
        t = (ids == i).nonzero()[:, 0]
        if not len(t):
            continue
        low = s[i] * (x[t] @ a[i].t())
        e_low = u * low.abs() + 1e-5 * s[i] * (x[t].abs() @ a[i].abs().t())
        y[t] += low @ b[i]
        e[t] += e_low @ b[i].abs() + 1e-5 * (low.abs() @ b[i].abs())
        if dY is not None:
            up = s[i] * (g[t] @ b[i].t())
            e_up = u * up.abs() + 1e-5 * s[i] * (g[t].abs() @ b[i].abs().t())
            dX[t] += up @ a[i]
            e_x[t] += e_up @ a[i].abs() + 1e-5 * (up.abs() @ a[i].abs())
            dA[i] = up.t() @ x[t]
            e_a[i] = e_up.t() @ x[t].abs() + 1e-5 * (up.abs().t() @ x[t].abs())
            dB[i] = low.t() @ g[t]
            e_b[i] = e_low.t() @ g[t].abs() + 1e-5 * (low.abs().t() @ g[t].abs())
    if bias is not None:
        y = y + bias.double()
        e = e + 2.0 ** -22 * bias.double().abs()
    if act == "relu":
        y = torch.relu(y)
    elif act == "gelu":
        e = 1.13 * e + 2.0 ** -22 * y.abs()
        y = y * torch.special.ndtr(y)
    o = {None: dt, "f32": torch.float32, "bf16": BF16, "f16": F16}[out]
    res["C"] = (y, (1 + U[o]) * e + U[o] * y.abs() + TINY[o])
    if dY is not None:
        for name, v, ev in (("dX", dX, e_x), ("dA", dA, e_a), ("dB", dB, e_b)):
            res[name] = (v, (1 + u) * ev + u * v.abs() + TINY[dt])
    return res


def check_adapters(X, W, A, B, ids, scales, dY=None, **kw):
    plan = tg.adapter_plan(ids, len(A), backward=dY is not None)
    want = exact_adapters(X, W, A, B, ids, scales, dY, kw.get("bias"), kw.get("act", "none"), kw.get("out"))
    got = [tg.gemm_adapters(X, W, A, B, plan, scales, **kw)]
    within(got[0], *want["C"], "C")
    if dY is not None:
        got += tg.gemm_adapters_backward(dY, X, W, A, B, plan, scales)
        for g, name in zip(got[1:], ("dX", "dA", "dB")):
            within(g, *want[name], name)
        none = [i for i in range(len(A)) if not bool((ids == i).any())]
        assert not bool(got[2][none].any()) and not bool(got[3][none].any())
    return got


@pytest.mark.parametrize("w_major", (0, 1))
@pytest.mark.parametrize("T", (1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 300, 512, 513, 800))
def test_adapters_and_their_gradients(T, w_major):
    X, W, A, B, ids, s = made_adapters(T, 200, 328, 16, 5, BF16, w_major=w_major, seed=T)
    check_adapters(X, W, A, B, ids, s, randn(T, 328, seed=99).to(BF16))


@pytest.mark.parametrize("dtype", (BF16, F16))
@pytest.mark.parametrize("rank", (1, 3, 8, 16, 17, 32, 33, 64, 65, 128))
@pytest.mark.parametrize("T", (40, 600))
def test_adapters_of_every_rank(T, rank, dtype):
    X, W, A, B, ids, s = made_adapters(T, 264, 136, rank, 7, dtype, seed=rank)
    check_adapters(X, W, A, B, ids, s, randn(T, 136, seed=98).to(dtype))


@pytest.mark.parametrize("dtype", (BF16, F16))
@pytest.mark.parametrize("T,rank,L", [(1, 1, 1), (2, 16, 2), (16, 3, 4), (32, 128, 3), (33, 1, 1), (90, 8, 30), (600, 1, 1), (600, 100, 3)])
def test_adapters_gradients_and_few_tokens_are_as_exact_as_their_result(T, rank, L, dtype):
    # low is two numbers of the type, together within u^2 / 2 relative (fp16: or 2^-25, half its smallest step) of the
    # sum in FP32: the bounds above with that for u
    X, W, A, B, ids, s = made_adapters(T, 136, 200, rank, L, dtype, seed=rank)
    dY = randn(T, 200, seed=97).to(dtype)
    plan = tg.adapter_plan(ids, L, backward=True)
    C = tg.gemm_adapters(X, W, A, B, plan, s)
    dX, dA, dB = tg.gemm_adapters_backward(dY, X, W, A, B, plan, s)
    u = U[dtype]
    try:
        U[dtype] = u * u
        want = exact_adapters(X, W, A, B, ids, s, dY)
    finally:
        U[dtype] = u
    pairs = [(dA, "dA", X), (dB, "dB", dY)] + ([(C, "C", B), (dX, "dX", A)] if T <= 32 else [])
    for got, name, other in pairs:
        v, e = want[name]
        floor = TINY[dtype] * (1 + float(other.abs().max()) * (T if name in ("dA", "dB") else rank))
        within(got, v, e * (1 + u) + u * v.abs() + floor, name)


@pytest.mark.parametrize("order", ("mixed", "sorted", "none", "one"))
@pytest.mark.parametrize("T,L", [(1, 1), (64, 300), (100, 2), (700, 40), (1100, 600)])
def test_adapters_in_any_order(T, L, order):
    X, W, A, B, ids, s = made_adapters(T, 136, 200, 8, L, BF16, order, seed=L)
    check_adapters(X, W, A, B, ids, s, randn(T, 200, seed=97).to(BF16))


@pytest.mark.parametrize("K,N", [(1, 1), (1, 300), (300, 1), (63, 65), (77, 129), (1001, 130), (130, 1001)])
@pytest.mark.parametrize("T", (1, 3, 130, 530))
def test_adapters_of_odd_sizes(T, K, N):
    X, W, A, B, ids, s = made_adapters(T, K, N, 12, 3, F16, seed=K)
    check_adapters(X, W, A, B, ids, s, randn(T, N, seed=96).to(F16))


@pytest.mark.parametrize("splits", (1, 2, 3, 4))
@pytest.mark.parametrize("T", (9, 30, 60, 200))
def test_adapters_in_ranges_of_k(T, splits):
    tg.gemm_set_option("product_splits", splits)
    X, W, A, B, ids, s = made_adapters(T, 1100, 1032, 16, 30, BF16, seed=T)
    check_adapters(X, W, A, B, ids, s, randn(T, 1032, seed=95).to(BF16))


@pytest.mark.parametrize("bn", (128, 256))
@pytest.mark.parametrize("w_major", (0, 1))
def test_adapters_of_many_tokens_in_both_tiles(bn, w_major):
    tg.gemm_set_option("product_bn", bn)
    X, W, A, B, ids, s = made_adapters(1000, 520, 1100, 64, 9, BF16, w_major=w_major, seed=3)
    check_adapters(X, W, A, B, ids, s, randn(1000, 1100, seed=94).to(BF16))


@pytest.mark.parametrize("T", (20, 150, 700))
@pytest.mark.parametrize("out", ("f32", "bf16", "f16"))
@pytest.mark.parametrize("act", ("none", "relu", "gelu"))
def test_adapters_epilogue_and_guarded_c(T, out, act):
    X, W, A, B, ids, s = made_adapters(T, 144, 181, 16, 4, BF16, seed=T)
    bias = randn(181, seed=5)
    dt = {"f32": torch.float32, "bf16": BF16, "f16": F16}[out]
    held = torch.full((T + 2, 200), 7.0, dtype=dt, device="cuda")
    C = held[1:-1, 8:189]
    check_adapters(X, W, A, B, ids, s, bias=bias, act=act, out=out, C=C)
    held[1:-1, 8:189] = 7
    assert bool((held == 7).all())


@pytest.mark.parametrize("T", (20, 150, 700))
def test_adapters_strides_and_scales(T):
    X, W, A, B, ids, s = made_adapters(T, 96, 120, 16, 4, BF16, seed=T)
    plan = tg.adapter_plan(ids, 4, backward=True)
    dY = randn(T, 120, seed=2).to(BF16)
    want = [tg.gemm_adapters(X, W, A, B, plan, s), *tg.gemm_adapters_backward(dY, X, W, A, B, plan, s)]
    wide = lambda t: torch.cat((t, t, t), 1)[:, t.shape[1] + 1:2 * t.shape[1] + 1]      # noqa: E731
    odd = lambda t: wide(torch.cat((t[:, -1:], t[:, :-1]), 1))                           # noqa: E731
    assert torch.equal(odd(X), X)
    big = lambda t: torch.stack((t, t + 1), 1).flatten(0, 1)[::2]                         # noqa: E731
    for x, g, a, b in ((padded(X), padded(dY), big(A), B), (odd(X), odd(dY), A, big(B))):
        got = [tg.gemm_adapters(x, W, a, b, plan, s), *tg.gemm_adapters_backward(g, x, W, a, b, plan, s)]
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    ones = [tg.gemm_adapters(X, W, A, B, plan), *tg.gemm_adapters_backward(dY, X, W, A, B, plan)]
    same = [tg.gemm_adapters(X, W, A, B, plan, torch.ones_like(s)),
            *tg.gemm_adapters_backward(dY, X, W, A, B, plan, torch.ones_like(s))]
    assert all(torch.equal(p, q) for p, q in zip(ones, same))
    only = tg.gemm_adapters_backward(dY, X, W, A, B, plan, s, want_adapters=False)
    assert torch.equal(only[0], want[1]) and only[1] is only[2] is None
    only = tg.gemm_adapters_backward(dY, X, W, A, B, plan, s, want_X=False)
    assert only[0] is None and torch.equal(only[1], want[2]) and torch.equal(only[2], want[3])


def test_adapters_ids_outside_take_none_and_unused_adapters_are_not_read():
    X, W, A, B, ids, s = made_adapters(90, 128, 128, 16, 6, BF16, seed=8)
    ids[ids == 2] = 3
    ids[:3] = torch.tensor([6, 2 ** 31 - 1, -2 ** 31], device="cuda", dtype=torch.int32)
    plain = torch.where((ids >= 0) & (ids < 6), ids, -1)
    dY = randn(90, 128, seed=2).to(BF16)
    want = check_adapters(X, W, A, B, plain, s, dY)
    A[2], B[2] = float("nan"), float("inf")
    plan = tg.adapter_plan(ids, 6, backward=True)
    got = [tg.gemm_adapters(X, W, A, B, plan, s), *tg.gemm_adapters_backward(dY, X, W, A, B, plan, s)]
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("T", (30, 100, 600))
def test_adapters_of_a_token_that_is_not_finite_stay_in_its_row(T):
    X, W, A, B, ids, s = made_adapters(T, 128, 160, 16, 4, BF16, seed=9)
    plan = tg.adapter_plan(ids, 4)
    want = tg.gemm_adapters(X, W, A, B, plan, s)
    X[7], X[11] = float("nan"), float("inf")
    got = tg.gemm_adapters(X, W, A, B, plan, s)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[7] = keep[11] = False
    assert torch.equal(got[keep], want[keep]) and bool(got[7].isnan().all()) and not bool(torch.isfinite(got[11]).any())


def test_adapters_gradients_against_differences():
    # f(A, B) = sum dY * C is linear in A and in B: differences of any step are exact but for rounding.  C in FP32
    # is off by 1e-5 of sums of magnitudes and low's rounding, 2^-8 of 16-term sums: against steps of 1 under 2e-2 of
    # the sum of |dY| |low| |B|, itself under 40 here.
    X, W, A, B, ids, s = made_adapters(24, 16, 16, 4, 2, BF16, seed=10)
    plan = tg.adapter_plan(ids, 2, backward=True)
    dY = randn(24, 16, seed=11).to(BF16)
    _, dA, dB = tg.gemm_adapters_backward(dY, X, W, A, B, plan, s)

    def f(a, b):
        return float((tg.gemm_adapters(X, W, a, b, plan, s, out="f32").double() * dY.double()).sum())
    for which, grad in ((0, dA), (1, dB)):
        for i, c, k in ((0, 0, 0), (1, 3, 15), (1, 2, 7), (0, 1, 8)):
            up, down = [A.clone(), B.clone()], [A.clone(), B.clone()]
            up[which][i, c, k] = 1.0
            down[which][i, c, k] = -1.0
            assert abs((f(*up) - f(*down)) / 2 - float(grad[i, c, k])) < 0.8


def test_adapters_of_nothing():
    X, W, A, B, ids, s = made_adapters(4, 24, 32, 8, 3, BF16, seed=12)
    plan = tg.adapter_plan(ids[:0], 3, backward=True)
    assert tg.gemm_adapters(X[:0], W, A, B, plan, s).shape == (0, 32)
    dX, dA, dB = tg.gemm_adapters_backward(X.new_empty(0, 32), X[:0], W, A, B, plan, s)
    assert dX.shape == (0, 24) and not bool(dA.any()) and not bool(dB.any())
    plan = tg.adapter_plan(ids, 3, backward=True)
    C = tg.gemm_adapters(X[:, :0], W[:0], A[..., :0], B, plan, s)
    assert C.shape == (4, 32) and not bool(C.any())
    dX, dA, dB = tg.gemm_adapters_backward(X.new_empty(4, 0), X, W[:, :0], A, B[..., :0], plan, s)
    assert not bool(dX.any()) and not bool(dA.any()) and dB.shape == (3, 8, 0)


def test_adapters_small_integers_are_exact():
    for T in (10, 100, 600):
        X, W = randint(-3, 4, T * 128).view(T, 128).to(BF16), randint(-3, 4, 128 * 136, seed=1).view(128, 136).to(BF16)
        A, B = randint(-1, 2, 4 * 8 * 128, seed=2).view(4, 8, 128).to(BF16), randint(-1, 2, 4 * 8 * 136, seed=3).view(4, 8, 136).to(BF16)
        A[..., 8:] = 0                                     # sums of 8 products of 3: exact in BF16
        ids = randint(-1, 4, T, seed=4, dtype=torch.int32)
        got = tg.gemm_adapters(X, W, A, B, tg.adapter_plan(ids, 4), out="f32")
        want = X.double() @ W.double()
        for i in range(4):
            t = (ids == i).nonzero()[:, 0]
            want[t] += (X[t].double() @ A[i].double().t()) @ B[i].double()
        assert torch.equal(got.double(), want)


@pytest.mark.parametrize("K,N", [(64, 31000), (22000, 64)])
def test_adapters_past_32_bits(K, N):
    # C and the rank-wide activations pass 2^31 elements; a wide K makes the latter long work, whose end is waited for
    T, L, r = 70000, 260, 128
    X, W, A, B, ids, s = made_adapters(T, K, N, r, L, BF16, seed=13)
    plan = tg.adapter_plan(ids, L)
    C = tg.gemm_adapters(X, W, A, B, plan, s)
    at = torch.tensor([0, 1, 255, 256, 34634, 34635, 69275, 69999], device="cuda")
    want = exact_adapters(X[at], W, A, B, ids[at], s)
    within(C[at], *want["C"], "C")


# ---------------------------------------------------------------- together ---
def test_products_repeat_bit_for_bit_on_other_streams():
    H, W, y = made_loss(520, 3000, 264, BF16, seed=20)
    X, P, A, B, ids, s = made_adapters(520, 264, 264, 16, 9, BF16, seed=21)
    g = torch.full((1,), 1.0 / 520, device="cuda").expand(520)

    def step():
        plan = tg.adapter_plan(ids, 9, backward=True)
        h = tg.gemm_adapters(H, P, A, B, plan, s, act="gelu")
        loss, lse = tg.project_loss(h, W, y)
        dh, dW = tg.project_loss_backward(g, h, W, y, lse)
        return (h, loss, lse, dh, dW, *tg.gemm_adapters_backward(dh, H, P, A, B, plan, s))
    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(step())
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_products_in_cuda_graphs_that_run_at_once():
    ids = randint(-1, 6, 40, seed=30, dtype=torch.int32)
    X, W, A, B, _, s = made_adapters(40, 256, 512, 16, 6, BF16, seed=31)
    H, V, y = made_loss(40, 2000, 512, BF16, seed=32)

    def step():
        h = tg.gemm_adapters(X, W, A, B, tg.adapter_plan(ids, 6), s)
        loss, lse = tg.project_loss(h, V, y)
        return h, loss, lse, *tg.project_loss_backward(torch.ones_like(loss), h, V, y, lse)
    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out, torch.cuda.Stream()))
    ids.copy_(randint(-1, 6, 40, seed=33, dtype=torch.int32))
    X.copy_(randn(40, 256, seed=34).to(BF16))
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, _, st in graphs:
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    want = step()
    for _, out, _ in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


FIRST_CALL_IN_A_CAPTURE = """
import torch
import tiled_tensor_core_gemm_gb300 as tg
gen = torch.Generator(device="cuda")
gen.manual_seed(1)
rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
X, W, A, B, V = rand(20, 129), rand(129, 136), rand(3, 8, 136)[..., :129], rand(3, 8, 136), rand(500, 136)
ids = torch.arange(20, device="cuda", dtype=torch.int32) % 4 - 1
y = torch.arange(20, device="cuda")
def step():
    h = tg.gemm_adapters(X, W, A, B, tg.adapter_plan(ids, 3))
    return h, *tg.project_loss(h, V, y)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
for _ in range(3):
    graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in out]
assert all(torch.equal(a, b) for a, b in zip(got, step()))
print("equal")
"""


def test_the_first_call_may_be_in_a_capture():
    run = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "equal" in run.stdout, run.stderr[-2000:]


@pytest.mark.parametrize("T", (8, 100, 600))
def test_a_wait_that_runs_out_is_reported_and_leaves_the_device_usable(T):
    X, W, A, B, ids, s = made_adapters(T, 600, 512, 16, 3, BF16, seed=40)
    H, V, y = made_loss(T, 2000, 512, BF16, seed=41)
    plan = tg.adapter_plan(ids, 3)
    want, loss = tg.gemm_adapters(X, W, A, B, plan, s), tg.project_loss(H, V, y)[0]
    stream = torch.cuda.current_stream().cuda_stream
    for call in (lambda: tg.gemm_adapters(X, W, A, B, plan, s), lambda: tg.project_loss(H, V, y)):
        assert tg.gemm_set_option("wait_timeout_ms", 100) == 0 and tg.gemm_set_option("debug_stall_mma", 1) == 0
        try:
            call()
            assert tg.gemm_get_status(stream) == tg.GEMM_ERR_TIMEOUT
            assert "role=mma" in tg.gemm_last_error()
        finally:
            tg.gemm_set_option("wait_timeout_ms", 2000)
            tg.gemm_set_option("debug_stall_mma", 0)
        while tg.gemm_get_status(stream) != tg.GEMM_OK:      # (each launch of the call reports its own)
            pass
    assert torch.equal(tg.gemm_adapters(X, W, A, B, plan, s), want) and torch.equal(tg.project_loss(H, V, y)[0], loss)


def test_weights_tma_cannot_address_are_refused():
    X, W, A, B, ids, s = made_adapters(10, 64, 72, 8, 3, BF16, seed=50)
    plan = tg.adapter_plan(ids, 3)
    odd = lambda t: torch.cat((t, t[..., :1]), -1)[..., :-1]          # noqa: E731   (a pitch of 65 or 73)
    for w, a, b in ((odd(W), A, B), (W, odd(A), B), (W, A, odd(B))):
        with pytest.raises(tg.GemmError, match="16 bytes"):
            tg.gemm_adapters(X, w, a, b, plan, s)


def test_the_example_runs_them_together():
    import importlib.util
    spec = importlib.util.spec_from_file_location("adapter_training", os.path.join(ROOT, "examples", "adapter_training.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    found = example.main(tokens=300, dim=256, inner=384, vocab=1000, rank=8, adapters=3, steps=2)
    # Two roundings to BF16 in a row on each way (half steps of 2^-8, 1.7e-3 rms each), three products deep, and
    # the loss's own d: under 1% of each gradient.
    assert all(v < 0.01 for v in found.values()), found


@pytest.mark.parametrize("T", (65536, 70000))           # statistics 65536 tokens at a time; dW without the rests beyond
def test_loss_of_many_tokens(T):
    H, W, y = made_loss(T, 320, 72, BF16, seed=21)
    check_loss(H[:, :65], W[:, :65], y, torch.full((1,), 1.0 / T, device="cuda").expand(T), smoothing=0.1)


def test_loss_past_32_bits():
    # W and dW pass 2^31 elements; labels at both ends
    T, V, D = 3, 530000, 4104
    W = torch.empty((V, D), dtype=BF16, device="cuda")
    for v in range(0, V, 50000):
        W[v:v + 50000] = randn(min(50000, V - v), D, seed=v) * D ** -0.5
    H, y = randn(T, D, seed=1).to(BF16), torch.tensor([V - 1, 0, V // 2], device="cuda")
    loss, lse = tg.project_loss(H, W, y)
    z = torch.cat([H.double() @ W[v:v + 50000].double().t() for v in range(0, V, 50000)], 1)
    want = torch.logsumexp(z, 1)
    # (the bounds above with D = max sum |h w| under 60)
    assert float((lse - want).abs().max()) < 6e-4 + 1e-5
    assert float((loss - (want - z.gather(1, y[:, None])[:, 0])).abs().max()) < 1.3e-3
    _, dW = tg.project_loss_backward(torch.ones(T, device="cuda"), H, W, y, lse, want_H=False)
    at = torch.tensor([0, 1, 523264, 523265, V // 2, V - 2, V - 1], device="cuda")
    d = torch.exp(z - want[:, None])
    d[torch.arange(T, device="cuda"), y] -= 1
    exact = d[:, at].t() @ H.double()
    bound = (U[BF16] * 2 + 1.5e-3) * (d[:, at].abs().t() @ H.double().abs()) + U[BF16] * exact.abs()
    within(dW[at], exact, bound, "dW")


@pytest.mark.parametrize("dtype", (BF16, F16))
@pytest.mark.parametrize("T", (1, 20, 32, 33, 200))
def test_adapters_of_a_token_with_an_infinity_are_infinite(T, dtype):
    # every factor positive: inf and nothing that could cancel it, whichever way low is held
    X, W, A, B, ids, s = made_adapters(T, 72, 88, 16, 3, dtype, seed=61)
    X, W, A, B, ids = X.abs() + 0.1, W.abs() + 0.01, A.abs() + 0.01, B.abs() + 0.01, ids.clamp_min(0)
    dY = randn(T, 88, seed=62).abs().to(dtype) + 0.1
    plan = tg.adapter_plan(ids, 3, backward=True)
    want = tg.gemm_adapters(X, W, A, B, plan, s), tg.gemm_adapters_backward(dY, X, W, A, B, plan, s, want_adapters=False)[0]
    t = min(T - 1, 5)
    X[t, 3], dY[t, 7] = float("inf"), float("inf")
    got = tg.gemm_adapters(X, W, A, B, plan, s), tg.gemm_adapters_backward(dY, X, W, A, B, plan, s, want_adapters=False)[0]
    keep = torch.arange(T, device="cuda") != t
    for g, w in zip(got, want):
        assert bool((g[t] == float("inf")).all()) and torch.equal(g[keep], w[keep])


def test_adapters_with_a_short_limit_on_waits():
    # low alone takes more than the limit (7e11 multiply-adds over the slots in use, 1.6 ms and more): the
    # projection's waits must not begin before it ends
    X, W, A, B, ids, s = made_adapters(8192, 4096, 256, 128, 256, BF16, seed=64)
    plan = tg.adapter_plan(ids, 256)
    want = tg.gemm_adapters(X, W, A, B, plan, s)
    stream = torch.cuda.current_stream().cuda_stream
    assert tg.gemm_get_status(stream) == tg.GEMM_OK
    assert tg.gemm_set_option("wait_timeout_ms", 1) == 0
    try:
        got = tg.gemm_adapters(X, W, A, B, plan, s)
        assert tg.gemm_get_status(stream) == tg.GEMM_OK, tg.gemm_last_error()
    finally:
        tg.gemm_set_option("wait_timeout_ms", 2000)
    assert torch.equal(got, want)


# What the rounding of d takes from its label entries and the products give back.  In the inputs below it is all
# there is: W's rows are alike within groups of 1 / p entries, the logits far lower outside a token's own group
# (sums exact in FP32: multiples of 2^-5 below 2^8), so d is grad p, exact in the type, but for the label's
# -grad (1 - p), and dH is 0.  Tokens come in pairs of one label, H = 1.5 h with grad = c and H = h with
# grad = -1.5 c, c a power of two: dW is 0 too.  1 - p has as many digits as the type, 1.5 (1 - p) one and a half
# more: a quarter of a step of its last digit goes, 2^-9 c (bf16) or 2^-12 c (fp16).
GROUP = {BF16: 256, F16: 2048}


def made_cancelling(runs, dtype, layout, seed, tokens=None):
    """Pairs by label, in a random order; tokens beyond them (up to `tokens`) do not count.  runs: pairs of each label."""
    size, groups, content = GROUP[dtype], 4, 24
    V, n = size * groups, len(runs)
    of = torch.arange(V, device="cuda") // size
    own = randint(0, 2, groups * content, seed=seed).view(groups, content) * 2 - 1
    W = torch.zeros(V, content + groups, device="cuda")
    W[:, :content] = (own * (0.5 + 0.5 * randint(0, 2, groups * content, seed=seed + 1).view(groups, content)))[of]
    W[torch.arange(V, device="cuda"), content + of] = 1.0
    labels = torch.randperm(V, generator=torch.Generator().manual_seed(seed))[:n].cuda()
    pair_label = labels.repeat_interleave(torch.tensor(runs, device="cuda"))
    pairs = len(pair_label)
    h = torch.zeros(pairs, content + groups, device="cuda")
    h[:, :content] = randint(-8, 9, pairs * content, seed=seed + 2).view(pairs, content) / 8.0
    h[torch.arange(pairs, device="cuda"), content + of[pair_label]] = 64.0
    c = 2.0 ** -randint(0, 3, pairs, seed=seed + 3).float()
    T = max(tokens or 0, 2 * pairs)
    H, g, y = torch.full((T, h.shape[1]), float("nan"), device="cuda"), torch.ones(T, device="cuda"), torch.full((T,), -100, device="cuda")
    at = torch.randperm(T, generator=torch.Generator().manual_seed(seed + 1))[:2 * pairs].cuda()
    H[at], g[at], y[at] = torch.cat((1.5 * h, h)), torch.cat((c, -1.5 * c)), torch.cat((pair_label, pair_label))
    W = W.to(dtype)
    return H.to(dtype), W.t().contiguous().t() if layout == "dv" else W, y, g


def check_cancelling(H, W, y, g):
    """dH and dW against 0, within FP32's error (a logit is exact, lse off by 2^-20 + 4 * 2^-24 |lse|, so p by
    twice that; d at the label by 2^-22 |grad| besides; products 1e-5 of the sum of magnitudes); and that the same
    without the labels' rests would be outside."""
    dtype = H.dtype
    _, lse = tg.project_loss(H, W, y)
    dH, dW = tg.project_loss_backward(g, H, W, y, lse)
    at = (y >= 0).nonzero()[:, 0]
    assert not bool(dH[y < 0].any())
    h, w, gg, yy, n = H[at].double(), W.double(), g[at].double(), y[at], torch.arange(len(at), device="cuda")
    dH_off, dW_off, dW_bound, dW_without = dH[at].double(), dW.double(), torch.zeros_like(w), torch.zeros_like(w)
    caught, tokens = 0, 0
    for s in range(0, len(at), 4096):
        m = slice(s, s + 4096)
        i = n[:len(yy[m])]
        z = h[m] @ w.t()
        l64 = torch.logsumexp(z, 1)
        p = torch.exp(z - l64[:, None])
        d = gg[m, None] * p
        d[i, yy[m]] -= gg[m]
        rounded = d.to(dtype).double() if dtype is BF16 else (d * 2.0 ** 12).to(dtype).double() * 2.0 ** -12
        e = gg[m].abs() * (2.0 ** -22 + p[i, yy[m]] * (2.0 ** -19 + 2.0 ** -21 * l64.abs()))
        beyond = torch.where(torch.arange(len(w), device="cuda") // GROUP[dtype] == (yy[m] // GROUP[dtype])[:, None], 0.0, 2 * d.abs())
        bound = e[:, None] * w[yy[m]].abs() + 1e-5 * (d.abs() @ w.abs()) + beyond @ w.abs() + TINY[dtype]
        assert float((dH_off[m].abs() - bound).max()) <= 0, "dH"
        wide = (gg[m] < 0)[:, None] & (w[yy[m]] != 0)
        caught += int(((rounded @ w).abs() > bound)[wide].sum())
        tokens += int(wide.sum())
        dW_bound += 1e-5 * (d.abs().t() @ h[m].abs()) + beyond.t() @ h[m].abs()
        dW_bound.index_add_(0, yy[m], e[:, None] * h[m].abs())
        dW_without += rounded.t() @ h[m]
    assert caught == tokens
    dW_bound += TINY[dtype]
    assert float((dW_off.abs() - dW_bound).max()) <= 0, "dW"
    used = torch.unique(yy)
    # (rows of several pairs may cancel in a column by chance)
    outside = (dW_without.abs() > dW_bound)[used].any(1)
    # Of 70000 tokens that count a group has 17500, whose p of 2^-8 make the bound 1e-5 * 17500 * 1.25 * 2^-8 |h| =
    # 8.5e-4 |h|: a single pair's rest, 2^-9 c |h|, is outside for c = 1, a third of them.
    assert bool(outside.all()) if len(at) <= 40000 else float(outside.double().mean()) > 0.25


@pytest.mark.parametrize("columns", (0, 512))
@pytest.mark.parametrize("layout", ("vd", "dv"))
@pytest.mark.parametrize("dtype", (BF16, F16))
def test_loss_gradients_lose_nothing_of_their_label_entries(dtype, layout, columns):
    tg.gemm_set_option("loss_columns", columns)
    check_cancelling(*made_cancelling([1] * 60 + list(range(2, 40)), dtype, layout, seed=70))


@pytest.mark.parametrize("layout", ("vd", "dv"))
@pytest.mark.parametrize("dtype", (BF16, F16))
@pytest.mark.parametrize("pairs", (1, 15, 16, 17, 40, 3000, 20000))
def test_loss_gradients_where_all_tokens_have_one_label(pairs, dtype, layout):
    check_cancelling(*made_cancelling([pairs], dtype, layout, seed=71))


def test_loss_gradient_takes_no_longer_where_all_tokens_have_one_label():
    # (six times as long when a label's tokens were summed one after another; measured 0.92)
    T, V, D = 65536, 256, 1024
    H, W, y = made_loss(T, V, D, BF16, seed=72, ignored=0.0)
    g, one = torch.ones(T, device="cuda"), torch.full_like(y, 5)

    def least(labels):
        _, lse = tg.project_loss(H, W, labels)
        took = []
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            tg.project_loss_backward(g, H, W, labels, lse)
            b.record()
            b.synchronize()
            took.append(a.elapsed_time(b))
        return min(took)
    mixed = least(y)
    assert least(one) < 2 * mixed


@pytest.mark.parametrize("labels", (torch.int64, torch.int32))
@pytest.mark.parametrize("tokens,pairs", [(4096, 2000), (4097, 2000), (70000, 4000), (70001, 35000), (200000, 900)])
def test_loss_gradients_lose_nothing_with_many_tokens(tokens, pairs, labels):
    # most of them do not count; labels of one pair and of many
    runs = [1] * 400 + [pairs // 4] + [2] * 100 + [pairs - 600 - pairs // 4]
    H, W, y, g = made_cancelling(runs, BF16, "vd", seed=73, tokens=tokens)
    check_cancelling(H, W, y.to(labels), g)


def test_loss_gradients_of_many_tokens_do_not_depend_on_how_they_are_ordered():
    # 4096 tokens are ordered by comparisons, with one more that does not count by passes over the labels' bits
    # (over a vocabulary of three such passes)
    T, V, D = 4096, 66000, 40
    H, W, y = made_loss(T, V, D, BF16, seed=74)
    y[::3] = 7
    g = randn(T, seed=75)
    _, lse = tg.project_loss(H, W, y)
    want = tg.project_loss_backward(g, H, W, y, lse)[1]
    more = lambda t, v: torch.cat((t[:100], t.new_full((1, *t.shape[1:]), v), t[100:]))       # noqa: E731
    H2, y2, g2, lse2 = more(H, 1.0), more(y, -1), more(g, 1.0), more(lse, 0.0)
    got = tg.project_loss_backward(g2, H2, W, y2, lse2)[1]
    # FP32 sums in another grouping (1e-5 of their magnitudes, over all 4096 tokens under 1e-5 * 4096 * |H|), and
    # one rounding: half a step of the larger
    off = (got.double() - want.double()).abs()
    p = torch.exp(H.double() @ W[:64].double().t() - lse.double()[:, None])
    p[torch.arange(T, device="cuda"), y.clamp(0, 63)] += ((y >= 0) & (y < 64)).double()
    d = torch.where((y >= 0)[:, None], g.double().abs()[:, None] * p, 0.0)
    bound = 2 * (1e-5 * (d.t() @ H.double().abs()) + U[BF16] * torch.maximum(got[:64].abs(), want[:64].abs()).double())
    assert float((off[:64] - bound).max()) <= 0


def test_loss_gradient_of_the_tokens_past_32_bits():
    # dH passes 2^31 elements, W's rows are gathered by label for its rests; checked at both ends and in the middle
    T, V, D = 65600, 300, 33000
    H, W = torch.empty((T, D), dtype=BF16, device="cuda"), (randn(V, D, seed=1) * D ** -0.5).to(BF16)
    for t in range(0, T, 8200):
        H[t:t + 8200] = randn(8200, D, seed=t)
    y, g = randint(0, V, T, seed=2), randn(T, seed=3)
    _, lse = tg.project_loss(H, W, y)
    dH, _ = tg.project_loss_backward(g, H, W, y, lse, want_W=False)
    at = torch.tensor([0, 1, 32800, 65074, 65075, 65076, T - 2, T - 1], device="cuda")
    want = exact_loss(H[at], W, y[at], g[at])["dH"]
    within(dH[at], *want, "dH")


@pytest.mark.parametrize("layout", ("vd", "dv"))
@pytest.mark.parametrize("T,V,D,columns", [(4097, 1, 8, 0), (4097, 255, 9, 64), (4100, 256, 1, 0), (5000, 65535, 16, 0), (4500, 65536, 24, 1024),
                                           (520, 40, 65, 0), (1030, 300, 130, 0)])
def test_loss_gradients_of_tokens_ordered_by_label(T, V, D, columns, layout):
    # labels of one, two and three bytes, tokens in several blocks of sums
    tg.gemm_set_option("loss_columns", columns)
    H, W, y = made_loss(T, V, D, BF16, layout, seed=80)
    y[1::2] = torch.where(y[1::2] >= 0, V // 2, y[1::2])
    g = randn(T, seed=81)
    _, lse, dH, dW = check_loss(H, W, y, g)
    again = tg.project_loss_backward(g, H, W, y, lse)
    assert torch.equal(again[0], dH) and torch.equal(again[1], dW)
    none = torch.full_like(y, V)
    dH, dW = tg.project_loss_backward(g, H, W, none, lse)
    assert not bool(dH.any()) and not bool(dW.any())
    only = tg.project_loss_backward(g, H, W, y, lse, want_W=False)
    assert torch.equal(only[0], again[0]) and only[1] is None


def test_loss_gradients_of_many_tokens_in_cuda_graphs_that_run_at_once():
    H, V, y = made_loss(5000, 700, 128, BF16, seed=82)
    g = randn(5000, seed=83)

    def step():
        loss, lse = tg.project_loss(H, V, y)
        return loss, *tg.project_loss_backward(g, H, V, y, lse)
    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out, torch.cuda.Stream()))
    y.copy_(randint(-1, 5, 5000, seed=84))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, _, st in graphs:
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    want = step()
    for _, out, _ in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
