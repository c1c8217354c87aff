"""The projection's loss and the adapters without a GPU: what the C entries and the
Python functions refuse, before any CUDA call, and what they do for nothing."""
import ctypes
import os
import re

import pytest
import torch

import tiled_tensor_core_gemm_gb300 as tg
from tiled_tensor_core_gemm_gb300 import build as tgbuild
from tiled_tensor_core_gemm_gb300 import projection

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD = tg.GEMM_ERR_INVALID_ARG
P = 1 << 24      # an aligned address no call below gets to touch


@pytest.fixture(scope="module")
def lib():
    tgbuild.build()
    return tg.load_library()


def refused(rc, frag, code=BAD):
    assert rc == code, (rc, tg.gemm_last_error())
    assert frag in tg.gemm_last_error(), tg.gemm_last_error()


def test_every_declared_entry_is_bound(lib):
    text = open(os.path.join(ROOT, "include", "gemm_project.h")).read()
    names = set(re.findall(r"GEMM_API \w+ (gemm_\w+)\(", text))
    assert len(names) == 6 and names <= set(tg.EXPORTED)
    for n in names:
        assert getattr(lib, n).argtypes is not None


# -------------------------------------------------------------------- loss ---
def loss(lib, T=8, V=100, D=64, dtype=tg.GEMM_BF16, H=P, ldh=64, W=P << 1, ldw=64, major=0, labels=P << 2, lb=8, how=None,
         out=P << 3, lse=P << 4):
    return lib.gemm_project_loss(T, V, D, dtype, H, ldh, W, ldw, major, labels, lb, how, out, lse, None)


def variant(softcap=0.0, smoothing=0.0, z_loss=0.0):
    return ctypes.byref(projection.Loss(softcap, smoothing, z_loss))


NAN = float("nan")


@pytest.mark.parametrize("kw,frag", [
    (dict(dtype=tg.GEMM_FP32), "BF16"), (dict(dtype=tg.GEMM_E4M3), "BF16"), (dict(T=-1), "size"), (dict(V=0), "size"),
    (dict(D=-1), "size"), (dict(V=1 << 31), "size"), (dict(T=1 << 31), "size"), (dict(major=2), "w_major"),
    (dict(lb=2), "label_bytes"), (dict(ldh=63), "leading"), (dict(ldw=63), "leading"), (dict(major=1, ldw=99), "leading"),
    (dict(ldh=0), "leading"), (dict(ldw=1 << 37), "leading"), (dict(H=0), "H is NULL"), (dict(W=0), "W is NULL"),
    (dict(labels=0), "labels is NULL"), (dict(lse=0), "lse is NULL"), (dict(H=P + 1), "aligned"),
    (dict(labels=(P << 2) + 4), "aligned"), (dict(lse=(P << 3) + 16), "overlap"), (dict(out=P + 64), "overlap"),
    (dict(how=variant(softcap=-1.0)), "softcap"), (dict(how=variant(softcap=NAN)), "softcap"),
    (dict(how=variant(smoothing=1.0)), "smoothing"), (dict(how=variant(smoothing=-0.1)), "smoothing"),
    (dict(how=variant(z_loss=-1.0)), "z_loss"), (dict(how=variant(z_loss=NAN)), "z_loss"),
    (dict(V=(1 << 31) - 600, ldw=1 << 36), "extent"),
])
def test_loss_refuses(lib, kw, frag):
    refused(loss(lib, **kw), frag)


def backward(lib, T=8, V=100, D=64, dtype=tg.GEMM_BF16, grad=P >> 1, gs=1, H=P, ldh=64, W=P << 1, ldw=64, major=0,
             labels=P << 2, lb=8, how=None, lse=P << 4, dH=P << 5, lddh=64, dW=P << 6, lddw=64):
    return lib.gemm_project_loss_backward(T, V, D, dtype, grad, gs, H, ldh, W, ldw, major, labels, lb, how, lse, dH, lddh, dW,
                                          lddw, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(gs=2), "grad_stride"), (dict(gs=-1), "grad_stride"), (dict(lddh=63), "leading"), (dict(lddw=63), "leading"),
    (dict(major=1, ldw=100, lddw=99), "leading"), (dict(grad=0), "grad is NULL"), (dict(lse=0), "lse is NULL"),
    (dict(dH=P), "overlap"), (dict(dW=P << 1), "overlap"), (dict(dW=(P << 5) + 64), "overlap"), (dict(dH=(P << 5) + 1), "aligned"),
    (dict(dtype=tg.GEMM_TF32), "BF16"),
])
def test_loss_backward_refuses(lib, kw, frag):
    refused(backward(lib, **kw), frag)


def test_loss_of_nothing(lib):
    assert loss(lib, T=0) == tg.GEMM_OK
    assert backward(lib, dH=None, dW=None) == tg.GEMM_OK
    assert backward(lib, D=0, ldh=1, ldw=1) == tg.GEMM_OK


def test_loss_pitches_of_what_is_not_wanted_are_not_looked_at(lib):
    for kw in (dict(dH=None, lddh=0), dict(dW=None, lddw=0)):
        rc = backward(lib, **kw)
        assert rc != tg.GEMM_OK and "leading" not in tg.gemm_last_error()


# ---------------------------------------------------------------- adapters ---
def stack(count=4, rank=8, A=P << 2, lda=64, sa=512, B=P << 3, ldb=96, sb=768, scales=None):
    return ctypes.byref(projection.Adapters(count, rank, A, lda, sa, B, ldb, sb, scales))


def adapters(lib, T=8, N=96, K=64, dtype=tg.GEMM_BF16, X=P, ldx=64, W=P << 1, ldw=96, major=0, ad=None, plan=P << 4, C=P << 5,
             ldc=96, epi=None):
    return lib.gemm_adapters(T, N, K, dtype, X, ldx, W, ldw, major, ad or stack(), plan, C, ldc, epi, None)


def epilogue(**kw):
    return ctypes.byref(tg.make_epilogue(kw["alpha"], kw["beta"], kw["bias"], kw["act"], kw["out"]))


@pytest.mark.parametrize("kw,frag", [
    (dict(dtype=tg.GEMM_FP32), "BF16"), (dict(T=-1), "size"), (dict(N=1 << 31), "size"), (dict(T=(1 << 23) + 1), "2^23"),
    (dict(major=2), "w_major"), (dict(ldw=95), "W"), (dict(major=1, ldw=63), "W"), (dict(ldx=63), "leading"),
    (dict(ldc=95), "leading"), (dict(ad=stack(count=0)), "4096"), (dict(ad=stack(count=4097)), "4096"),
    (dict(ad=stack(rank=0)), "128"), (dict(ad=stack(rank=129)), "128"), (dict(ad=stack(lda=63)), "adapters"),
    (dict(ad=stack(ldb=95)), "adapters"), (dict(ad=stack(sa=-8)), "adapters"), (dict(ad=stack(sa=0)), "adapters"),
    (dict(ad=stack(sb=1 << 39)), "adapters"), (dict(X=0), "X is NULL"), (dict(W=0), "W is NULL"),
    (dict(ad=stack(A=0)), "A is NULL"), (dict(ad=stack(B=0)), "B is NULL"), (dict(plan=0), "plan is NULL"),
    (dict(C=0), "C is NULL"), (dict(C=P + 64), "overlap"), (dict(C=(P << 4)), "overlap"), (dict(X=P + 1), "aligned"),
    (dict(plan=(P << 4) + 2), "aligned"), (dict(ad=stack(scales=(P << 6) + 1)), "aligned"),
])
def test_adapters_refuse(lib, kw, frag):
    refused(adapters(lib, **kw), frag)


def test_adapters_refuse_alpha_and_beta(lib):
    refused(adapters(lib, epi=epilogue(alpha=2.0, beta=0.0, bias=0, act="none", out="bf16")), "alpha")
    refused(adapters(lib, epi=epilogue(alpha=1.0, beta=1.0, bias=0, act="none", out="bf16")), "alpha")
    refused(lib.gemm_adapters(8, 96, 64, tg.GEMM_BF16, P, 64, P << 1, 96, 0, None, P << 4, P << 5, 96, None, None), "adapters is NULL")


@pytest.mark.parametrize("kw", [dict(W=(P << 1) + 2), dict(ldw=97), dict(ad=stack(A=(P << 2) + 8)), dict(ad=stack(lda=65)),
                                dict(ad=stack(sa=513)), dict(ad=stack(ldb=97)), dict(ad=stack(sb=769))])
def test_adapters_refuse_weights_tma_cannot_address(lib, kw):
    refused(adapters(lib, **kw), "16 bytes", tg.GEMM_ERR_UNSUPPORTED)


def grads(lib, T=8, N=96, K=64, dtype=tg.GEMM_BF16, dY=P >> 1, ldy=96, X=P, ldx=64, W=P << 1, ldw=96, major=0, ad=None,
          plan=P << 4, dX=P << 5, lddx=64, dA=P << 6, dB=P << 7):
    return lib.gemm_adapters_backward(T, N, K, dtype, dY, ldy, X, ldx, W, ldw, major, ad or stack(), plan, dX, lddx, dA, dB, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(ldy=95), "leading"), (dict(ldx=63), "leading"), (dict(lddx=63), "leading"), (dict(dY=0), "dY is NULL"),
    (dict(X=0), "X is NULL"), (dict(plan=0), "plan is NULL"), (dict(dX=P >> 1), "overlap"), (dict(dA=P), "overlap"),
    (dict(dB=(P << 6) + 64), "overlap"), (dict(ad=stack(rank=200)), "128"),
])
def test_adapters_backward_refuses(lib, kw, frag):
    refused(grads(lib, **kw), frag)


def test_adapters_of_nothing(lib):
    assert adapters(lib, T=0) == tg.GEMM_OK and adapters(lib, N=0, ldc=1, ldw=1, ad=stack(ldb=1)) == tg.GEMM_OK
    assert grads(lib, dX=None, dA=None, dB=None) == tg.GEMM_OK


def test_adapter_plans(lib):
    words = lib.gemm_adapter_plan_words
    assert words(0, 1, 0) == 0 and words(-1, 1, 0) == -1 and words(1, 0, 0) == -1 and words(1, 4097, 0) == -1
    assert words((1 << 23) + 1, 1, 0) == -1 and words(1 << 23, 4096, 1) > 0
    # counts, slots and the tokens' slots, by granules of 16, 128 and 256 tokens
    assert words(5, 3, 0) == 1 + 3 + 5 and words(129, 1000, 0) == 2 + 2 * 128 + 129 and words(600, 8, 0) == 3 + 3 * 8 + 600
    assert words(600, 8, 1) == words(600, 8, 0) + 8 + 8 * 3                  # and each adapter's list
    refused(lib.gemm_adapter_plan(8, 0, P, 0, P << 1, None), "adapters")
    refused(lib.gemm_adapter_plan((1 << 23) + 1, 4, P, 0, P << 1, None), "tokens")
    refused(lib.gemm_adapter_plan(8, 4, 0, 0, P << 1, None), "ids is NULL")
    refused(lib.gemm_adapter_plan(8, 4, P, 0, 0, None), "plan is NULL")
    refused(lib.gemm_adapter_plan(8, 4, P, 0, P + 16, None), "overlap")
    assert lib.gemm_adapter_plan(0, 4, 0, 0, 0, None) == tg.GEMM_OK


# ------------------------------------------------------------------ Python ---
def test_python_refuses_what_is_not_on_a_gpu_or_does_not_fit():
    h, w, y = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(9, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        tg.project_loss(h, w, y)
    with pytest.raises(TypeError, match="bfloat16"):
        tg.project_loss(h.float(), w.float(), y)
    with pytest.raises(TypeError, match="bfloat16"):
        tg.project_loss(h, w.half(), y)
    with pytest.raises(TypeError, match="labels"):
        tg.project_loss(h, w, y.float())
    with pytest.raises(ValueError, match="shapes"):
        tg.project_loss(h, w[:, :7], y)
    with pytest.raises(ValueError, match="shapes"):
        tg.project_loss(h, w, y[:3])
    with pytest.raises(ValueError, match="empty"):
        tg.project_loss(h, w[:0], y)
    with pytest.raises(ValueError, match="rows of its own"):
        tg.project_loss(h[:1].expand(4, 8), w, y)
    with pytest.raises(ValueError, match="not expanded"):
        tg.project_loss(h, w[:1].expand(9, 8), y)
    with pytest.raises(TypeError, match="grad"):
        tg.project_loss_backward(torch.zeros(8)[::2], h, w, y, torch.zeros(4))
    with pytest.raises(TypeError, match="lse"):
        tg.project_loss_backward(torch.zeros(4), h, w, y, torch.zeros(4, dtype=torch.float64))
    x, p = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.bfloat16)
    a, b = torch.zeros(3, 2, 8, dtype=torch.bfloat16), torch.zeros(3, 2, 16, dtype=torch.bfloat16)
    plan = tg.AdapterPlan(4, 3, False, torch.zeros(8, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        tg.gemm_adapters(x, p, a, b, plan)
    with pytest.raises(ValueError, match="CUDA"):
        tg.adapter_plan(torch.zeros(4, dtype=torch.int32), 3)
    with pytest.raises(ValueError, match="1-D"):
        tg.adapter_plan(torch.zeros(4, 1, dtype=torch.int32), 3)
    for bad in (dict(A=a[:2]), dict(B=b[..., :15]), dict(plan=plan._replace(adapters=2)), dict(plan=None), dict(A=a[:1].expand(3, 2, 8)),
                dict(B=b[:, :1].expand(3, 2, 16)), dict(plan=plan._replace(tokens=5)), dict(X=x[:, :7])):
        kw = dict(X=x, W=p, A=a, B=b, plan=plan)
        kw.update(bad)
        with pytest.raises(ValueError):
            tg.gemm_adapters(**kw)
    with pytest.raises(TypeError):
        tg.gemm_adapters(x, p, a.half(), b, plan)
    with pytest.raises(TypeError, match="scales"):
        tg.gemm_adapters(x, p, a, b, plan, scales=torch.zeros(2))
    with pytest.raises(ValueError, match="backward=True"):
        tg.gemm_adapters_backward(torch.zeros(4, 16, dtype=torch.bfloat16), x, p, a, b, plan)


def test_options(lib):
    for key, good, bad in (("product_bn", (128, 256, 0), (64, -1)), ("product_splits", (1, 2, 3, 4, 0), (5, -1)),
                           ("loss_columns", (64, 1024, 0), (63, -64, 1 << 25))):
        for v in good:
            assert tg.gemm_set_option(key, v) == tg.GEMM_OK and tg.gemm_get_option(key) == v
        for v in bad:
            assert tg.gemm_set_option(key, v) == BAD and tg.gemm_get_option(key) == 0


def test_the_series_of_tanh_is_within_a_unit_in_the_last_place():
    # the kernel's coefficients and steps (fused multiply-adds in FP32) against tanh in 64 bits on (0, 1/2]
    import numpy as np
    src = open(os.path.join(ROOT, "tiled_tensor_core_gemm_gb300", "csrc", "project.cu")).read()
    body = src[src.index("void tanh_64("):]
    body = body[:body.index("tanhf")]
    coeffs = [np.float32(np.float32(a) / np.float32(b)) for a, b in re.findall(r"both\((-?\d+)\.f / (\d+)\.f\)", body)]
    assert "most <= 0.5f" in body and len(coeffs) >= 6
    x = np.linspace(2.0 ** -12, 0.5, 200001).astype(np.float32)

    def fma(a, b, c):
        return (a.astype(np.float64) * b + c).astype(np.float32)
    q = x * x
    r = np.full_like(x, coeffs[0])
    for c in coeffs[1:]:
        r = fma(r, q, np.float64(c))
    got = fma(r * q, x, x)
    want = np.tanh(x.astype(np.float64))
    assert float((np.abs(got - want) / np.spacing(want.astype(np.float32))).max()) <= 1.0
