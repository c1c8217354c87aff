"""The products around a language model's weights in bfloat16 or float16 on CUDA
tensors: the loss of the output projection over a vocabulary with its gradients,
and low-rank adapters of many requests beside a shared projection with theirs.

As ops.py's, each function checks shapes and types, allocates its outputs, and
makes one call of the C ABI in include/gemm_project.h (which has the formulas) on
the current stream (or ``stream``, a cudaStream_t as int).  There is no CPU path.

A training step's loss (H: tokens x D, W: V x D, labels: tokens):

    loss, lse = project_loss(H, W, labels)
    n = (labels >= 0).sum()
    dH, dW = project_loss_backward((1 / n).expand(len(labels)), H, W, labels, lse)

A projection with an adapter per token (ids: tokens, -1 for none), and its
gradients:

    plan = adapter_plan(ids, adapters, backward=True)     # once a step, for every layer
    Y = gemm_adapters(X, W, A, B, plan, scales)
    dX, dA, dB = gemm_adapters_backward(dY, X, W, A, B, plan, scales)
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import ops
from .ops import _cuda, _dense, _epilogue, _fail, _rows


class Loss(ctypes.Structure):
    """gemm_loss_t."""
    _fields_ = [("softcap", ctypes.c_float), ("smoothing", ctypes.c_float), ("z_loss", ctypes.c_float)]


class Adapters(ctypes.Structure):
    """gemm_adapters_t."""
    _fields_ = [("count", ctypes.c_int64), ("rank", ctypes.c_int64), ("A", ctypes.c_void_p), ("lda", ctypes.c_int64),
                ("a_stride", ctypes.c_int64), ("B", ctypes.c_void_p), ("ldb", ctypes.c_int64),
                ("b_stride", ctypes.c_int64), ("scales", ctypes.c_void_p)]


class AdapterPlan(NamedTuple):
    """What adapter_plan returns: which tokens take which adapter, as the products read it."""
    tokens: int
    adapters: int
    backward: bool
    data: "torch.Tensor"      # noqa: F821


def declare(lib):
    """The C entries' argument types."""
    i64, i32, p = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    lib.gemm_project_loss.argtypes = [i64, i64, i64, i32, p, i64, p, i64, i32, p, i32, p, p, p, p]
    lib.gemm_project_loss_backward.argtypes = [i64, i64, i64, i32, p, i64, p, i64, p, i64, i32, p, i32, p, p, p, i64, p,
                                               i64, p]
    lib.gemm_adapter_plan_words.argtypes = [i64, i64, i32]
    lib.gemm_adapter_plan.argtypes = [i64, i64, p, i32, p, p]
    lib.gemm_adapters.argtypes = [i64, i64, i64, i32, p, i64, p, i64, i32, p, p, p, i64, p, p]
    lib.gemm_adapters_backward.argtypes = [i64, i64, i64, i32, p, i64, p, i64, p, i64, i32, p, p, p, i64, p, p, p]
    for name in ("gemm_project_loss", "gemm_project_loss_backward", "gemm_adapter_plan", "gemm_adapters",
                 "gemm_adapters_backward"):
        getattr(lib, name).restype = i32
    lib.gemm_adapter_plan_words.restype = i64


_codes = None
_losses = {}


def _tables():
    """ops._tables, and torch's 16-bit types -> the ABI's operand codes and the names of outputs."""
    global _codes
    torch, tg, lib, _, _, outs, raw = ops._tables()
    if _codes is None:
        _codes = {torch.bfloat16: (tg.GEMM_BF16, "bf16"), torch.float16: (tg.GEMM_FP16, "f16")}
    return torch, tg, lib, _codes, outs, raw


def _major(name, t):
    """(pitch, 1 if the first dimension is the contiguous one) of a matrix."""
    rows, cols = t.shape
    sr, sc = t.stride()
    if (sc == 1 or cols <= 1) and (rows <= 1 or sr >= cols):
        return (sr if rows > 1 and cols > 0 else max(cols, 1)), 0
    if (sr == 1 or rows <= 1) and (cols <= 1 or sc >= rows):
        return (sc if cols > 1 and rows > 0 else max(rows, 1)), 1
    raise ValueError(f"{name} must be row-major or the transpose of a row-major matrix, not expanded")


def _how(softcap, smoothing, z_loss):
    key = (softcap, smoothing, z_loss)
    h = _losses.get(key)
    if h is None:
        h = ctypes.byref(Loss(*key))
        if len(_losses) < 256:
            _losses[key] = h
    return h


def _projection(H, W, labels):
    torch, tg, lib, codes, _, raw = _tables()
    if H.dim() != 2 or W.dim() != 2 or labels.dim() != 1:
        raise ValueError("H and W must be 2-D, labels 1-D")
    code = codes.get(H.dtype)
    if code is None or W.dtype is not H.dtype:
        raise TypeError("H and W must both be bfloat16 or both float16")
    if labels.dtype is torch.int64:
        label_bytes = 8
    elif labels.dtype is torch.int32:
        label_bytes = 4
    else:
        raise TypeError("labels must be int64 or int32")
    tokens, dim = H.shape
    vocab = W.shape[0]
    if W.shape[1] != dim or labels.shape[0] != tokens:
        raise ValueError("shapes do not match: H (tokens, dim), W (vocabulary, dim), labels (tokens)")
    if vocab < 1:
        raise ValueError("the vocabulary is empty")
    if not labels.is_contiguous():
        raise TypeError("labels must be contiguous")
    ldh = _rows("H", H, tokens, dim)
    ldw, w_major = _major("W", W)
    return torch, tg, lib, code[0], raw, tokens, vocab, dim, ldh, ldw, w_major, label_bytes


def project_loss(H, W, labels, softcap=0.0, smoothing=0.0, z_loss=0.0, stream=None):
    """(loss, lse): softmax cross entropy of the logits H.W^T, which are never stored.

    H: (T, D), W: (V, D), both bfloat16 or both float16; W row-major or the
    transpose of a row-major (D, V).  labels: (T,) int64 or int32; one outside
    [0, V) (-100, say) marks a token that does not count, whose loss is 0.
    softcap: logits are softcap * tanh(z / softcap) if not 0.  smoothing: the
    part of the target spread over the vocabulary.  z_loss: the factor of lse^2
    added.  Both results are float32 (T,); lse is the log of the sum of
    exponentials, which the backward pass takes.
    """
    torch, tg, lib, code, raw, T, V, D, ldh, ldw, w_major, label_bytes = _projection(H, W, labels)
    index = _cuda(H, W, labels)
    out = torch.empty((2, T), dtype=torch.float32, device=H.device)
    loss, lse = out[0], out[1]
    rc = lib.gemm_project_loss(T, V, D, code, H.data_ptr(), ldh, W.data_ptr(), ldw, w_major, labels.data_ptr(), label_bytes,
                               _how(softcap, smoothing, z_loss), loss.data_ptr(), lse.data_ptr(),
                               raw(index) if stream is None else stream)
    if rc:
        _fail(tg, rc)
    return loss, lse


def project_loss_backward(grad, H, W, labels, lse, softcap=0.0, smoothing=0.0, z_loss=0.0, want_H=True, want_W=True,
                          stream=None):
    """(dH, dW) of project_loss from grad, the gradient of its losses.

    grad: (T,) float32, or one value expanded over the tokens.  The other
    arguments as given to project_loss, lse as it returned it.  dH is (T, D) and
    dW (V, D) in the layout of W, both in H's type; None for one that is not
    wanted.  A token that does not count adds nothing, whatever its row of H
    and its grad hold.
    """
    torch, tg, lib, code, raw, T, V, D, ldh, ldw, w_major, label_bytes = _projection(H, W, labels)
    if grad.dtype is not torch.float32 or grad.shape != (T,) or (T > 1 and grad.stride(0) not in (0, 1)):
        raise TypeError(f"grad must be a contiguous ({T},) float32 tensor or one value expanded")
    _dense("lse", lse, (T,), torch.float32)
    index = _cuda(H, W, labels, grad, lse)
    dH = torch.empty((T, D), dtype=H.dtype, device=H.device) if want_H else None
    dW = None
    if want_W:
        dW = torch.empty((D, V) if w_major else (V, D), dtype=H.dtype, device=H.device)
    rc = lib.gemm_project_loss_backward(T, V, D, code, grad.data_ptr(), grad.stride(0) if T > 1 else 1, H.data_ptr(), ldh,
                                        W.data_ptr(), ldw, w_major, labels.data_ptr(), label_bytes,
                                        _how(softcap, smoothing, z_loss), lse.data_ptr(),
                                        dH.data_ptr() if want_H else None, D or 1, dW.data_ptr() if want_W else None,
                                        (V if w_major else D) or 1, raw(index) if stream is None else stream)
    if rc:
        _fail(tg, rc)
    return dH, dW.t() if want_W and w_major else dW


def adapter_plan(ids, adapters, backward=False, stream=None) -> AdapterPlan:
    """Which tokens take which adapter, for gemm_adapters (and, with backward, its gradients).

    ids: (T,) int32; values outside [0, adapters) take none.  Tokens may come in
    any order, but many of them cost least sorted by adapter (8192 tokens over 64
    adapters of rank 64 beside 4096 x 4096: 200 us sorted, 640 in random order, and
    320 and 1960 for the gradients): neighbours share the products of their adapters.
    The plan holds for every projection of a step with these tokens.
    """
    torch, tg, lib, _, _, raw = _tables()
    if ids.dim() != 1:
        raise ValueError("ids must be 1-D")
    tokens = ids.shape[0]
    index = _cuda(ids)
    _dense("ids", ids, (tokens,), torch.int32)
    words = lib.gemm_adapter_plan_words(tokens, adapters, backward)
    if words < 0:
        raise ValueError("at most 2^23 tokens and between 1 and 4096 adapters")
    data = torch.empty(words, dtype=torch.int32, device=ids.device)
    rc = lib.gemm_adapter_plan(tokens, adapters, ids.data_ptr(), backward, data.data_ptr(),
                               raw(index) if stream is None else stream)
    if rc:
        _fail(tg, rc)
    return AdapterPlan(tokens, adapters, bool(backward), data)


def _adapted(X, W, A, B, plan, scales):
    """Checks what both directions share; (torch, tg, lib, code, type name, raw, N, K, ldw, w_major, Adapters)."""
    torch, tg, lib, codes, _, raw = _tables()
    if X.dim() != 2 or W.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        raise ValueError("activations and W must be 2-D, A and B 3-D")
    dt = X.dtype
    code = codes.get(dt)
    if code is None or W.dtype is not dt or A.dtype is not dt or B.dtype is not dt:
        raise TypeError("activations, W, A and B must all be bfloat16 or all float16")
    k, n = W.shape
    count, rank = A.shape[:2]
    if A.shape[2] != k or B.shape != (count, rank, n):
        raise ValueError("shapes do not match: W (K, N), A (adapters, rank, K), B (adapters, rank, N)")
    if not isinstance(plan, AdapterPlan) or plan.adapters != count:
        raise ValueError("plan must be adapter_plan's for these adapters")
    if scales is not None:
        _dense("scales", scales, (count,), torch.float32)
    ldw, w_major = _major("W", W)
    lds = []
    for name, t in (("A", A), ("B", B)):
        sl, sr, sc = t.stride()
        cols = t.shape[2]
        if cols > 1 and sc != 1:
            raise ValueError(f"{name} must have unit stride along its columns")
        if (rank > 1 and sr < cols) or (count > 1 and sl < cols):
            raise ValueError(f"{name} must have rows and matrices of its own (it is expanded)")
        lds += [sr if rank > 1 and cols > 0 else max(cols, 1), sl if count > 1 else 0]
    ad = Adapters(count, rank, A.data_ptr(), lds[0], lds[1], B.data_ptr(), lds[2], lds[3],
                  scales.data_ptr() if scales is not None else None)
    return torch, tg, lib, code, raw, n, k, ldw, w_major, ad


def gemm_adapters(X, W, A, B, plan, scales=None, C=None, bias=None, act="none", out=None, stream=None):
    """C[t] = act(X[t].W + scales[i] (X[t].A_i^T).B_i + bias), i the adapter of token t.

    X: (T, K); W: (K, N), row-major or the transpose of a row-major matrix; A:
    (L, rank, K) and B: (L, rank, N) with unit stride along their columns; all
    bfloat16 or all float16.  W's, A's and B's addresses and pitches are
    multiples of 16 bytes; rank is at most 128.  plan: adapter_plan's for the T
    tokens and L adapters.  scales: (L,) float32 or None (ones).  bias: N
    float32 values or None; act: "none", "relu" or "gelu"; out: C's type ("f32",
    "bf16" or "f16"; X's by default).  Adapters must be finite.
    """
    torch, tg, lib, code, raw, n, k, ldw, w_major, ad = _adapted(X, W, A, B, plan, scales)
    tokens = X.shape[0]
    if X.shape[1] != k:
        raise ValueError("inner dimensions differ")
    if plan.tokens != tokens:
        raise ValueError(f"plan is for {plan.tokens} tokens")
    index = _cuda(X, W, A, B, plan.data, scales, C, bias)
    if out is None:
        out = code[1]
    cdt = _tables()[4][out]
    if C is None:
        C = torch.empty((tokens, n), dtype=cdt, device=X.device)
        ldc = n or 1
    elif C.dtype is not cdt or C.shape != (tokens, n):
        raise TypeError(f"C must be a ({tokens}, {n}) {cdt} tensor")
    else:
        ldc = _rows("C", C, tokens, n)
    if bias is not None:
        _dense("bias", bias, (n,), torch.float32)
    rc = lib.gemm_adapters(tokens, n, k, code[0], X.data_ptr(), _rows("X", X, tokens, k), W.data_ptr(), ldw, w_major,
                           ctypes.byref(ad), plan.data.data_ptr(), C.data_ptr(), ldc,
                           _epilogue(tg, 1.0, 0.0, bias, act, out), raw(index) if stream is None else stream)
    if rc:
        _fail(tg, rc)
    return C


def gemm_adapters_backward(dY, X, W, A, B, plan, scales=None, want_X=True, want_adapters=True, stream=None):
    """(dX, dA, dB) of gemm_adapters without bias and activation, W frozen.

    dY: (T, N), the gradient of X.W + ...; the other arguments as given to
    gemm_adapters, the plan made with backward=True.  dX is (T, K), dA (L, rank,
    K), dB (L, rank, N), zero for an adapter without tokens, all in X's type;
    None for what is not wanted.  Every row of X and dY must be finite, padding
    included, where dA and dB are wanted: a token adds a zero multiple of its row
    to its neighbours' adapters.
    """
    torch, tg, lib, code, raw, n, k, ldw, w_major, ad = _adapted(X, W, A, B, plan, scales)
    tokens = X.shape[0]
    if X.shape[1] != k or dY.shape != (tokens, n) or dY.dtype is not X.dtype:
        raise ValueError(f"X must be (tokens, {k}) and dY (tokens, {n}), of one type")
    if plan.tokens != tokens or not plan.backward:
        raise ValueError(f"plan must be made with backward=True for {tokens} tokens")
    index = _cuda(X, dY, W, A, B, plan.data, scales)
    dX = torch.empty((tokens, k), dtype=X.dtype, device=X.device) if want_X else None
    dA = torch.empty(A.shape, dtype=X.dtype, device=X.device) if want_adapters else None
    dB = torch.empty(B.shape, dtype=X.dtype, device=X.device) if want_adapters else None
    rc = lib.gemm_adapters_backward(tokens, n, k, code[0], dY.data_ptr(), _rows("dY", dY, tokens, n), X.data_ptr(),
                                    _rows("X", X, tokens, k), W.data_ptr(), ldw, w_major, ctypes.byref(ad),
                                    plan.data.data_ptr(), dX.data_ptr() if want_X else None, k or 1,
                                    dA.data_ptr() if want_adapters else None, dB.data_ptr() if want_adapters else None,
                                    raw(index) if stream is None else stream)
    if rc:
        _fail(tg, rc)
    return dX, dA, dB
