"""The operators of an expert layer on CUDA tensors: FP8 matrices with a scale
for each block of 128 and their products, the routing of tokens to experts and
the weighted combination of the experts' rows.

Each function checks shapes and types, allocates the outputs it is not given,
and makes one call of the C ABI in include/gemm_ops.h (which has the formulas);
every step of the computation runs in the library's CUDA kernels on the current
stream (or ``stream``, a cudaStream_t as int).  There is no CPU path.  Inputs
that are read row by row (x, logits, Y, grad) may be one row expanded over all;
operands of a product and outputs may not (ValueError).

A dense layer Y = X W^T (X: tokens x K, W: N x K) and its gradients, every
operand read as it was stored:

    xq, xs = quantize_block(X, "row");    wq, ws = quantize_block(W, "tile")
    Y  = gemm_scaled(xq, xs, wq.t(), ws.t(), out="bf16")
    gq, gs = quantize_block(dY, "row")
    dX = gemm_scaled(gq, gs, wq, ws, out="bf16")
    xc, xcs = quantize_block(X, "col");   gc, gcs = quantize_block(dY, "col")
    dW = gemm_scaled(gc.t(), gcs.t(), xc, xcs)

An expert layer with weights W1 (E x N x K) and W2 (E x K x N), quantised once:

    r = route(logits, top_k=8)
    xq, xs = quantize_block(X, "row", scatter=r.slots)
    h = gemm_experts(xq, xs, w1q.transpose(1, 2), w1s.transpose(1, 2), r.offsets, act="gelu", out="bf16")
    hq, hs = quantize_block(h, "row")
    y = gemm_experts(hq, hs, w2q.transpose(1, 2), w2s.transpose(1, 2), r.offsets, out="bf16")
    out = combine(y, r.slots, r.weights)
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

BLOCK = 128
_BLOCKS = {"row": 0, "col": 1, "tile": 2}
_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}


class BlockScale(ctypes.Structure):
    """gemm_block_scale_t."""
    _fields_ = [("scale", ctypes.c_void_p), ("stride_k", ctypes.c_int64), ("stride_i", ctypes.c_int64),
                ("block", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class RouteHow(ctypes.Structure):
    """gemm_route_t."""
    _fields_ = [("top_k", ctypes.c_int32), ("score", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("group_score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class Routing(NamedTuple):
    """What route returns; every array is on the logits' device.

    indices  (T, top_k) int32: the chosen experts, best first; -1 where none was left
    weights  (T, top_k) float32
    offsets  (E + 1) int32: expert e has rows offsets[e] .. offsets[e + 1]
    order    (T * top_k) int32: row -> pair t * top_k + j; -1 past the last row
    slots    (T, top_k) int32: pair -> row, -1 without an expert
    """
    indices: "torch.Tensor"   # noqa: F821
    weights: "torch.Tensor"   # noqa: F821
    offsets: "torch.Tensor"   # noqa: F821
    order: "torch.Tensor"     # noqa: F821
    slots: "torch.Tensor"     # noqa: F821


def declare(lib):
    """The C entries' argument types."""
    i64, i32, p, f = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_float
    bs, ep = ctypes.POINTER(BlockScale), p
    lib.gemm_quantize_block.argtypes = [i64, i64, i64, i32, p, i64, i64, i32, i32, p, i64, i64, p, i64, i64, i64, p,
                                        i64, i64, p]
    lib.gemm_run_scaled.argtypes = [i64, i64, i64, i32, p, i64, i32, bs, p, i64, i32, bs, p, i64, ep, p]
    lib.gemm_run_experts.argtypes = [i64, i64, i64, i64, i32, p, i64, bs, p, p, i64, i64, i32, bs, i64, p, i64, ep, p]
    lib.gemm_route.argtypes = [i64, i64, i32, p, i64, p, ctypes.POINTER(RouteHow), p, p, p, p, p, p]
    lib.gemm_route_backward.argtypes = [i64, i64, i32, p, i64, ctypes.POINTER(RouteHow), p, p, p, i64, p]
    lib.gemm_combine.argtypes = [i64, i64, i64, i64, i32, p, i64, p, p, p, i64, p]
    lib.gemm_combine_backward.argtypes = [i64, i64, i64, i64, i32, p, i64, p, i64, p, p, p, p, i64, p, p]
    for name in ("gemm_quantize_block", "gemm_run_scaled", "gemm_run_experts", "gemm_route", "gemm_route_backward",
                 "gemm_combine", "gemm_combine_backward"):
        getattr(lib, name).restype = i32


# ----------------------------------------------------------------- helpers ---
# A decode step calls these operators for microseconds of GPU work each, so the
# marshalling is kept short: integer device indices, the raw stream, and argument
# structures that depend on scalars only are built once.
_types = None
_epilogues = {}
_hows = {}


def _tables():
    """(torch, the package, the library, torch element types -> the ABI's codes, ...)"""
    global _types
    if _types is None:
        import torch
        import tiled_tensor_core_gemm_gb300 as tg
        _types = (torch, tg, tg.load_library(),
                  {torch.float32: tg.GEMM_OUT_F32, torch.bfloat16: tg.GEMM_OUT_BF16, torch.float16: tg.GEMM_OUT_F16},
                  {torch.float8_e4m3fn: tg.GEMM_E4M3, torch.float8_e5m2: tg.GEMM_E5M2},
                  {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16},
                  torch._C._cuda_getCurrentRawStream)
    return _types


def _fail(tg, rc):
    raise tg.GemmError(rc, tg.gemm_last_error())


def _cuda(first, *others):
    """The CUDA device index every tensor given (None entries skipped) is on."""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must be CUDA tensors (this library has no CPU path)")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on different devices: {first.device} and {t.device}")
    return index


def _rows(name, t, rows, cols, shared=False):
    """Row pitch of a rows x cols tensor with unit stride along its columns.

    shared: the operator reads row by row, so that the rows may be one row's
    memory (a row expanded, as autograd hands back the gradient of a sum over
    them); the pitch is then 0.  Matrices that are written or read by TMA may not.
    """
    sr, sc = t.stride()
    if cols > 1 and sc != 1:
        raise ValueError(f"{name} must have unit stride along its columns")
    if rows <= 1 or cols == 0:
        return cols or 1
    if sr == 0 and not shared:
        raise ValueError(f"{name} must have rows of its own (it is one row expanded)")
    return sr


def _dense(name, t, shape, dtype):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor")


def _major(name, t):
    """(pitch, 1 if the last-but-one dimension is contiguous) of a matrix, or of each of a batch."""
    rows, cols = t.shape[-2:]
    sr, sc = t.stride()[-2:]
    if sc == 1 or cols <= 1:
        if rows <= 1 or cols == 0:
            return max(cols, 1), 0
        if sc == 1 and sr >= cols:
            return sr, 0
        if cols == 1 and sr > 1:
            return sr, 0
    if sr == 1 or rows <= 1:
        if cols <= 1 or rows == 0:
            return max(rows, 1), 1
        if sc >= rows:
            return sc, 1
    raise ValueError(f"{name} must be row-major or the transpose of a row-major matrix, not expanded")


def _scale(name, s, f32, extent, num_kb, k_dim, tiles_ok):
    """A BlockScale over a 2-D (or batched) scale tensor; k_dim: its dimension along K (-1 or -2)."""
    if s.dtype is not f32:
        raise TypeError(f"{name} must be float32")
    shape, stride = s.shape, s.stride()
    n, kb = shape[-3 - k_dim], shape[k_dim]
    if kb == num_kb and n == extent:
        block = 1
    elif kb == num_kb and tiles_ok and n == -(-extent // BLOCK):
        block = BLOCK
    else:
        raise ValueError(f"{name}: {tuple(shape)} is not a scale for each block of 128 along K, for each row or "
                         f"column{' or 128 of them' if tiles_ok else ''} (extent {extent}, {num_kb} blocks)")
    # (a dimension of one element has no stride)
    return BlockScale(s.data_ptr(), stride[k_dim] if kb > 1 else 0, stride[-3 - k_dim] if n > 1 else 0, block, 0)


def _epilogue(tg, alpha, beta, bias, act, out):
    if bias is not None:
        return ctypes.byref(tg.GemmEpilogue(alpha, beta, bias.data_ptr(), tg.ACTIVATIONS[act], tg.OUT_TYPES[out]))
    key = (alpha, beta, act, out)
    e = _epilogues.get(key)
    if e is None:
        e = ctypes.byref(tg.GemmEpilogue(alpha, beta, None, tg.ACTIVATIONS[act], tg.OUT_TYPES[out]))
        if len(_epilogues) < 256:
            _epilogues[key] = e
    return e


# --------------------------------------------------------------- operators ---
def quantize_block(x, block="row", dtype="e4m3", scatter=None, out_rows=None, stream=None):
    """FP8 values and scales of x, one scale for each block of 128.

    x: (M, N) or a batch (B, M, N) of float32, bfloat16 or float16 with unit
    stride along N.  block: "row" (1 x 128), "col" (128 x 1) or "tile"
    (128 x 128).  dtype: "e4m3" or "e5m2".

    Returns (q, scale): q like x in FP8, its rows padded to 16 bytes in memory;
    scale float32 (M, ceil(N/128)), (ceil(M/128), N) or (ceil(M/128),
    ceil(N/128)), batched like x.  Row scales lie with the rows of one block
    side by side (the transpose of a contiguous array), as the products read
    them.  q * scale stands for x.

    scatter: an int32 (M, copies) tensor; row m then goes to rows scatter[m] of
    the outputs, which have out_rows rows (M * copies by default); entries
    outside [0, out_rows) are skipped, and rows no entry names hold nothing
    defined.
    """
    torch, tg, lib, types, _, _, raw = _tables()
    dims = x.dim()
    if dims != 2 and dims != 3:
        raise ValueError("x must be a matrix or a batch of matrices")
    kind = types.get(x.dtype)
    if kind is None:
        raise TypeError("x must be float32, bfloat16 or float16")
    code = _BLOCKS[block]
    if dtype == "e4m3":
        to, qdt = tg.GEMM_E4M3, torch.float8_e4m3fn
    elif dtype == "e5m2":
        to, qdt = tg.GEMM_E5M2, torch.float8_e5m2
    else:
        raise TypeError("dtype must be e4m3 or e5m2")
    index = _cuda(x, scatter)
    shape, stride = x.shape, x.stride()
    m, n = shape[-2], shape[-1]
    batch = shape[0] if dims == 3 else 1
    if n > 1 and stride[-1] != 1:
        raise ValueError("x must have unit stride along its columns")
    ldx = stride[-2] if m > 1 and n > 0 else n or 1     # (0: one row expanded, which is read as it is)
    rows, copies, slots = m, 1, None
    if scatter is not None:
        if dims != 2 or code != 0:
            raise ValueError("scatter takes one matrix and row blocks")
        if scatter.dim() != 2 or scatter.shape[0] != m:
            raise ValueError("scatter must have a row for each row of x")
        copies = scatter.shape[1]
        _dense("scatter", scatter, (m, copies), torch.int32)
        rows, slots = (m * copies if out_rows is None else int(out_rows)), scatter.data_ptr()
    elif out_rows is not None:
        raise ValueError("out_rows goes with scatter")
    pitch = -(-n // 16) * 16
    mb = rows if code == 0 else -(-m // BLOCK)
    nb = n if code == 1 else -(-n // BLOCK)
    device = x.device
    # (one allocation each, with the strides they are to have)
    if code == 0:
        held = -(-mb // 4) * 4
        s_row, s_col, s_batch = 1, held or 1, nb * held
    else:
        s_row, s_col, s_batch = nb, 1, mb * nb
    if dims == 2:
        q = torch.empty_strided((rows, n), (pitch or 1, 1), dtype=qdt, device=device)
        s = torch.empty_strided((mb, nb), (s_row, s_col), dtype=torch.float32, device=device)
    else:
        q = torch.empty_strided((batch, rows, n), (rows * pitch, pitch or 1, 1), dtype=qdt, device=device)
        s = torch.empty_strided((batch, mb, nb), (s_batch, s_row, s_col), dtype=torch.float32, device=device)
    if copies == 0 or (scatter is not None and rows == 0):
        return q, s
    rc = lib.gemm_quantize_block(batch, m, n, kind, x.data_ptr(), ldx, stride[0] if batch > 1 else 0, code, to,
                                 q.data_ptr(), pitch or 1, rows * pitch, s.data_ptr(), s_row, s_col, s_batch, slots, copies, rows,
                                 raw(index) if stream is None else stream)
    if rc:
        _fail(tg, rc)
    return q, s


def gemm_scaled(A, a_scale, B, b_scale, C=None, alpha=1.0, beta=0.0, bias=None, act="none", out="f32", stream=None):
    """C = act(alpha * A.B + beta * C + bias) of FP8 matrices under their block scales.

    A: (M, K), B: (K, N), both float8_e4m3fn or both float8_e5m2, each row-major
    or the transpose of a row-major matrix.  a_scale: float32 (M, ceil(K/128))
    or (ceil(M/128), ceil(K/128)); b_scale: (ceil(K/128), N) or (ceil(K/128),
    ceil(N/128)); any strides.  out: C's type, "f32", "bf16" or "f16"
    (allocated if None; beta must then be 0).  bias: N float32 values or None.
    The activations keep a NaN.
    """
    torch, tg, lib, _, fp8, outs, raw = _tables()
    if A.dim() != 2 or B.dim() != 2 or a_scale.dim() != 2 or b_scale.dim() != 2:
        raise ValueError("operands and scales must be 2-D")
    code = fp8.get(A.dtype)
    if code is None or B.dtype is not A.dtype:
        raise TypeError("A and B must both be float8_e4m3fn or both float8_e5m2")
    m, k = A.shape
    k2, n = B.shape
    if k != k2:
        raise ValueError("inner dimensions differ")
    index = _cuda(A, B, a_scale, b_scale, C, bias)
    num_kb = -(-k // BLOCK)
    lda, a_major = _major("A", A)
    ldb, b_major = _major("B", B)
    sa = _scale("a_scale", a_scale, torch.float32, m, num_kb, -1, True)
    sb = _scale("b_scale", b_scale, torch.float32, n, num_kb, -2, True)
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = torch.empty((m, n), dtype=outs[out], device=A.device)
        ldc = n or 1
    elif C.dtype is not outs[out] or C.shape != (m, n):
        raise TypeError(f"C must be a ({m}, {n}) {outs[out]} tensor")
    else:
        ldc = _rows("C", C, m, n)
    if bias is not None:
        _dense("bias", bias, (n,), torch.float32)
    rc = lib.gemm_run_scaled(m, n, k, code, A.data_ptr(), lda, a_major, ctypes.byref(sa), B.data_ptr(), ldb, b_major,
                             ctypes.byref(sb), C.data_ptr(), ldc, _epilogue(tg, alpha, beta, bias, act, out),
                             raw(index) if stream is None else stream)
    if rc:
        _fail(tg, rc)
    return C


def gemm_experts(A, a_scale, W, w_scale, offsets, C=None, alpha=1.0, act="none", out="f32", stream=None):
    """Rows offsets[e] .. offsets[e + 1] of C = act(alpha * A . W[e]) for every expert e.

    A: (R, K) FP8 row-major, rows in expert order; a_scale: float32 (R,
    ceil(K/128)).  W: (E, K, N) FP8, each matrix row-major or the transpose of
    one (weights held as (E, N, K): pass W.transpose(1, 2)), addresses and
    pitches multiples of 16 bytes; w_scale: (E, ceil(K/128), ceil(N/128)) or
    (E, ceil(K/128), N).  offsets: (E + 1) int32 on the device, ascending.
    Rows outside every expert keep what C holds (undefined if C is None).
    """
    torch, tg, lib, _, fp8, outs, raw = _tables()
    if A.dim() != 2 or W.dim() != 3 or a_scale.dim() != 2 or w_scale.dim() != 3:
        raise ValueError("A and a_scale must be 2-D, W and w_scale 3-D")
    code = fp8.get(A.dtype)
    if code is None or W.dtype is not A.dtype:
        raise TypeError("A and W must both be float8_e4m3fn or both float8_e5m2")
    rows, k = A.shape
    experts, k2, n = W.shape
    if k != k2 or w_scale.shape[0] != experts:
        raise ValueError("shapes do not match")
    index = _cuda(A, W, a_scale, w_scale, offsets, C)
    _dense("offsets", offsets, (experts + 1,), torch.int32)
    num_kb = -(-k // BLOCK)
    lda = _rows("A", A, rows, k)
    ldb, b_major = _major("W", W)
    sa = _scale("a_scale", a_scale, torch.float32, rows, num_kb, -1, False)
    sw = _scale("w_scale", w_scale, torch.float32, n, num_kb, -2, True)
    if C is None:
        C = torch.empty((rows, n), dtype=outs[out], device=A.device)
        ldc = n or 1
    elif C.dtype is not outs[out] or C.shape != (rows, n):
        raise TypeError(f"C must be a ({rows}, {n}) {outs[out]} tensor")
    else:
        ldc = _rows("C", C, rows, n)
    rc = lib.gemm_run_experts(rows, n, k, experts, code, A.data_ptr(), lda, ctypes.byref(sa), offsets.data_ptr(),
                              W.data_ptr(), ldb, W.stride(0) if experts > 1 else 0, b_major, ctypes.byref(sw),
                              w_scale.stride(0) if experts > 1 else 0, C.data_ptr(), ldc,
                              _epilogue(tg, alpha, 0.0, None, act, out), raw(index) if stream is None else stream)
    if rc:
        _fail(tg, rc)
    return C


def _how(*rules):
    """A reference to the RouteHow of (top_k, score, groups, top_groups, group_score, renormalize, scale)."""
    h = _hows.get(rules)
    if h is None:
        top_k, score, groups, top_groups, group_score, renormalize, scale = rules
        h = ctypes.byref(RouteHow(top_k, _SCORES[score], groups, groups if top_groups is None else top_groups,
                                  _GROUP_SCORES[group_score], 1 if renormalize else 0, scale))
        if len(_hows) < 256:
            _hows[rules] = h
    return h


def route(logits, top_k, score="softmax", bias=None, groups=1, top_groups=None, group_score="max", renormalize=True,
          scale=1.0, stream=None) -> Routing:
    """Routes tokens to experts and orders the (token, choice) pairs by expert.

    logits: (T, E) float32, bfloat16 or float16.  Experts are ranked by
    score(logits) + bias (by the logits without a bias), with groups among the
    top_groups groups with the largest "max" or "top2" sum; ties go to the
    lower index.  Weights are the chosen experts' scores (without the bias),
    divided by their sum if renormalize, times scale.  A logit of -inf or NaN
    masks its expert.  The full rules are gemm_route's in include/gemm_ops.h.
    """
    torch, tg, lib, types, _, _, raw = _tables()
    kind = types.get(logits.dtype)
    if kind is None or logits.dim() != 2:
        raise TypeError("logits must be a (tokens, experts) float32, bfloat16 or float16 tensor")
    tokens, experts = logits.shape
    index = _cuda(logits, bias)
    if bias is not None:
        _dense("bias", bias, (experts,), torch.float32)
    how = _how(top_k, score, groups, top_groups, group_score, renormalize, scale)
    device, i32, empty = logits.device, torch.int32, torch.empty
    shape = (tokens, top_k)
    indices, slots = empty(shape, dtype=i32, device=device), empty(shape, dtype=i32, device=device)
    weights = empty(shape, dtype=torch.float32, device=device)
    order = empty(tokens * top_k, dtype=i32, device=device)
    offsets = empty(experts + 1, dtype=i32, device=device)
    rc = lib.gemm_route(tokens, experts, kind, logits.data_ptr(), _rows("logits", logits, tokens, experts, True),
                        bias.data_ptr() if bias is not None else None, how, indices.data_ptr(), weights.data_ptr(),
                        offsets.data_ptr(), order.data_ptr(), slots.data_ptr(), raw(index) if stream is None else stream)
    if rc:
        _fail(tg, rc)
    return Routing(indices, weights, offsets, order, slots)


def route_backward(grad_weights, logits, indices, score="softmax", renormalize=True, scale=1.0, stream=None):
    """The logits' gradient (in their type) from the gradient of route's weights.

    grad_weights: (T, top_k) float32; logits, score, renormalize and scale as
    given to route; indices as it returned them.
    """
    torch, tg, lib, types, _, _, raw = _tables()
    kind = types.get(logits.dtype)
    if kind is None or logits.dim() != 2:
        raise TypeError("logits must be a (tokens, experts) float32, bfloat16 or float16 tensor")
    if indices.dim() != 2:
        raise ValueError("indices must be (tokens, top_k)")
    tokens, experts = logits.shape
    shape = (tokens, indices.shape[1])
    index = _cuda(logits, indices, grad_weights)
    _dense("indices", indices, shape, torch.int32)
    _dense("grad_weights", grad_weights, shape, torch.float32)
    out = torch.empty((tokens, experts), dtype=logits.dtype, device=logits.device)
    rc = lib.gemm_route_backward(tokens, experts, kind, logits.data_ptr(), _rows("logits", logits, tokens, experts, True),
                                 _how(shape[1], score, 1, 1, "max", renormalize, scale), indices.data_ptr(),
                                 grad_weights.data_ptr(), out.data_ptr(), experts or 1,
                                 raw(index) if stream is None else stream)
    if rc:
        _fail(tg, rc)
    return out


def combine(Y, slots, weights: Optional["torch.Tensor"] = None, out=None, stream=None):   # noqa: F821
    """out[t] = sum_j weights[t, j] * Y[slots[t, j]], summed in float32 in the order of j.

    Y: (R, H) float32, bfloat16 or float16; slots: (T, top_k) int32, entries
    outside [0, R) add nothing; weights: (T, top_k) float32, or None for ones
    (the gradient of quantize_block's scatter of each token to its rows).
    """
    torch, tg, lib, types, _, _, raw = _tables()
    kind = types.get(Y.dtype)
    if kind is None or Y.dim() != 2:
        raise TypeError("Y must be a 2-D float32, bfloat16 or float16 tensor")
    if slots.dim() != 2:
        raise ValueError("slots must be (tokens, top_k)")
    shape = slots.shape
    tokens, top_k = shape
    rows, hidden = Y.shape
    index = _cuda(Y, slots, weights, out)
    _dense("slots", slots, shape, torch.int32)
    if weights is not None:
        _dense("weights", weights, shape, torch.float32)
    if out is None:
        out = torch.empty((tokens, hidden), dtype=Y.dtype, device=Y.device)
        ldo = hidden or 1
    elif out.dtype is not Y.dtype or out.shape != (tokens, hidden):
        raise TypeError(f"out must be a ({tokens}, {hidden}) {Y.dtype} tensor")
    else:
        ldo = _rows("out", out, tokens, hidden)
    rc = lib.gemm_combine(tokens, top_k, hidden, rows, kind, Y.data_ptr(), _rows("Y", Y, rows, hidden, True),
                          slots.data_ptr(), weights.data_ptr() if weights is not None else None, out.data_ptr(), ldo,
                          raw(index) if stream is None else stream)
    if rc:
        _fail(tg, rc)
    return out


def combine_backward(grad, Y, slots, weights, order=None, stream=None):
    """(dY, dweights) of combine from grad, the gradient of its output.

    dY[slots[t, j]] = weights[t, j] * grad[t] and dweights[t, j] =
    <grad[t], Y[slots[t, j]]>.  order: route's; with it the rows past the last
    get a zero gradient.  Without it rows that no slot names are zeroed too (by
    an extra pass over dY).  The entries of slots are distinct.
    """
    torch, tg, lib, types, _, _, raw = _tables()
    kind = types.get(Y.dtype)
    if kind is None or Y.dim() != 2 or grad.dtype is not Y.dtype:
        raise TypeError("grad and Y must be 2-D tensors of one type: float32, bfloat16 or float16")
    if slots.dim() != 2:
        raise ValueError("slots must be (tokens, top_k)")
    shape = slots.shape
    tokens, top_k = shape
    rows, hidden = Y.shape
    if grad.shape != (tokens, hidden):
        raise ValueError(f"grad must be ({tokens}, {hidden})")
    index = _cuda(Y, grad, slots, weights, order)
    _dense("slots", slots, shape, torch.int32)
    _dense("weights", weights, shape, torch.float32)
    if order is not None:
        _dense("order", order, (tokens * top_k,), torch.int32)
        if rows != tokens * top_k:
            raise ValueError("order goes with tokens * top_k rows")
    if order is not None:
        dY = torch.empty((rows, hidden), dtype=Y.dtype, device=Y.device)
    elif stream is None:
        dY = torch.zeros((rows, hidden), dtype=Y.dtype, device=Y.device)
    else:
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=Y.device)):
            dY = torch.zeros((rows, hidden), dtype=Y.dtype, device=Y.device)
    dw = torch.empty(shape, dtype=torch.float32, device=Y.device)
    rc = lib.gemm_combine_backward(tokens, top_k, hidden, rows, kind, grad.data_ptr(),
                                   _rows("grad", grad, tokens, hidden, True), Y.data_ptr(), _rows("Y", Y, rows, hidden, True),
                                   slots.data_ptr(), weights.data_ptr(), order.data_ptr() if order is not None else None,
                                   dY.data_ptr(), hidden or 1, dw.data_ptr(), raw(index) if stream is None else stream)
    if rc:
        _fail(tg, rc)
    return dY, dw
