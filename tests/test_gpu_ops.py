"""The expert-layer operators on the GPU, each against its definition in 64 bits.

Bounds (stated before any run):

* Products: |C - C_ref| <= 1e-5 * D, D the same sum over absolute values (the
  library's gate for FP8 inputs).  A K-block of 128 takes four accumulations in
  Tensor Memory, each within 2^-22 of its terms' magnitude, then three FP32
  roundings for the scales and the sum; up to 64 blocks add 64 * 2^-24 more:
  under 6e-6.  The epilogue multiplies that by its slope (GELU 1.13) and adds
  2^-22 of its own magnitude; a 16-bit output half a unit in the last place.
* Quantisation is elementwise IEEE arithmetic and a rounding: equal to the same
  steps on the CPU, bit for bit.
* Routing: whole numbers equal.  Weights: expf within 2 units in the last
  place, a sum of E <= 1024 terms in 32 chains (at most 32 + 5 additions), three
  divisions and a product: under 48 * 2^-24 relative.
* Combination: FP32 sums of k terms: (k + 1) * 2^-24 of the sum of magnitudes,
  and half a unit of the output type; its dots run at most hidden / 8 / threads
  chains of 8, then 13 additions: under 64 * 2^-24 of the sum of magnitudes for
  hidden <= 8192.
"""
import math

import pytest
import torch

import tiled_tensor_core_gemm_gb300 as tg
from tiled_tensor_core_gemm_gb300 import build as tgbuild

pytestmark = pytest.mark.gpu

FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
OUT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
GUARD = 64


@pytest.fixture(scope="module", autouse=True)
def lib():
    tgbuild.build()
    return tg.load_library()


@pytest.fixture(autouse=True)
def status_is_clean():
    yield
    s = torch.cuda.current_stream().cuda_stream
    assert tg.gemm_get_status(s) == tg.GEMM_OK, tg.gemm_last_error()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(*shape, seed=0, dtype=torch.float32):
    return torch.randn(shape, generator=gen(seed), device="cuda").to(dtype)


def cdiv(a, b):
    return -(-a // b)


# ---------------------------------------------------------------- quantise ---
def expect_quantized(x, block, to):
    """The same IEEE steps on the CPU."""
    dt, top = FP8[to]
    x = x.cpu().float()
    m, n = x.shape[-2:]
    bm, bn = (1 if block == "row" else 128), (1 if block == "col" else 128)
    mb, nb = cdiv(m, bm), cdiv(n, bn)
    pad = torch.zeros(x.shape[:-2] + (mb * bm, nb * bn))
    pad[..., :m, :n] = x
    v = pad.view(x.shape[:-2] + (mb, bm, nb, bn))
    big = torch.where(v.isnan(), torch.zeros(()), v.abs()).amax(dim=(-3, -1))
    s = torch.maximum(big / torch.full((), top), torch.full((), 2.0 ** -126))
    q = (v * (torch.ones(()) / s)[..., :, None, :, None]).to(dt)
    return q.view(pad.shape)[..., :m, :n], s


def same_bits(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))


@pytest.mark.parametrize("to", ("e4m3", "e5m2"))
@pytest.mark.parametrize("block", ("row", "col", "tile"))
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 1), (1, 128), (3, 129), (128, 128), (130, 1000), (257, 77), (2, 4104), (1000, 40)])
def test_quantize_is_exact(shape, dtype, block, to):
    x = (randn(*shape, seed=1) * torch.exp(2 * randn(shape[0], 1, seed=2))).to(dtype)
    q, s = tg.quantize_block(x, block, to)
    eq, es = expect_quantized(x, block, to)
    assert q.shape == x.shape and q.dtype == FP8[to][0] and q.stride(0) % 16 == 0
    assert torch.equal(s.cpu(), es)
    assert same_bits(q, eq)
    # what it stands for: half a unit in the last place of the 3- or 2-bit mantissa
    bits = 4 if to == "e4m3" else 3
    step = (2.0 ** -10 if to == "e4m3" else 2.0 ** -17) * s.double()
    rep = lambda t: t.repeat_interleave(1 if block == "row" else 128, 0).repeat_interleave(1 if block == "col" else 128, 1)[:shape[0], :shape[1]]  # noqa: E731
    err = (q.double() * rep(s.double()) - x.double()).abs()
    assert bool((err <= 2.0 ** -bits * x.double().abs() * (1 + 2.0 ** -20) + rep(step)).all())


def test_quantize_extremes():
    x = torch.zeros(4, 256, device="cuda")
    x[0, 3], x[0, 200] = 1e-42, -3e38           # denormal block; a block at the type's end
    x[1, :128] = torch.finfo(torch.float32).min
    x[2, 5], x[2, 130] = math.inf, math.nan
    q, s = tg.quantize_block(x, "row")
    eq, es = expect_quantized(x, "row", "e4m3")
    assert torch.equal(s.cpu(), es)
    assert bool(torch.isfinite(1 / s[:2]).all()) and s[3, 0].item() == 2.0 ** -126
    assert torch.equal(q.float().isnan().cpu(), eq.float().isnan())
    assert torch.equal(q.float().nan_to_num().cpu(), eq.float().nan_to_num())
    v = q.double() * s.double().repeat_interleave(128, 1)
    assert not torch.isfinite(v[2, 5]) and torch.isnan(v[2, 130]) and bool(torch.isfinite(v[[0, 1, 3]]).all())


def test_quantize_strides_batches_and_odd_addresses():
    for dtype in TYPES:
        big = randn(3, 200, 301, seed=3, dtype=dtype)
        for x in (big[:, :, 1:], big[:, ::2, 3:260], big[1:, 5:, :]):
            q, s = tg.quantize_block(x, "tile")
            eq, es = expect_quantized(x, "tile", "e4m3")
            assert torch.equal(s.cpu(), es) and same_bits(q, eq)


def test_quantize_scatter():
    T, k, n = 37, 3, 520
    x = randn(T, n, seed=4, dtype=torch.bfloat16)
    rows = torch.randperm(T * k + 9, generator=gen(5), device="cuda")[:T * k].view(T, k).to(torch.int32)
    rows[3, 1], rows[4, 0], rows[5, 2] = -1, T * k + 9, -7
    q, s = tg.quantize_block(x, "row", scatter=rows.contiguous(), out_rows=T * k + 9)
    eq, es = expect_quantized(x, "row", "e4m3")
    assert q.shape == (T * k + 9, n) and s.shape == (T * k + 9, 5)
    for t in range(T):
        for j in range(k):
            r = int(rows[t, j])
            if 0 <= r < T * k + 9:
                assert same_bits(q[r], eq[t]) and torch.equal(s[r].cpu(), es[t])


def test_quantize_past_32_bits():
    rows, cols = 300000, 8192                   # 2.46e9 elements
    x = torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-1] = randn(cols, seed=6, dtype=torch.bfloat16)
    q, s = tg.quantize_block(x, "row")
    eq, es = expect_quantized(x[-1:], "row", "e4m3")
    assert same_bits(q[-1:], eq) and torch.equal(s[-1:].cpu(), es)
    assert bool((q[:2].float() == 448.0).all())


# ---------------------------------------------------------------- products ---
def values(q, s):
    v = q.double()
    if s.shape[-2] != v.shape[-2]:
        s = s.repeat_interleave(128, -2)[..., :v.shape[-2], :]
    if s.shape[-1] != v.shape[-1]:
        s = s.repeat_interleave(128, -1)[..., :v.shape[-1]]
    return v * s.double()


def act64(y, act):
    return y.clamp_min(0) if act == "relu" else y * torch.special.ndtr(y) if act == "gelu" else y


def held(q, pad, offset):
    """q in memory with `pad` more columns a row and `offset` bytes past an aligned address."""
    rows, cols = q.shape
    flat = torch.zeros(offset + rows * (cols + pad), dtype=torch.uint8, device="cuda")
    v = flat[offset:].view(rows, cols + pad)[:, :cols]
    v.copy_(q.view(torch.uint8))
    return v.view(q.dtype)


def made(rows, cols, block, to, seed, pad=None, offset=0):
    x = randn(rows, cols, seed=seed) * torch.exp(0.5 * randn(rows, 1, seed=seed + 1))
    q, s = tg.quantize_block(x, block, to)
    return (q if pad is None and not offset else held(q, pad or 0, offset)), s


def check_product(C, A, B, sa, sb, out, alpha=1.0, beta=0.0, old=None, bias=None, act="none"):
    a, b = values(A, sa), values(B, sb)
    z, D = alpha * (a @ b), abs(alpha) * (a.abs() @ b.abs())
    if beta:
        z, D = z + beta * old.double(), D + abs(beta) * old.double().abs()
    if bias is not None:
        z, D = z + bias.double(), D + bias.double().abs()
    y = act64(z, act)
    slope = 1.13 if act == "gelu" else 1.0
    tol = slope * (1e-5 + 2.0 ** -22) * D + 2.0 ** -22 * y.abs()
    tol = tol + HALF_ULP[out] * (y.abs() + tol) + (2.0 ** -25 if out == "f16" else 0.0)
    bad = ~((C.double() - y).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((C.double() - y).abs().max()))


# (M, N, K): one token, tile edges, each tile width, K of one, odd everything, K ranges
SHAPES = [(1, 1, 1), (1, 128, 128), (1, 4096, 2048), (7, 130, 300), (16, 256, 4096), (17, 200, 129), (33, 515, 640),
          (64, 1024, 1024), (65, 129, 257), (128, 128, 127), (129, 1, 1000), (200, 300, 1), (257, 513, 777),
          (300, 2048, 512), (1000, 777, 1100)]


@pytest.mark.parametrize("layout", ("forward", "input", "weight"))
@pytest.mark.parametrize("shape", SHAPES)
def test_scaled_product(shape, layout):
    M, N, K = shape
    to = "e5m2" if (M + N) % 3 == 0 else "e4m3"
    if layout == "weight":                       # dW = dY^T X, both token-major, scales along the tokens
        A, sa = made(K, M, "col", to, 10)
        A, sa = A.t(), sa.t()
        B, sb = made(K, N, "col", to, 20)
    else:
        A, sa = made(M, K, "row", to, 10)
        if layout == "forward":                  # W held N x K
            B, sb = made(N, K, "tile", to, 20)
            B, sb = B.t(), sb.t()
        else:                                    # W held K x N
            B, sb = made(K, N, "tile", to, 20)
    for out in ("f32", "bf16"):
        check_product(tg.gemm_scaled(A, sa, B, sb, out=out), A, B, sa, sb, out)


# on this device's 152 SMs the first takes 256 x 256 tiles, the second 256 x 192, both on CTA
# pairs with several tiles in flight and ragged ends
@pytest.mark.parametrize("M,N,K", [(2000, 2001, 2100), (2600, 2296, 1000)])
@pytest.mark.parametrize("layout", ("forward", "input", "weight"))
@pytest.mark.parametrize("out,act", [("f32", "none"), ("bf16", "gelu")])
def test_scaled_pair_tiles(M, N, K, layout, out, act):
    if layout == "weight":
        A, sa = made(K, M, "col", "e4m3", 12)
        A, sa = A.t(), sa.t()
        B, sb = made(K, N, "col", "e4m3", 22)
    else:
        A, sa = made(M, K, "row", "e4m3", 12)
        B, sb = made(N, K, "tile", "e4m3", 22) if layout == "forward" else made(K, N, "tile", "e4m3", 22)
        if layout == "forward":
            B, sb = B.t(), sb.t()
    bias = randn(N, seed=32)
    got = tg.gemm_scaled(A, sa, B, sb, bias=bias, act=act, out=out)
    check_product(got, A, B, sa, sb, out, bias=bias, act=act)
    assert torch.equal(got, tg.gemm_scaled(A, sa, B, sb, bias=bias, act=act, out=out))


@pytest.mark.parametrize("M,N,K", [(5, 300, 500), (150, 260, 390), (150, 1030, 4200)])
@pytest.mark.parametrize("a_block,b_block", [("row", "row"), ("tile", "tile"), ("tile", "row"), ("row", "tile")])
def test_scaled_block_kinds(M, N, K, a_block, b_block):
    A, sa = made(M, K, a_block, "e4m3", 30)
    B, sb = made(N, K, b_block, "e4m3", 40)
    check_product(tg.gemm_scaled(A, sa, B.t(), sb.t()), A, B.t(), sa, sb.t(), "f32")


@pytest.mark.parametrize("M,N,K", [(9, 260, 700), (140, 390, 300)])
@pytest.mark.parametrize("out", ("f32", "bf16", "f16"))
@pytest.mark.parametrize("act", ("none", "relu", "gelu"))
def test_scaled_epilogue_and_guarded_c(M, N, K, out, act):
    A, sa = made(M, K, "row", "e4m3", 50)
    B, sb = made(N, K, "tile", "e4m3", 60)
    bias, old = randn(N, seed=70), randn(M, N, seed=71).to(OUT[out])
    for pad in (0, 1, 8):
        flat = torch.full((2 * GUARD + M * (N + pad),), math.nan, dtype=OUT[out], device="cuda")
        C = flat[GUARD:GUARD + M * (N + pad)].view(M, N + pad)[:, :N]
        C.copy_(old)
        tg.gemm_scaled(A, sa, B.t(), sb.t(), C=C, alpha=0.5, beta=-1.5, bias=bias, act=act, out=out)
        check_product(C, A, B.t(), sa, sb.t(), out, 0.5, -1.5, old, bias, act)
        rest = flat.clone()
        rest[GUARD:GUARD + M * (N + pad)].view(M, N + pad)[:, :N] = math.nan
        assert bool(rest.isnan().all())


@pytest.mark.parametrize("M", (3, 150))
def test_scaled_operands_tma_cannot_address(M):
    N, K = 270, 333
    for pad, offset in ((0, 0), (1, 0), (16 - K % 16, 3), (5, 16)):
        A, sa = made(M, K, "row", "e4m3", 80, pad, offset)
        B, sb = made(N, K, "tile", "e4m3", 90, pad, offset)
        check_product(tg.gemm_scaled(A, sa, B.t(), sb.t()), A, B.t(), sa, sb.t(), "f32")
        B2, sb2 = made(K, N, "tile", "e4m3", 95, pad, offset)
        check_product(tg.gemm_scaled(A, sa, B2, sb2), A, B2, sa, sb2, "f32")


def test_scaled_scales_of_any_stride():
    M, N, K = 140, 300, 520
    A, sa = made(M, K, "row", "e4m3", 100)
    B, sb = made(N, K, "tile", "e4m3", 110)
    want = tg.gemm_scaled(A, sa, B.t(), sb.t())
    wide = torch.full((M, 3 * sa.shape[1]), math.nan, device="cuda")
    wide[:, ::3] = sa
    assert torch.equal(tg.gemm_scaled(A, wide[:, ::3], B.t(), sb.contiguous().t()), want)
    one = torch.ones(1, 1, device="cuda")
    ones = tg.gemm_scaled(A, one.expand(M, sa.shape[1]), B.t(), one.expand(*sb.t().shape))
    assert torch.equal(ones, tg.gemm_scaled(A, torch.ones_like(sa), B.t(), torch.ones_like(sb).t()))


def test_scaled_k_of_zero_is_the_epilogue_of_nothing():
    for M in (3, 200):
        A, B = (torch.empty(s, dtype=torch.float8_e4m3fn, device="cuda") for s in ((M, 0), (0, 130)))
        bias = randn(130, seed=1)
        C = tg.gemm_scaled(A, torch.empty(M, 0, device="cuda"), B, torch.empty(0, 2, device="cuda"), bias=bias)
        assert torch.equal(C, bias.expand(M, 130))


def test_scaled_small_integers_are_exact():
    # products and sums are whole numbers below 2^24, scales powers of two
    for M, N, K in ((5, 200, 3000), (130, 300, 1000)):
        a = torch.randint(-4, 5, (M, K), generator=gen(1), device="cuda").float()
        b = torch.randint(-4, 5, (N, K), generator=gen(2), device="cuda").float()
        kb = cdiv(K, 128)
        sa = 2.0 ** torch.randint(-1, 2, (M, kb), generator=gen(3), device="cuda").float()
        sb = 2.0 ** torch.randint(-1, 2, (cdiv(N, 128), kb), generator=gen(4), device="cuda").float()
        A, B = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
        C = tg.gemm_scaled(A, sa, B.t(), sb.t())
        assert torch.equal(C.double(), values(A, sa) @ values(B.t(), sb.t()))


def test_scaled_a_nan_or_infinity_stays_in_its_row():
    for M in (6, 140):
        A, sa = made(M, 400, "row", "e4m3", 120)
        B, sb = made(200, 400, "tile", "e4m3", 130)
        sa = sa.clone()
        want = tg.gemm_scaled(A, sa, B.t(), sb.t())
        sa[2, 1], sa[4, 3] = math.nan, math.inf
        got = tg.gemm_scaled(A, sa, B.t(), sb.t())
        keep = [i for i in range(M) if i not in (2, 4)]
        assert torch.equal(got[keep], want[keep])
        assert bool(got[2].isnan().all()) and not bool(torch.isfinite(got[4]).any())


@pytest.mark.parametrize("M,N,K", [(8, 512, 4096), (150, 300, 700), (600, 1024, 2048)])
def test_scaled_wait_that_runs_out_is_reported_and_leaves_the_device_usable(M, N, K):
    A, sa = made(M, K, "row", "e4m3", 160)
    B, sb = made(N, K, "tile", "e4m3", 170)
    want = tg.gemm_scaled(A, sa, B.t(), sb.t())
    s = torch.cuda.current_stream().cuda_stream
    assert tg.gemm_set_option("wait_timeout_ms", 100) == tg.GEMM_OK
    assert tg.gemm_set_option("debug_stall_mma", 1) == tg.GEMM_OK
    try:
        tg.gemm_scaled(A, sa, B.t(), sb.t())
        assert tg.gemm_get_status(s) == tg.GEMM_ERR_TIMEOUT
        assert "role=mma" in tg.gemm_last_error()
    finally:
        tg.gemm_set_option("wait_timeout_ms", 2000)
        tg.gemm_set_option("debug_stall_mma", 0)
    assert tg.gemm_get_status(s) == tg.GEMM_OK
    assert torch.equal(tg.gemm_scaled(A, sa, B.t(), sb.t()), want)


def test_scaled_runs_on_other_streams_in_order_and_repeats_bit_for_bit():
    A, sa = made(24, 4096, "row", "e4m3", 140)
    B, sb = made(2048, 4096, "tile", "e4m3", 150)
    want = tg.gemm_scaled(A, sa, B.t(), sb.t(), out="bf16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        outs = []
        for _ in range(6):
            x = want.float()
            q, qs = tg.quantize_block(x, "row")
            outs.append((tg.gemm_scaled(A, sa, B.t(), sb.t(), out="bf16"),
                         tg.gemm_scaled(q, qs, B, sb)))
    s.synchronize()
    for o, y in outs:
        assert torch.equal(o, want) and torch.equal(y, outs[0][1])


# ------------------------------------------------------------------ experts ---
def check_experts(C, A, sa, W, sw, off, out, act="none", fill=None):
    off = off.tolist()
    for e in range(W.shape[0]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            check_product(C[lo:hi], A[lo:hi], W[e], sa[lo:hi], sw[e], out, act=act)
    if fill is not None:
        assert bool((C[:off[0]] == fill).all()) and bool((C[off[-1]:] == fill).all())


@pytest.mark.parametrize("major", ("k", "n"))
@pytest.mark.parametrize("counts,N,K", [
    ([1], 128, 128), ([0, 0, 3, 0], 200, 130), ([5, 0, 16, 1, 17, 2], 300, 520), ([40, 64, 0, 33], 129, 1000),
    ([100, 0, 129, 300, 128, 1], 515, 384), ([700, 1, 0, 257], 256, 77)])
def test_experts_product(counts, N, K, major):
    E, R = len(counts), sum(counts)
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    A, sa = made(R, K, "row", "e4m3", 200)
    x = randn(E, *((N, K) if major == "k" else (K, N)), seed=210)
    W, sw = tg.quantize_block(x, "tile")
    if major == "k":
        W, sw = W.transpose(1, 2), sw.transpose(1, 2)
    for out, act in (("f32", "none"), ("bf16", "gelu")):
        check_experts(tg.gemm_experts(A, sa, W, sw, off, act=act, out=out), A, sa, W, sw, off, out, act)


@pytest.mark.parametrize("rows", (40, 900))
def test_experts_rows_of_no_expert_are_left_alone(rows):
    E, N, K = 5, 150, 260
    A, sa = made(rows, K, "row", "e4m3", 220)
    W, sw = tg.quantize_block(randn(E, N, K, seed=221), "tile")
    W, sw = W.transpose(1, 2), sw.transpose(1, 2)
    off = torch.tensor([3, 3, rows // 2, rows // 2 + 1, rows - 8, rows - 5], dtype=torch.int32, device="cuda")
    C = torch.full((rows, N), 7.0, device="cuda")
    tg.gemm_experts(A, sa, W, sw, off, C=C)
    check_experts(C, A, sa, W, sw, off, "f32", fill=7.0)
    # offsets that do not ascend, or leave the rows, are clamped: nothing is written outside the rows
    flat = torch.full((rows + 2, N), 7.0, device="cuda")
    wild = torch.tensor([-5, rows + 100, 2, rows - 1, 0, 1 << 30], dtype=torch.int32, device="cuda")
    tg.gemm_experts(A, sa, W, sw, wild, C=flat[1:-1])
    assert bool((flat[0] == 7.0).all()) and bool((flat[-1] == 7.0).all())
    check_product(flat[1:-1], A, W[0], sa, sw[0], "f32")


def test_experts_scale_per_column_a_that_tma_cannot_address_and_no_rows():
    E, N, K = 3, 200, 300
    A, sa = made(70, K, "row", "e4m3", 230, 3, 1)
    W, sw = tg.quantize_block(randn(E, N, K, seed=231), "row")
    W, sw = W.transpose(1, 2), sw.transpose(1, 2)
    off = torch.tensor([0, 30, 30, 70], dtype=torch.int32, device="cuda")
    check_experts(tg.gemm_experts(A, sa, W, sw, off), A, sa, W, sw, off, "f32")
    A, sa = made(900, K, "row", "e4m3", 232, 3, 1)
    off = torch.tensor([0, 300, 301, 900], dtype=torch.int32, device="cuda")
    check_experts(tg.gemm_experts(A, sa, W, sw, off), A, sa, W, sw, off, "f32")
    none = tg.gemm_experts(A[:0], sa[:0], W, sw, torch.zeros(E + 1, dtype=torch.int32, device="cuda"))
    assert none.shape == (0, N)


@pytest.mark.parametrize("out", ("f32", "bf16"))
def test_experts_many_tiles_a_block(out):
    # whole and ragged tiles in turn on every block: boxes of C leave by TMA and by ordinary stores
    E, N, K = 48, 1024, 256
    counts = [260 + (37 * e) % 90 for e in range(E)]
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    A, sa = made(int(off[-1]), K, "row", "e4m3", 260)
    W, sw = tg.quantize_block(randn(E, N, K, seed=261), "tile")
    W, sw = W.transpose(1, 2), sw.transpose(1, 2)
    first = tg.gemm_experts(A, sa, W, sw, off, out=out)
    check_experts(first, A, sa, W, sw, off, out)
    for _ in range(5):
        assert torch.equal(tg.gemm_experts(A, sa, W, sw, off, out=out), first)


def test_experts_many_and_weights_past_32_bits():
    E, N, K = 700, 1536, 2048                    # 2.2e9 bytes of weights
    W = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda")
    q, s = made(N, K, "tile", "e4m3", 240)
    W[-1], W[0] = q.view(torch.uint8), q.view(torch.uint8)
    sw = s.expand(E, *s.shape).contiguous()
    W = W.view(torch.float8_e4m3fn).transpose(1, 2)
    A, sa = made(20, K, "row", "e4m3", 250)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = 9
    off[-1] = 20
    C = tg.gemm_experts(A, sa, W, sw.transpose(1, 2), off)
    check_product(C[:9], A[:9], W[0], sa[:9], s.t(), "f32")
    check_product(C[9:], A[9:], W[-1], sa[9:], s.t(), "f32")


# -------------------------------------------------------------------- route ---
def route_reference(x, k, score, bias, groups, top_groups, group_score, renorm, scale):
    """The rules, token by token, in 64 bits."""
    T, E = x.shape
    x = x.double().cpu()
    x = torch.where(x > -math.inf, x, torch.full((), -math.inf, dtype=torch.float64))
    per = E // groups
    idx = torch.full((T, k), -1, dtype=torch.int64)
    w = torch.zeros((T, k), dtype=torch.float64)
    for t in range(T):
        r = x[t]
        real = r > -math.inf
        if score == "sigmoid":
            s = torch.sigmoid(r)
        elif bool((r == math.inf).any()):
            s = (r == math.inf).double() / (r == math.inf).sum()
        elif bool(real.any()):
            s = torch.softmax(r, 0)
        else:
            s = torch.zeros(E, dtype=torch.float64)
        s = torch.where(real, s, torch.zeros((), dtype=torch.float64))
        key = s + bias.double().cpu() if bias is not None else r
        key = [float(key[e]) if bool(real[e]) and float(key[e]) > -math.inf else None for e in range(E)]
        if groups > 1 and top_groups < groups:
            worth = []
            for g in range(groups):
                v = [(float(s[e]) if bias is None and group_score == "top2" else key[e])
                     for e in range(g * per, (g + 1) * per) if key[e] is not None]
                v.sort(reverse=True)
                worth.append(None if not v else v[0] + (v[1] if group_score == "top2" and len(v) > 1 else 0.0))
            order = sorted((g for g in range(groups) if worth[g] is not None), key=lambda g: (-worth[g], g))
            for g in range(groups):
                if g not in order[:top_groups]:
                    for e in range(g * per, (g + 1) * per):
                        key[e] = None
        order = sorted((e for e in range(E) if key[e] is not None), key=lambda e: (-key[e], e))[:k]
        for j, e in enumerate(order):
            idx[t, j], w[t, j] = e, s[e]
        if renorm and float(w[t].sum()) > 0:
            w[t] /= w[t].sum()
        w[t] *= scale
    return idx, w


def order_reference(idx, E):
    flat = idx.reshape(-1)
    rows = [[] for _ in range(E)]
    for i, e in enumerate(flat.tolist()):
        if e >= 0:
            rows[e].append(i)
    order = [i for r in rows for i in r]
    off = [0]
    for r in rows:
        off.append(off[-1] + len(r))
    slots = torch.full_like(flat, -1)
    for r, i in enumerate(order):
        slots[i] = r
    return off, order + [-1] * (flat.numel() - len(order)), slots.view(idx.shape)


def check_route(x, k, score="softmax", bias=None, groups=1, top_groups=None, group_score="max", renorm=True, scale=1.0):
    r = tg.route(x, k, score=score, bias=bias, groups=groups, top_groups=top_groups, group_score=group_score,
                 renormalize=renorm, scale=scale)
    idx, w = route_reference(x, k, score, bias, groups, groups if top_groups is None else top_groups, group_score,
                             renorm, scale)
    assert torch.equal(r.indices.cpu().long(), idx)
    assert bool(((r.weights.cpu().double() - w).abs() <= 48 * 2.0 ** -24 * w.abs() + 2.0 ** -126).all())
    off, order, slots = order_reference(idx, x.shape[1])
    assert r.offsets.tolist() == off and r.order.tolist() == order
    assert torch.equal(r.slots.cpu().long(), slots)
    return r


def spread_logits(T, E, dtype, seed):
    """Each token's logits are a permutation of evenly spaced values: no two keys close."""
    p = torch.stack([torch.randperm(E, generator=gen(seed + t), device="cuda") for t in range(T)])
    return ((p.float() - E / 2) * (6.0 / E)).to(dtype)


@pytest.mark.parametrize("T", (1, 31, 33, 128, 129, 300))
@pytest.mark.parametrize("E,k,groups,top", [(1, 1, 1, 1), (8, 2, 1, 1), (60, 6, 1, 1), (256, 8, 8, 4), (160, 6, 4, 1),
                                            (24, 5, 24, 7), (96, 7, 3, 2)])
def test_route(T, E, k, groups, top):
    for score in ("softmax", "sigmoid"):
        for gs in (("max", "top2") if groups > 1 else ("max",)):
            check_route(spread_logits(T, E, torch.float32, 7), k, score, None, groups, top, gs, True, 2.5)
    b = 0.01 * ((torch.arange(E, device="cuda") * 7) % 11).float()
    check_route(spread_logits(T, E, torch.float32, 8), k, "sigmoid", b, groups, top, "top2", False)


@pytest.mark.parametrize("E", (512, 1000, 1024))
def test_route_many_experts(E):
    for T in (5, 140):
        check_route(spread_logits(T, E, torch.float32, 9), 32, "softmax")
        if E % 8 == 0:
            check_route(spread_logits(T, E, torch.float32, 9), 16, "softmax", None, 8, 3, "max")


@pytest.mark.parametrize("dtype", TYPES)
def test_route_ties_go_to_the_lower_index(dtype):
    x = torch.randint(0, 4, (200, 64), generator=gen(1), device="cuda").to(dtype)
    x[0] = 0.0
    x[1, ::2], x[1, 1::2] = -0.0, 0.0
    check_route(x, 9)
    check_route(x, 9, "sigmoid", None, 8, 3, "max")


@pytest.mark.parametrize("T", (40, 200))
@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
def test_route_masks(T, score):
    for dtype in TYPES:
        x = spread_logits(T, 32, dtype, 11)
        x[1] = -math.inf                                     # nothing left
        x[2, 5:] = -math.inf                                 # fewer than k
        x[3] = torch.finfo(dtype).min                        # the type's lowest value is a value
        x[4, :30] = torch.finfo(dtype).min
        x[5, 3], x[5, 9] = math.nan, math.nan
        x[6, 7], x[6, 20] = math.inf, math.inf
        x[7, 1:] = -math.inf
        r = check_route(x, 8, score)
        assert r.indices[1].tolist() == [-1] * 8 and bool((r.weights[1] == 0).all())
        x[8, :16] = -math.inf                                # whole groups masked
        x[9, 1:8] = -math.inf                                # a group with one expert
        check_route(x, 6, score, None, 4, 3, "top2")
        check_route(x, 6, score, None, 4, 3, "max")
    b = torch.zeros(32, device="cuda")
    b[3], b[4] = -math.inf, math.nan
    r = check_route(x.float(), 8, "sigmoid", b)
    assert not bool(((r.indices == 3) | (r.indices == 4)).any())


def test_route_strided_logits_and_no_tokens():
    x = spread_logits(50, 64, torch.bfloat16, 12)
    wide = torch.zeros(50, 71, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:67] = x
    a, b = tg.route(wide[:, 3:67], 4), tg.route(x, 4)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    r = tg.route(x[:0], 4)
    assert r.offsets.tolist() == [0] * 65 and r.indices.shape == (0, 4)


def test_route_many_tokens_repeats_bit_for_bit():
    x = randn(20000, 128, seed=13, dtype=torch.bfloat16)
    a, b = tg.route(x, 8), tg.route(x, 8)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    flat = a.indices.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(a.order.long(), order)
    assert torch.equal(a.offsets.long()[1:], torch.bincount(flat, minlength=128).cumsum(0))
    assert torch.equal(a.slots.reshape(-1).long()[order], torch.arange(flat.numel(), device="cuda"))


def weights64(x, idx, score, renorm, scale):
    s = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    w = torch.where(idx >= 0, s.gather(1, idx.clamp_min(0)), torch.zeros((), dtype=x.dtype, device=x.device))
    if renorm:
        z = w.sum(1, keepdim=True)
        w = w / torch.where(z > 0, z, torch.ones_like(z))
    return scale * w


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("renorm", (True, False))
@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (9, 8, 8), (130, 60, 4), (40, 256, 8), (5, 1024, 32)])
def test_route_backward(T, E, k, score, renorm, dtype):
    x = randn(T, E, seed=14, dtype=dtype)
    if E > 8:
        x[0, 0] = -math.inf
    r = tg.route(x, k, score=score, renormalize=renorm, scale=1.5)
    idx = r.indices.clone()
    if k > 2:
        idx[-1, 1] = -1
    g = randn(T, k, seed=15)
    got = tg.route_backward(g, x, idx, score=score, renormalize=renorm, scale=1.5).double()
    # against the formula in 64 bits (by autograd of the definition)
    xd = x.double().requires_grad_(True)
    w = weights64(xd, idx.long(), score, renorm, 1.5)
    want, = torch.autograd.grad((w * g.double()).sum(), xd)
    want = want.nan_to_num()
    # each of the few terms of a logit's gradient is at most its weight times |g| over the sum
    size = (w.detach().abs() * g.double().abs()).sum(1, keepdim=True) + (g.double().abs().amax(1, keepdim=True) * 1.5)
    half = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dtype]
    tol = 64 * 2.0 ** -24 * size * (4.0 if renorm else 1.0) + half * want.abs() + (2.0 ** -25 if dtype == torch.float16 else 0)
    assert bool(((got - want).abs() <= tol).all())
    # against differences of the definition along random directions
    for seed in (1, 2):
        d = randn(T, E, seed=20 + seed).double()
        h = 1e-5
        base = torch.where(x.double() > -math.inf, x.double(), torch.full((), -math.inf, device="cuda", dtype=torch.float64))
        up, down = (weights64(base + sgn * h * d, idx.long(), score, renorm, 1.5) for sgn in (1, -1))
        slope = ((up - down) / (2 * h) * g.double()).sum(1)
        mine = (got * d).sum(1)
        assert bool(((mine - slope).abs() <= (tol * d.abs()).sum(1) + 1e-8 * (1 + size[:, 0] * E)).all())


def test_route_backward_of_one_renormalised_expert_is_zero():
    x = randn(50, 64, seed=16)
    r = tg.route(x, 1)
    assert bool((tg.route_backward(randn(50, 1, seed=17), x, r.indices) == 0).all())


# ------------------------------------------------------------------ combine ---
def combine64(y, slots, w):
    s = slots.long()
    real = (s >= 0) & (s < y.shape[0])
    rows = torch.where(real[:, :, None], y.double()[s.clamp(0, y.shape[0] - 1)], torch.zeros((), dtype=torch.float64, device="cuda"))
    w = torch.ones_like(slots, dtype=torch.float64) if w is None else w.double()
    return (w[:, :, None] * rows).sum(1), (w[:, :, None] * rows).abs().sum(1)


HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (5, 8, 64), (33, 3, 1000), (7, 11, 4104), (100, 2, 77), (3, 1, 8192)])
def test_combine_and_its_gradients(T, k, H, dtype):
    R = T * k
    y = randn(R, H, seed=30, dtype=dtype)
    slots = torch.randperm(R, generator=gen(31), device="cuda").view(T, k).to(torch.int32)
    order = torch.empty(R, dtype=torch.int32, device="cuda")
    order[slots.reshape(-1).long()] = torch.arange(R, dtype=torch.int32, device="cuda")
    if R > 4:                                   # a pair without an expert: its row has no pair
        order[slots[1, 0].long()] = -1
        slots[1, 0] = -1
    w = randn(T, k, seed=32)
    for ww in (w, None):
        want, size = combine64(y, slots, ww)
        got = tg.combine(y, slots, ww)
        tol = (k + 1) * 2.0 ** -24 * size + HALF[dtype] * want.abs() * (1 + 2.0 ** -20) + (2.0 ** -25 if dtype == torch.float16 else 0)
        assert got.dtype == dtype and bool(((got.double() - want).abs() <= tol).all())
    g = randn(T, H, seed=33, dtype=dtype)
    real = slots.reshape(-1) >= 0
    at = slots.reshape(-1)[real].long()
    for o in (order, None):
        dy, dw = tg.combine_backward(g, y, slots, w, o)
        want = torch.zeros_like(y)
        want[at] = (w[:, :, None] * g.float()[:, None, :]).to(dtype).reshape(R, H)[real]
        assert torch.equal(dy, want)
        z = torch.zeros((), dtype=torch.float64, device="cuda")
        prod = torch.where((slots >= 0)[:, :, None], y.double()[slots.clamp_min(0).long()] * g.double()[:, None, :], z)
        assert bool(((dw.double() - prod.sum(2)).abs() <= 64 * 2.0 ** -24 * prod.abs().sum(2)).all())
    # against differences of the definition (which is linear in y and in w)
    d, dv = randn(R, H, seed=34).double(), randn(T, k, seed=35).double()
    h = 2.0 ** -10
    f = lambda a, b: (combine64(a, slots, b)[0] * g.double()).sum()   # noqa: E731
    along_y = (f(y.double() + h * d, w) - f(y.double() - h * d, w)) / (2 * h)
    along_w = (f(y, w.double() + h * dv) - f(y, w.double() - h * dv)) / (2 * h)
    assert abs(float((dy.double() * d).sum() - along_y)) <= (HALF[dtype] + 2.0 ** -24) * float((want.double() * d).abs().sum()) * 1.01 + 1e-6
    assert abs(float((dw.double() * dv).sum() - along_w)) <= 64 * 2.0 ** -24 * float((prod.abs().sum(2) * dv.abs()).sum()) + 1e-6


def test_combine_strides_and_rows_outside():
    y = randn(20, 200, seed=40, dtype=torch.bfloat16)
    slots = torch.tensor([[0, 19], [20, 5], [-1, -3], [1 << 30, 7]], dtype=torch.int32, device="cuda")
    w = randn(4, 2, seed=41)
    for a, b in ((1, 70), (8, 72), (3, 130)):
        out = torch.full((4, 140), 9.0, dtype=torch.bfloat16, device="cuda")
        tg.combine(y[:, a:b], slots, w, out=out[:, 5:5 + b - a])
        assert torch.equal(out[:, 5:5 + b - a], tg.combine(y[:, a:b].contiguous(), slots, w))
        assert bool((out[:, :5] == 9.0).all()) and bool((out[:, 5 + b - a:] == 9.0).all())
    assert bool((tg.combine(y, slots, w)[2] == 0).all())


def test_combine_past_32_bits():
    R, H = 600000, 4096                          # 2.46e9 elements
    y = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    y[-1], y[0] = 3.0, 5.0
    slots = torch.tensor([[R - 1, 0]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, 2.0]], device="cuda")
    assert bool((tg.combine(y, slots, w) == 13.0).all())
    g = torch.ones((1, H), dtype=torch.bfloat16, device="cuda")
    dy, dw = tg.combine_backward(g, y, slots, w)
    assert dw.tolist() == [[3.0 * H, 5.0 * H]] and bool((dy[-1] == 1.0).all()) and bool((dy[0] == 2.0).all())


# ------------------------------------------------------------- all together ---
@pytest.mark.parametrize("T", (1, 40, 700))
def test_an_expert_layer(T):
    E, k, H, F = 16, 4, 384, 520
    x = randn(T, H, seed=50, dtype=torch.bfloat16)
    w1, w2 = randn(E, F, H, seed=51) * H ** -0.5, randn(E, H, F, seed=52) * F ** -0.5
    logits = randn(T, E, seed=53)
    w1q, w1s = tg.quantize_block(w1, "tile")
    w2q, w2s = tg.quantize_block(w2, "tile")
    r = tg.route(logits, k, score="sigmoid")
    xq, xs = tg.quantize_block(x, "row", scatter=r.slots)
    h = tg.gemm_experts(xq, xs, w1q.transpose(1, 2), w1s.transpose(1, 2), r.offsets, act="gelu", out="bf16")
    hq, hs = tg.quantize_block(h, "row")
    y = tg.gemm_experts(hq, hs, w2q.transpose(1, 2), w2s.transpose(1, 2), r.offsets, out="bf16")
    out = tg.combine(y, r.slots, r.weights).double()
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(r.indices[t, j])
            want[t] += r.weights[t, j].double() * (act64(x[t].double() @ w1[e].double().t(), "gelu") @ w2[e].double().t())
    # two FP8 roundings of activations and two of weights, each 2^-4 relative at most and
    # about 2^-5.8 rms: the norm of the error stays well under 8 %
    assert float((out - want).norm() / want.norm()) < 0.08


def test_the_example_runs_them_together():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    found = example.main(hidden=512, inner=384, experts=16, top_k=4, tokens=(5, 300))
    # one FP8 rounding of each operand: 2^-4 relative at most, about 0.025 rms each; two
    # products in a row for the experts
    assert found["Y"] < 0.05 and found["dX"] < 0.05 and found["dW"] < 0.05
    assert all(v < 0.08 for v in found.values())


@pytest.mark.parametrize("T", (40, 300))         # 300: the routing takes a workspace
def test_operators_in_a_cuda_graph(T):
    x = randn(T, 512, seed=60, dtype=torch.bfloat16)
    w, ws = tg.quantize_block(randn(8, 256, 512, seed=61), "tile")
    logits = randn(T, 8, seed=62)

    def layer():
        r = tg.route(logits, 2)
        q, s = tg.quantize_block(x, "row", scatter=r.slots)
        y = tg.gemm_experts(q, s, w.transpose(1, 2), ws.transpose(1, 2), r.offsets, out="bf16")
        return tg.combine(y, r.slots, r.weights)

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    logits.copy_(randn(T, 8, seed=63))
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    assert torch.equal(got, layer())


# --------------------------------------------------- one row expanded over all ---
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,H", [(5, 2, 64), (70, 4, 1000), (33, 3, 77)])
def test_a_row_expanded_is_read_like_its_copies(T, k, H, dtype):
    # a neighbour in the same storage that a dense pitch would read: equal results come from the row alone
    def expanded(rows, cols, seed):
        held = randn(rows + 1, cols, seed=seed, dtype=dtype)
        held[1:] = math.nan
        return held[:1].expand(rows, cols)
    R = T * k
    slots = torch.randperm(R, generator=gen(70), device="cuda").view(T, k).to(torch.int32)
    w, y, g = randn(T, k, seed=71), randn(R, H, seed=72, dtype=dtype), randn(T, H, seed=73, dtype=dtype)
    ye, ge = expanded(R, H, 74), expanded(T, H, 75)
    assert torch.equal(tg.combine(ye, slots, w), tg.combine(ye.contiguous(), slots, w))
    for a, b in ((ge, y), (g, ye), (ge, ye)):
        got, want = tg.combine_backward(a, b, slots, w), tg.combine_backward(a.contiguous(), b.contiguous(), slots, w)
        assert all(torch.equal(u, v) for u, v in zip(got, want))
    x = expanded(T, 64, 76)
    r = tg.route(x, 3)
    assert all(torch.equal(u, v) for u, v in zip(r, tg.route(x.contiguous(), 3)))
    gw = randn(T, 3, seed=77)
    assert torch.equal(tg.route_backward(gw, x, r.indices), tg.route_backward(gw, x.contiguous(), r.indices))
    for block in ("row", "col", "tile"):
        for z in (ye, expanded(R, 1, 78)):
            q, s = tg.quantize_block(z, block)
            eq, es = tg.quantize_block(z.contiguous(), block)
            assert same_bits(q, eq) and torch.equal(s, es)


def test_combine_backward_takes_the_gradient_of_a_sum_over_tokens():
    T, k, H = 40, 2, 264
    slots = torch.randperm(T * k, generator=gen(80), device="cuda").view(T, k).to(torch.int32)
    w, y = randn(T, k, seed=81), randn(T * k, H, seed=82)
    out = tg.combine(y, slots, w).requires_grad_(True)
    grad, = torch.autograd.grad(out.sum(0), out, randn(H, seed=83))
    assert grad.stride() == (0, 1)
    got, want = tg.combine_backward(grad, y, slots, w), tg.combine_backward(grad.contiguous(), y, slots, w)
    assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_expanded_rows_are_refused_where_they_are_written_or_go_through_tma():
    A, sa = made(8, 128, "row", "e4m3", 84)
    B, sb = made(64, 128, "tile", "e4m3", 85)
    one = torch.zeros(1, 64, device="cuda").expand(8, 64)
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    slots = torch.zeros(8, 1, dtype=torch.int32, device="cuda")
    A1 = A[:1].expand(8, 128)
    for call in (lambda: tg.gemm_scaled(A, sa, B.t(), sb.t(), C=one), lambda: tg.gemm_scaled(A1, sa, B.t(), sb.t()),
                 lambda: tg.gemm_scaled(A, sa, B[:1].expand(64, 128).t(), sb.t()),
                 lambda: tg.gemm_experts(A, sa, B.t()[None], sb.t()[None], off, C=one),
                 lambda: tg.gemm_experts(A1, sa, B.t()[None], sb.t()[None], off),
                 lambda: tg.combine(randn(8, 64), slots, out=one)):
        with pytest.raises(ValueError, match="expanded"):
            call()


# ------------------------------------------------ NaN and infinity through an activation ---
# on this device: tiles of 16 columns, the same with K in ranges, 64 columns, 128 x 128, and the two
# pair tiles; the last has a pitch of C that TMA cannot store to
@pytest.mark.parametrize("M,N,K", [(6, 200, 400), (6, 256, 4096), (50, 300, 1024), (140, 200, 400), (2600, 2296, 1000),
                                   (2000, 2001, 2100)])
@pytest.mark.parametrize("act", ("relu", "gelu"))
@pytest.mark.parametrize("out", ("f32", "bf16"))
def test_scaled_a_nan_or_infinity_passes_the_activation(M, N, K, act, out):
    x = randn(M, K, seed=300)
    x[2, 130], x[4, 259] = math.nan, math.inf
    A, sa = tg.quantize_block(x, "row")
    B, sb = made(N, K, "tile", "e4m3", 310)
    got = tg.gemm_scaled(A, sa, B.t(), sb.t(), act=act, out=out)
    keep = [i for i in range(M) if i not in (2, 4)]
    assert bool(got[2].isnan().all()) and bool(got[4].isnan().all())
    check_product(got[keep], A[keep], B.t(), sa[keep], sb.t(), out, act=act)


@pytest.mark.parametrize("counts", ([1, 5, 0, 3], [60, 70, 0, 100], [300, 0, 257, 129]))
@pytest.mark.parametrize("act", ("relu", "gelu"))
def test_experts_a_nan_or_infinity_passes_the_activation(counts, act):
    E, R, N, K = len(counts), sum(counts), 260, 300
    x = randn(R, K, seed=320)
    x[2, 130], x[4, 259] = math.nan, math.inf
    A, sa = tg.quantize_block(x, "row")
    W, sw = tg.quantize_block(randn(E, N, K, seed=321), "tile")
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    got = tg.gemm_experts(A, sa, W.transpose(1, 2), sw.transpose(1, 2), off, act=act)
    assert bool(got[2].isnan().all()) and bool(got[4].isnan().all())
    keep = [i for i in range(R) if i not in (2, 4)]
    assert bool(torch.isfinite(got[keep]).all())


# expf within 2 units in the last place twice, four additions and divisions, three products, each half a
# unit: under 16 * 2^-24 of the gradient itself (and what is below the type's normal numbers)
@pytest.mark.parametrize("dtype", TYPES)
def test_route_backward_of_large_sigmoid_logits_is_relatively_exact(dtype):
    k = 16
    x = torch.linspace(-30, 30, 61, device="cuda").to(dtype)[torch.randperm(61, generator=gen(90), device="cuda")]
    x = torch.stack([x.roll(i) for i in range(61)])
    idx = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32)    # 15 .. 30
    idx[::2] = torch.sort(x, dim=1, stable=True).indices[::2, :k].to(torch.int32)              # -30 .. -15
    g = randn(61, k, seed=91)
    got = tg.route_backward(g, x, idx, score="sigmoid", renormalize=False, scale=2.0).double()
    sel = x.double().gather(1, idx.long())
    want = torch.zeros_like(x, dtype=torch.float64)
    want.scatter_(1, idx.long(), 2.0 * g.double() * torch.sigmoid(sel) * torch.sigmoid(-sel))
    half = 0.0 if dtype == torch.float32 else HALF[dtype]
    tol = (16 * 2.0 ** -24 + half) * want.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    assert bool(((got - want).abs() <= tol).all())
    assert bool((got.gather(1, idx.long()) != 0).all()) or dtype == torch.float16


@pytest.mark.parametrize("counts", ([3, 0, 9], [200, 1, 300]))
@pytest.mark.parametrize("N,K,major", [(1, 100, "k"), (77, 1, "n"), (1, 1, "k"), (1, 1, "n"), (1, 333, "n"), (77, 1, "k")])
def test_experts_of_one_row_or_column(counts, N, K, major):
    E, R = len(counts), sum(counts)
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    A, sa = made(R, K, "row", "e4m3", 270)
    W, sw = tg.quantize_block(randn(E, *((N, K) if major == "k" else (K, N)), seed=271), "tile")
    if major == "k":
        W, sw = W.transpose(1, 2), sw.transpose(1, 2)
    check_experts(tg.gemm_experts(A, sa, W, sw, off), A, sa, W, sw, off, "f32")


FIRST_CALL_IN_A_CAPTURE = """
import torch
import tiled_tensor_core_gemm_gb300 as tg
gen = torch.Generator(device="cuda")
gen.manual_seed(1)
rand = lambda *s: torch.randn(s, generator=gen, device="cuda")
logits, more, x = rand(300, 16), rand(300, 16), rand(300, 256).to(torch.bfloat16)
held = torch.zeros(300 * 257, dtype=torch.uint8, device="cuda")
def layer():
    r = tg.route(logits, 3)                                       # takes a workspace
    a = held.view(300, 257)[:, :256].view(torch.float8_e4m3fn)    # TMA cannot address its rows: another
    one = torch.ones(300, 2, device="cuda")
    q, s = tg.quantize_block(x, "row")
    return r, tg.gemm_scaled(a, one, q.t(), s.t())
held.copy_(rand(300 * 257).to(torch.float8_e4m3fn).view(torch.uint8))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    r, c = layer()
logits.copy_(more)
for _ in range(3):
    graph.replay()
torch.cuda.synchronize()
got, gc = [t.clone() for t in r], c.clone()
want, wc = layer()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(gc, wc)
assert bool(torch.isfinite(wc).all())
print("equal")
"""


def test_the_first_call_may_be_in_a_capture():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "equal" in run.stdout, run.stderr[-2000:]


# Tensors that end where their allocation does (each is one of its own here), at sizes no multiple of 16 bytes.
ROWS_THAT_END_THEIR_ALLOCATION = """
import torch
import tiled_tensor_core_gemm_gb300 as tg
gen = torch.Generator(device="cuda")
gen.manual_seed(1)
rand = lambda *s: torch.randn(s, generator=gen, device="cuda")
def roomy(t):
    held = torch.zeros(t.numel() + 64, dtype=t.dtype, device="cuda")
    held[:t.numel()] = t.reshape(-1)
    return held[:t.numel()].view(t.shape)
def same(a, b):
    plain = lambda t: t.clone(memory_format=torch.contiguous_format).view(torch.uint8)
    return all(torch.equal(plain(x), plain(y)) for x, y in zip(a, b))
for dtype in (torch.float32, torch.bfloat16, torch.float16):
    for T, k, H in ((1, 1, 5), (3, 1, 77), (5, 2, 131), (37, 3, 1001)):
        y, g, w = rand(T * k, H).to(dtype), rand(T, H).to(dtype), rand(T, k)
        slots = torch.randperm(T * k, generator=gen, device="cuda").view(T, k).to(torch.int32)
        assert y.numel() * y.element_size() % 16 and y.data_ptr() % 256 == 0
        assert same([tg.combine(y, slots, w)], [tg.combine(roomy(y), slots, w)])
        assert same(tg.combine_backward(g, y, slots, w), tg.combine_backward(roomy(g), roomy(y), slots, w))
        for block in ("row", "col", "tile"):
            assert same(tg.quantize_block(y, block), tg.quantize_block(roomy(y), block))
        assert same(tg.quantize_block(g, "row", scatter=slots), tg.quantize_block(roomy(g), "row", scatter=slots))
torch.cuda.synchronize()
print("equal")
"""


def test_rows_that_end_their_allocation():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", ROWS_THAT_END_THEIR_ALLOCATION], cwd=root, capture_output=True, text=True,
                         timeout=300, env=dict(os.environ, PYTORCH_NO_CUDA_MEMORY_CACHING="1"))
    assert run.returncode == 0 and "equal" in run.stdout, run.stderr[-2000:]


# ------------------------------------------------------------ forms and their corners ---
# rows an expert on average: tiles of 16 and of 64 columns, 128 x 128, pairs of 256 x 192 (short K) and, with
# one scale a column, of 256 x 256
@pytest.mark.parametrize("counts,N,K,w_block", [
    ([3, 0, 9, 1], 150, 260, "tile"), ([40, 33, 0, 61], 300, 390, "tile"), ([90, 128, 0, 100], 260, 520, "tile"),
    ([300, 0, 257, 640], 520, 300, "tile"), ([300, 129, 0, 555], 520, 300, "row")])
@pytest.mark.parametrize("to,out,act,alpha", [("e5m2", "f16", "none", 0.5), ("e5m2", "f32", "relu", -1.5),
                                              ("e4m3", "bf16", "relu", 0.25), ("e4m3", "f16", "gelu", -0.5)])
def test_experts_types_activations_and_guarded_c(counts, N, K, w_block, to, out, act, alpha):
    E, R = len(counts), sum(counts)
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    A, sa = made(R, K, "row", to, 400)
    W, sw = tg.quantize_block(randn(E, N, K, seed=410), w_block, to)
    W, sw = W.transpose(1, 2), sw.transpose(1, 2)
    for pad, offset in ((0, 0), (1, 0), (8, 3)):
        flat = torch.full((2 * GUARD + offset + R * (N + pad),), math.nan, dtype=OUT[out], device="cuda")
        inside = slice(GUARD + offset, GUARD + offset + R * (N + pad))
        C = flat[inside].view(R, N + pad)[:, :N]
        assert tg.gemm_experts(A, sa, W, sw, off, C=C, alpha=alpha, act=act, out=out) is C
        lo = 0
        for e, n in enumerate(counts):
            if n:
                check_product(C[lo:lo + n], A[lo:lo + n], W[e], sa[lo:lo + n], sw[e], out, alpha, act=act)
            lo += n
        rest = flat.clone()
        rest[inside].view(R, N + pad)[:, :N] = math.nan
        assert bool(rest.isnan().all())


@pytest.mark.parametrize("T", (0, 1, 100, 200))
def test_route_without_the_order(T):
    import ctypes
    from tiled_tensor_core_gemm_gb300 import ops
    x = spread_logits(max(T, 1), 48, torch.float32, 430)[:T]
    want = tg.route(x, 5, score="sigmoid", scale=2.5)
    idx, w = torch.full((T + 1, 5), 77, dtype=torch.int32, device="cuda"), torch.full((T + 1, 5), 7.0, device="cuda")
    how = ops.RouteHow(5, 1, 1, 1, 0, 1, 2.5)
    s = torch.cuda.current_stream().cuda_stream
    rc = tg.load_library().gemm_route(T, 48, 0, x.data_ptr(), 48, None, ctypes.byref(how), idx.data_ptr(), w.data_ptr(),
                                      None, None, None, s)
    assert rc == tg.GEMM_OK, tg.gemm_last_error()
    assert torch.equal(idx[:T], want.indices) and torch.equal(w[:T], want.weights)
    assert bool((idx[T:] == 77).all()) and bool((w[T:] == 7.0).all())


@pytest.mark.parametrize("act", ("none", "relu", "gelu"))
def test_scaled_epilogue_of_extreme_sums(act):
    # sums far past the activation's flat ends, and a whole row of zeros
    for M in (4, 150):
        A, sa = made(M, 256, "row", "e4m3", 440)
        B, sb = made(130, 256, "tile", "e4m3", 450)
        sa = sa.clone()
        sa[1], sa[2], sa[3] = 1e6, 0.0, 1e-12
        check_product(tg.gemm_scaled(A, sa, B.t(), sb.t(), act=act), A, B.t(), sa, sb.t(), "f32", act=act)


@pytest.mark.parametrize("rows", (20, 500))
def test_experts_that_share_their_weights(rows):
    E, N, K = 4, 260, 300
    A, sa = made(rows, K, "row", "e4m3", 460)
    W, sw = tg.quantize_block(randn(N, K, seed=461), "tile")
    W, sw = W.t()[None].expand(E, K, N), sw.t()[None].expand(E, 3, 3)
    off = torch.tensor([0, rows // 4, rows // 4 + 3, rows - 7, rows], dtype=torch.int32, device="cuda")
    check_experts(tg.gemm_experts(A, sa, W, sw, off), A, sa, W, sw, off, "f32")
