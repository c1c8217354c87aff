"""The expert-layer operators without a GPU: what the C entries and the Python
functions refuse, before any CUDA call, and what they do for nothing."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import tiled_tensor_core_gemm_gb300 as tg
from tiled_tensor_core_gemm_gb300 import build as tgbuild
from tiled_tensor_core_gemm_gb300 import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAD = tg.GEMM_ERR_INVALID_ARG
P = 1 << 20      # an aligned address no call below gets to touch


@pytest.fixture(scope="module")
def lib():
    tgbuild.build()
    return tg.load_library()


def refused(rc, frag):
    assert rc == BAD, rc
    assert frag in tg.gemm_last_error(), tg.gemm_last_error()


def test_every_declared_entry_is_bound(lib):
    text = open(os.path.join(ROOT, "include", "gemm_ops.h")).read()
    names = set(re.findall(r"GEMM_API int (gemm_\w+)\(", text))
    assert len(names) == 7 and names <= set(tg.EXPORTED)
    for n in names:
        assert getattr(lib, n).argtypes is not None


# ---------------------------------------------------------------- quantise ---
def quant(lib, batch=1, rows=256, cols=256, type_=0, X=P, ldx=256, xs=0, block=0, to=tg.GEMM_E4M3, Q=P << 4, ldq=256,
          qs=0, S=P << 6, s_row=1, s_col=256, s_batch=0, slots=None, copies=1, out_rows=0):
    return lib.gemm_quantize_block(batch, rows, cols, type_, X, ldx, xs, block, to, Q, ldq, qs, S, s_row, s_col,
                                   s_batch, slots, copies, out_rows, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(type_=3), "element type"), (dict(to=tg.GEMM_BF16), "E4M3"), (dict(block=3), "block"),
    (dict(rows=-1), "size"), (dict(rows=1 << 31), "size"), (dict(ldx=255), "leading"), (dict(ldq=255), "leading"),
    (dict(X=0), "X is NULL"), (dict(Q=0), "Q is NULL"), (dict(S=0), "S is NULL"), (dict(X=P + 2), "aligned"),
    (dict(S=P + 1), "aligned"), (dict(Q=P + 64), "overlap"), (dict(s_row=0), "scales overlap"),
    (dict(s_row=1, s_col=1), "scales overlap"), (dict(s_col=-1), "stride"),
    (dict(batch=2), "overlap"), (dict(block=1, slots=P), "slots need"), (dict(slots=P << 8, copies=0), "copies"),
    (dict(slots=P << 8, out_rows=-1), "copies or out_rows"),
])
def test_quantize_refuses(lib, kw, frag):
    refused(quant(lib, **kw), frag)


@pytest.mark.parametrize("kw", [dict(rows=0), dict(cols=0), dict(batch=0), dict(slots=P << 8, out_rows=0)])
def test_quantize_of_nothing(lib, kw):
    assert quant(lib, **kw) == tg.GEMM_OK


# ---------------------------------------------------------------- products ---
def bs(scale=P << 8, sk=1024, si=1, block=1):
    return ctypes.byref(ops.BlockScale(scale, sk, si, block, 0))


def scaled(lib, M=64, N=64, K=256, dtype=tg.GEMM_E4M3, A=P, lda=256, am=0, sa=None, B=P << 4, ldb=256, bm=1, sb=None,
           C=P << 6, ldc=64, epi=None):
    return lib.gemm_run_scaled(M, N, K, dtype, A, lda, am, sa or bs(), B, ldb, bm, sb or bs(P << 9), C, ldc, epi, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(dtype=tg.GEMM_BF16), "E4M3"), (dict(M=-1), "size"), (dict(K=1 << 31), "size"), (dict(am=2), "a_major"),
    (dict(lda=255), "leading"), (dict(bm=0, ldb=63), "leading"), (dict(ldc=63), "leading"),
    (dict(A=0), "A is NULL"), (dict(B=0), "B is NULL"), (dict(C=0), "C is NULL"), (dict(C=P + 64), "overlap"),
    (dict(C=(P << 6) + 2), "aligned"), (dict(sa=bs(block=2)), "a_scale"), (dict(sb=bs(sk=-1)), "b_scale"),
    (dict(sa=bs(scale=0)), "a_scale is NULL"), (dict(sb=bs(scale=P << 6)), "overlap"),
])
def test_scaled_refuses(lib, kw, frag):
    refused(scaled(lib, **kw), frag)


def test_scaled_refuses_a_bad_epilogue(lib):
    e = tg.make_epilogue()
    e.activation = 9
    refused(scaled(lib, epi=ctypes.byref(e)), "activation")


def test_scaled_of_nothing(lib):
    assert scaled(lib, M=0) == tg.GEMM_OK
    assert scaled(lib, N=0) == tg.GEMM_OK


def experts(lib, rows=64, N=64, K=256, E=4, dtype=tg.GEMM_E4M3, A=P, lda=256, sa=None, off=P << 10, B=P << 4, ldb=256,
            be=64 * 256, bm=1, sb=None, sbe=2, C=P << 6, ldc=64, epi=None):
    return lib.gemm_run_experts(rows, N, K, E, dtype, A, lda, sa or bs(), off, B, ldb, be, bm, sb or bs(P << 9), sbe, C,
                                ldc, epi, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(dtype=0), "E4M3"), (dict(rows=-1), "size"), (dict(E=0), "experts"), (dict(E=1025), "experts"),
    (dict(bm=2), "b_major"), (dict(lda=255), "leading"), (dict(sa=bs(block=128)), "a_scale"),
    (dict(off=0), "offsets is NULL"), (dict(off=(P << 10) + 2), "aligned"), (dict(be=-16), "b_expert"),
    (dict(C=P), "overlap"), (dict(sbe=-1), "b_scale"),
])
def test_experts_refuses(lib, kw, frag):
    refused(experts(lib, **kw), frag)


def test_experts_refuses_weights_tma_cannot_address(lib):
    for kw in (dict(B=(P << 4) + 8), dict(ldb=257, be=64 * 257), dict(be=64 * 256 + 8)):
        assert experts(lib, **kw) == tg.GEMM_ERR_UNSUPPORTED
        assert "16 bytes" in tg.gemm_last_error()


def test_experts_takes_no_bias_and_no_beta(lib):
    for e in (tg.make_epilogue(beta=1.0), tg.make_epilogue(bias=P)):
        refused(experts(lib, epi=ctypes.byref(e)), "beta = 0")


# ------------------------------------------------------------------- route ---
def how(top_k=2, score=0, groups=1, top_groups=1, group_score=0, renorm=1, scale=1.0):
    return ctypes.byref(ops.RouteHow(top_k, score, groups, top_groups, group_score, renorm, scale))


def route(lib, T=4, E=16, type_=0, L=P, ldl=16, bias=None, h=None, ix=P << 2, w=P << 3, off=P << 4, order=P << 5,
          slots=P << 6):
    return lib.gemm_route(T, E, type_, L, ldl, bias, h or how(), ix, w, off, order, slots, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(type_=7), "element type"), (dict(T=-1), "tokens"), (dict(E=0), "experts"), (dict(E=1025, ldl=1025), "experts"),
    (dict(ldl=15), "leading"), (dict(h=how(top_k=0)), "top_k"), (dict(h=how(top_k=17)), "top_k"),
    (dict(E=64, ldl=64, h=how(top_k=33)), "top_k"), (dict(h=how(score=2)), "score"), (dict(h=how(groups=3)), "groups"),
    (dict(h=how(groups=0)), "groups"), (dict(h=how(groups=4, top_groups=5)), "top_groups"),
    (dict(h=how(groups=4, top_groups=0)), "top_groups"), (dict(h=how(groups=8, top_groups=1, top_k=3)), "top_k"),
    (dict(h=how(group_score=2)), "group score"), (dict(L=0), "logits is NULL"), (dict(ix=0), "indices is NULL"),
    (dict(off=None), "all given"), (dict(slots=None), "all given"), (dict(order=P << 6), "overlap"),
    (dict(bias=P + 2), "aligned"),
])
def test_route_refuses(lib, kw, frag):
    refused(route(lib, **kw), frag)


def test_route_refuses_no_rules(lib):
    refused(lib.gemm_route(4, 16, 0, P, 16, None, None, P << 2, P << 3, None, None, None, None), "how is NULL")


def test_route_of_no_tokens_without_the_order(lib):
    assert route(lib, T=0, off=None, order=None, slots=None) == tg.GEMM_OK


def test_route_backward_refuses(lib):
    def call(**kw):
        a = dict(T=4, E=16, L=P, ldl=16, ix=P << 2, g=P << 3, d=P << 4, ldd=16, h=how())
        a.update(kw)
        return lib.gemm_route_backward(a["T"], a["E"], 0, a["L"], a["ldl"], a["h"], a["ix"], a["g"], a["d"], a["ldd"],
                                       None)
    refused(call(ldd=15), "leading")
    refused(call(d=P), "overlap")
    refused(call(g=0), "grad is NULL")
    assert call(T=0) == tg.GEMM_OK


# ----------------------------------------------------------------- combine ---
def combine(lib, T=4, k=2, H=64, R=8, type_=1, Y=P, ldy=64, slots=P << 4, w=P << 5, out=P << 6, ldo=64):
    return lib.gemm_combine(T, k, H, R, type_, Y, ldy, slots, w, out, ldo, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(type_=4), "element type"), (dict(T=-1), "size"), (dict(k=0), "top_k"), (dict(ldy=63), "leading"),
    (dict(ldo=63), "leading"), (dict(Y=0), "Y is NULL"), (dict(slots=0), "slots is NULL"), (dict(out=P + 2), "overlap"),
    (dict(Y=P + 1), "aligned"), (dict(out=0), "out is NULL"),
])
def test_combine_refuses(lib, kw, frag):
    refused(combine(lib, **kw), frag)


def test_combine_of_nothing(lib):
    assert combine(lib, T=0) == tg.GEMM_OK
    assert combine(lib, H=0, ldy=0, ldo=0) == tg.GEMM_OK


def test_combine_backward_refuses(lib):
    def call(**kw):
        a = dict(T=4, k=2, H=64, R=8, g=P, ldg=64, Y=P << 1, ldy=64, s=P << 2, w=P << 3, o=P << 4, d=P << 5, ldd=64,
                 dw=P << 6)
        a.update(kw)
        return lib.gemm_combine_backward(a["T"], a["k"], a["H"], a["R"], 1, a["g"], a["ldg"], a["Y"], a["ldy"], a["s"],
                                         a["w"], a["o"], a["d"], a["ldd"], a["dw"], None)
    refused(call(R=9), "order needs")
    refused(call(w=0), "weights is NULL")
    refused(call(d=P << 1), "overlap")
    refused(call(ldg=63), "leading")
    assert call(T=0, R=0) == tg.GEMM_OK


# ------------------------------------------------------------------ Python ---
def test_tensors_on_the_host_are_refused():
    f8 = torch.zeros(4, 128, dtype=torch.float8_e4m3fn)
    s = torch.zeros(4, 1)
    for call in (lambda: tg.quantize_block(torch.zeros(4, 4)),
                 lambda: tg.gemm_scaled(f8, s, f8.t(), s.t()),
                 lambda: tg.gemm_experts(f8, s, f8[None].transpose(1, 2), s[None].transpose(1, 2),
                                         torch.zeros(2, dtype=torch.int32)),
                 lambda: tg.route(torch.zeros(4, 8), 2),
                 lambda: tg.route_backward(torch.zeros(4, 2), torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)),
                 lambda: tg.combine(torch.zeros(4, 8), torch.zeros(2, 2, dtype=torch.int32)),
                 lambda: tg.combine_backward(torch.zeros(2, 8), torch.zeros(4, 8), torch.zeros(2, 2, dtype=torch.int32),
                                             torch.zeros(2, 2))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_types_are_refused():
    f8, s = torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.zeros(4, 1)
    with pytest.raises(TypeError):
        tg.quantize_block(torch.zeros(4, 4, dtype=torch.int32))
    with pytest.raises(TypeError):
        tg.quantize_block(torch.zeros(4, 4), dtype="bf16")
    with pytest.raises(TypeError):
        tg.gemm_scaled(f8, s, f8.t().to(torch.float8_e5m2), s.t())
    with pytest.raises(TypeError):
        tg.gemm_scaled(torch.zeros(4, 128), s, torch.zeros(128, 4), s.t())
    with pytest.raises(TypeError):
        tg.route(torch.zeros(4, 8, dtype=torch.float64), 2)
    with pytest.raises(TypeError):
        tg.combine(torch.zeros(4, 8, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32))


def test_majors_of_views():
    t = torch.zeros(40, 32)
    assert ops._major("t", t[:, :20]) == (32, 0)
    assert ops._major("t", t[:, :20].t()) == (32, 1)
    assert ops._major("t", t[:1, :20]) == (20, 0)
    assert ops._major("t", t[:, :1]) == (32, 0)
    assert ops._major("t", t[:, :1].t()) == (1, 0) or ops._major("t", t[:, :1].t()) == (32, 1)
    with pytest.raises(ValueError):
        ops._major("t", t[:, ::2])


# ------------------------------------------- one row (or column) expanded ---
def test_row_pitch_of_an_expanded_row():
    row = torch.zeros(1, 64)
    z = torch.zeros(5, 64, requires_grad=True)
    kept = []
    z.register_hook(kept.append)
    z.sum(0).backward(torch.ones(64))
    assert kept[0].stride() == (0, 1)             # what autograd hands back from a sum over the rows
    for t in (row.expand(4096, 64), kept[0], torch.zeros(1, 1).expand(6, 1)):
        assert ops._rows("t", t, *t.shape, True) == 0
        with pytest.raises(ValueError, match="t must have rows of its own"):
            ops._rows("t", t, *t.shape)
    assert ops._rows("t", row, 1, 64) == 64
    assert ops._rows("t", torch.zeros(3, 64)[:, :7], 3, 7) == 64
    assert ops._rows("t", torch.zeros(1, 0).expand(4, 0), 4, 0) == 1


def test_majors_of_expanded_matrices_are_refused():
    one = torch.zeros(1, 1)
    for t in (one.expand(6, 1), one.expand(1, 6), torch.zeros(1, 64).expand(6, 64), torch.zeros(64, 1).expand(64, 6),
              torch.zeros(2, 1, 1).expand(2, 6, 1)):
        with pytest.raises(ValueError, match="not expanded"):
            ops._major("t", t)
    assert ops._major("t", torch.zeros(6, 1)) == (1, 0)
    assert ops._major("t", torch.zeros(1, 0).expand(6, 0)) == (1, 0)


def test_a_pitch_of_zero_is_for_matrices_that_are_only_read(lib):
    def backward(**kw):
        a = dict(ldg=64, ldy=64, ldd=64)
        a.update(kw)
        return lib.gemm_combine_backward(4, 2, 64, 8, 1, P, a["ldg"], P << 1, a["ldy"], P << 2, P << 3, P << 4, P << 5,
                                         a["ldd"], P << 6, None)

    def route_backward(ldl, ldd):
        return lib.gemm_route_backward(4, 16, 0, P, ldl, how(), P << 2, P << 3, P << 4, ldd, None)
    for call in (lambda: quant(lib, ldx=0), lambda: route(lib, ldl=0), lambda: route_backward(0, 16),
                 lambda: combine(lib, ldy=0), lambda: backward(ldg=0), lambda: backward(ldy=0)):
        assert call() != tg.GEMM_OK               # (the addresses are no device's)
        assert "leading" not in tg.gemm_last_error()
    for call in (lambda: quant(lib, ldq=0), lambda: route_backward(16, 0), lambda: combine(lib, ldo=0),
                 lambda: backward(ldd=0), lambda: scaled(lib, lda=0), lambda: scaled(lib, ldc=0),
                 lambda: experts(lib, lda=0), lambda: experts(lib, ldc=0)):
        refused(call(), "leading")


def test_experts_of_one_stored_row_have_no_pitch(lib):
    # N = 1, K-major, and K = 1, N-major, at extents that are no multiple of 16
    for kw in (dict(N=1, K=100, lda=112, ldb=100, be=112, ldc=1), dict(N=77, K=1, lda=16, ldb=77, be=80, bm=0, ldc=77)):
        rc = experts(lib, **kw)
        assert rc != tg.GEMM_ERR_UNSUPPORTED and "16 bytes" not in tg.gemm_last_error()
    assert experts(lib, N=1, K=100, lda=112, ldb=100, be=100, ldc=1) == tg.GEMM_ERR_UNSUPPORTED
    assert experts(lib, N=2, K=100, lda=112, ldb=100, be=256, ldc=2) == tg.GEMM_ERR_UNSUPPORTED


# The blocks a shifted load touches (from the aligned address at or before the first element, 16 bytes at a
# time, while they hold an element), for every chunk of eight of the last row, against the allocation's end.
ACCESS_PROGRAM = r"""
#include "ops.h"
#include <cstdio>
using namespace tcgemm;
int main() {
    const uint64_t base = 1 << 20;
    long exact = 0, shifted = 0;
    for (int elem = 2; elem <= 4; elem += 2)
        for (int off = 0; off < 16; off += elem)
            for (int cols = 1; cols <= 40; ++cols)
                for (int slack = 0; slack <= 20; ++slack) {
                    OpSpan s = {"X", reinterpret_cast<void *>(base + off), (uint64_t)cols * elem, elem, false};
                    s.memory_end = base + off + s.bytes + slack;
                    uint64_t last = 0;
                    for (int c = 0; c < cols; c += 8) {
                        const uint64_t at = base + off + (uint64_t)c * elem, have = cols - c < 8 ? cols - c : 8;
                        for (uint64_t b = at & ~15ull; b < at + have * elem; b += 16) last = b + 16;
                    }
                    const int how = op_access(false, &s, 1);
                    if (op_access(true, &s, 1) != kOpWide || how != (last > s.memory_end ? kOpExact : kOpShifted)) {
                        printf("elem %d off %d cols %d slack %d: %d\n", elem, off, cols, slack, how);
                        return 1;
                    }
                    ++(how == kOpExact ? exact : shifted);
                }
    OpSpan two[2] = {{"Y", reinterpret_cast<void *>(base), 64, 2, false}, {"Z", reinterpret_cast<void *>(base + 128), 10, 2, false}};
    two[0].memory_end = two[1].memory_end = base + 138;
    if (op_access(false, two, 1) != kOpShifted || op_access(false, two, 2) != kOpExact) return 1;
    two[1].bytes = 0;
    if (op_access(false, two, 2) != kOpShifted) return 1;
    printf("%ld exact, %ld shifted\n", exact, shifted);
    return exact && shifted ? 0 : 1;
}
"""


def test_shifted_loads_are_not_taken_past_the_end_of_an_allocation(tmp_path):
    src = tmp_path / "access.cpp"
    src.write_text(ACCESS_PROGRAM)
    cuda = os.path.dirname(os.path.dirname(tgbuild._nvcc()))
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "tiled_tensor_core_gemm_gb300", "csrc"),
                    "-I", os.path.join(cuda, "include"), str(src), "-o", str(tmp_path / "access")], check=True)
    run = subprocess.run([str(tmp_path / "access")], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout


# ------------------------------------------------ footprints past 64 bits ---
FAR = (1 << 28) + 1        # rows that, 2^36 elements apart, come round to the first one in 64 bits
LD = 1 << 36


def test_footprints_that_do_not_fit_64_bits_are_refused(lib):
    q = dict(rows=FAR, X=1 << 20, Q=1 << 50, S=1 << 54, s_col=1 << 29)
    far = [
        quant(lib, ldx=LD, **q), quant(lib, ldq=LD, **q), quant(lib, block=2, batch=2, qs=1 << 46, s_batch=1 << 46,
                                                                 **dict(q, s_row=LD, s_col=1, ldq=1 << 10)),
    ]
    assert far == [BAD] * 3
    for kw, frag in ((dict(ldx=LD), "X: extent"), (dict(ldq=LD), "Q: extent"), (dict(batch=1 << 15, xs=1 << 46, rows=256,
                     qs=1 << 17, s_batch=1 << 31, type_=0), "X: extent"), (dict(s_row=LD), "S: extent")):
        refused(quant(lib, **dict(q, **kw)), frag)
    refused(combine(lib, T=1, R=FAR, ldy=LD), "Y: extent")
    refused(combine(lib, T=FAR, ldo=LD), "out: extent")
    refused(route(lib, T=FAR, ldl=LD), "logits: extent")
    refused(scaled(lib, M=FAR, lda=LD), "A: extent")
    refused(scaled(lib, N=FAR, ldc=1 << 29, ldb=LD), "B: extent")
    refused(scaled(lib, M=FAR, ldc=LD), "C: extent")
    refused(scaled(lib, M=FAR, sa=bs(si=LD)), "a_scale: extent")
    refused(scaled(lib, N=FAR, ldc=1 << 29, sb=bs(P << 9, si=LD)), "b_scale: extent")
    refused(experts(lib, N=FAR, ldb=LD, ldc=1 << 29, E=2), "B: extent")
    refused(experts(lib, rows=FAR, sa=bs(si=LD)), "a_scale: extent")
