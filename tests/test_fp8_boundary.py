"""include/moe_fp8.h and include/moe_balance.h without a GPU: the library exports what the headers
declare and every argument error comes back as its status before any launch; the binding refuses what is
no GPU tensor."""
import ctypes
import os
import re

import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
A, B, C, D, E, F, G, H, W = (P(0x10000 * (i + 1)) for i in range(9))
ODD = P(0x10008)   # 8-byte aligned
BAD = P(0x10002)   # 2-byte aligned
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from w4a16_int4_grouped_moe_amd import build

        build.build()
    from w4a16_int4_grouped_moe_amd import _balance, _fp8

    _balance._library()
    return _fp8._library()


def text(header):
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)


def test_declared_entry_points_are_exported(lib):
    fp8 = sorted(set(re.findall(r"\b(moe_fp8_\w+)\s*\(", text("moe_fp8.h"))))
    balance = sorted(set(re.findall(r"\b(moe_balance_\w+)\s*\(", text("moe_balance.h"))))
    assert fp8 == sorted("moe_fp8_" + n for n in (
        "quantize", "dequantize", "matmul", "matmul_workspace_size", "matmul_backward",
        "matmul_backward_workspace_size", "experts_workspace_size", "experts_forward"))
    assert balance == sorted("moe_balance_" + n for n in ("workspace_size", "loss", "loss_backward"))
    for name in fp8 + balance:
        assert hasattr(lib, name), name


def test_constants_match_the_headers():
    for header, names in (("moe_fp8.h", ("MOE_FP8_ROW_BLOCKS", "MOE_FP8_SQUARE_BLOCKS")),
                          ("moe_balance.h", ("MOE_MAX_SEQUENCES",))):
        for name in names:
            assert int(re.search(r"#define %s (\d+)" % name, text(header)).group(1)) == getattr(moe, name)


BAD_MATRICES = [(-1, 128), ((1 << 31) - 255, 128), (4, 0), (4, -16), (4, 24), (4, (1 << 20) + 16)]


@pytest.mark.parametrize("rows,width", BAD_MATRICES)
def test_bad_matrices(lib, rows, width):
    n = ctypes.c_size_t(0)
    s = moe.MOE_ERR_SHAPE
    assert lib.moe_fp8_quantize(A, 0, rows, width, 1, B, C, None) == s
    assert lib.moe_fp8_dequantize(A, B, rows, width, 1, 0, C, None) == s
    assert lib.moe_fp8_matmul_workspace_size(rows, 8, width, 1, ctypes.byref(n)) == s
    assert lib.moe_fp8_matmul(A, B, C, D, 128, rows, 8, width, 0, E, W, BIG, None) == s
    assert lib.moe_fp8_matmul_backward_workspace_size(rows, 8, width, ctypes.byref(n)) == s
    assert lib.moe_fp8_matmul_backward(A, B, C, D, rows, 8, width, 0, E, F, W, BIG, None) == s


@pytest.mark.parametrize("cols", [0, -8, 4, (1 << 31) - 248])
def test_bad_columns(lib, cols):
    n = ctypes.c_size_t(0)
    s = moe.MOE_ERR_SHAPE
    assert lib.moe_fp8_matmul_workspace_size(4, cols, 128, 1, ctypes.byref(n)) == s
    assert lib.moe_fp8_matmul_backward_workspace_size(4, cols, 128, ctypes.byref(n)) == s


def test_largest_sizes(lib):
    n = ctypes.c_size_t(0)
    most = (1 << 31) - 256
    assert lib.moe_fp8_matmul_workspace_size(most, 8, 16, 1, ctypes.byref(n)) == moe.MOE_OK
    assert n.value >= most * 20
    assert lib.moe_fp8_matmul_workspace_size(8, most, 16, 0, ctypes.byref(n)) == moe.MOE_OK
    for rows, cols in ((1 << 20, 8), (8, 1 << 20)):
        assert lib.moe_fp8_matmul_backward_workspace_size(rows, cols, 16, ctypes.byref(n)) == moe.MOE_OK
    for rows, cols in (((1 << 20) + 1, 8), (8, (1 << 20) + 8)):
        assert lib.moe_fp8_matmul_backward_workspace_size(rows, cols, 16, ctypes.byref(n)) == \
            moe.MOE_ERR_SHAPE


def test_quantize_errors(lib):
    def q(x=A, kind=0, rows=4, width=128, block=1, codes=B, scales=C):
        return lib.moe_fp8_quantize(x, kind, rows, width, block, codes, scales, None)

    def d(codes=A, scales=B, rows=4, width=128, block=128, kind=0, out=C):
        return lib.moe_fp8_dequantize(codes, scales, rows, width, block, kind, out, None)

    for call in (q, d):
        for kind in (-1, 3):
            assert call(kind=kind) == moe.MOE_ERR_UNSUPPORTED
        for block in (0, 2, 64, 129, -1):
            assert call(block=block) == moe.MOE_ERR_UNSUPPORTED
        assert call(codes=None) == moe.MOE_ERR_NULL and call(codes=ODD) == moe.MOE_ERR_ALIGNMENT
        assert call(scales=None) == moe.MOE_ERR_NULL and call(scales=BAD) == moe.MOE_ERR_ALIGNMENT
    assert q(x=None) == moe.MOE_ERR_NULL and q(x=ODD) == moe.MOE_ERR_ALIGNMENT
    assert d(out=None) == moe.MOE_ERR_NULL and d(out=ODD) == moe.MOE_ERR_ALIGNMENT
    assert q(x=None, codes=None, scales=None, rows=0) == moe.MOE_OK
    assert d(codes=None, scales=None, out=None, rows=0) == moe.MOE_OK


def test_matmul_errors(lib):
    need = moe.fp8_matmul_workspace_size(100, 64, 128, True)
    assert need >= 100 * 128 + 400

    def call(a=A, sa=None, b=B, sb=C, block=128, rows=100, kind=0, out=D, ws=W, n=need):
        return lib.moe_fp8_matmul(a, sa, b, sb, block, rows, 64, 128, kind, out, ws, n, None)

    for key in ("a", "b", "out", "ws"):
        assert call(**{key: None}) == moe.MOE_ERR_NULL, key
        assert call(**{key: ODD}) == moe.MOE_ERR_ALIGNMENT, key
    assert call(sb=None) == moe.MOE_ERR_NULL and call(sb=BAD) == moe.MOE_ERR_ALIGNMENT
    assert call(sa=BAD) == moe.MOE_ERR_ALIGNMENT
    assert call(n=need - 1) == moe.MOE_ERR_WORKSPACE
    for kind in (moe.MOE_TYPE_FP16, 3, -1):
        assert call(kind=kind) == moe.MOE_ERR_UNSUPPORTED
    assert call(block=64) == moe.MOE_ERR_UNSUPPORTED
    assert call(a=None, b=None, out=None, ws=None, n=0, rows=0) == moe.MOE_OK
    n = ctypes.c_size_t(0)
    assert lib.moe_fp8_matmul_workspace_size(4, 8, 128, 1, None) == moe.MOE_ERR_NULL
    assert moe.fp8_matmul_workspace_size(0, 8, 128, True) == 0
    del n


def test_backward_errors(lib):
    need = moe.fp8_matmul_backward_workspace_size(100, 64, 128)

    def call(d=A, a=B, b=C, sb=D, da=E, db=F, rows=100, kind=0, ws=W, n=need):
        return lib.moe_fp8_matmul_backward(d, a, b, sb, rows, 64, 128, kind, da, db, ws, n, None)

    for key in ("d", "a", "b", "ws"):
        assert call(**{key: None}) == moe.MOE_ERR_NULL, key
    for key in ("d", "a", "b", "da", "db", "ws"):
        assert call(**{key: ODD}) == moe.MOE_ERR_ALIGNMENT, key
    assert call(sb=None) == moe.MOE_ERR_NULL and call(sb=BAD) == moe.MOE_ERR_ALIGNMENT
    assert call(da=None, db=None) == moe.MOE_ERR_NULL
    assert call(n=need - 1) == moe.MOE_ERR_WORKSPACE
    assert call(kind=moe.MOE_TYPE_FP16) == moe.MOE_ERR_UNSUPPORTED
    assert moe.fp8_matmul_backward_workspace_size(0, 64, 128) == 0


def experts(T=4, H=256, I=128, E=8, base=0, k=2):
    return moe.Fp8ExpertsProblem(T, H, I, E, base, k)


@pytest.mark.parametrize("changes,status", [
    (dict(T=-1), "SHAPE"), (dict(H=0), "SHAPE"), (dict(I=0), "SHAPE"), (dict(H=144), "SHAPE"), (dict(I=64), "SHAPE"),
    (dict(H=(1 << 20) + 128), "SHAPE"), (dict(I=(1 << 20) + 128), "SHAPE"), (dict(E=0), "SHAPE"), (dict(E=513), "UNSUPPORTED"),
    (dict(k=0), "SHAPE"), (dict(k=17), "SHAPE"), (dict(base=-1), "SHAPE"), (dict(base=0x7fffffff), "SHAPE"),
    (dict(T=1 << 30, k=2), "SHAPE"), (dict(T=1 << 23, k=1), "UNSUPPORTED")])
def test_bad_experts(lib, changes, status):
    p, n = experts(**changes), ctypes.c_size_t(0)
    want = getattr(moe, "MOE_ERR_" + status)
    assert lib.moe_fp8_experts_workspace_size(ctypes.byref(p), ctypes.byref(n)) == want
    assert lib.moe_fp8_experts_forward(A, B, C, D, E, F, G, H, ctypes.byref(p), W, BIG, None) == want


def test_experts_errors(lib):
    for T in (4, 600):  # the kernels for a few rows, and tiles
        p = experts(T=T)
        need = moe.fp8_experts_workspace_size(T, 256, 128, 8, 2)

        def call(x=A, ids=B, w=C, c13=D, s13=E, c2=F, s2=G, out=H, pp=p, ws=W, n=need):
            return lib.moe_fp8_experts_forward(x, ids, w, c13, s13, c2, s2, out,
                                               ctypes.byref(pp) if pp else None, ws, n, None)

        for key in ("x", "ids", "w", "c13", "s13", "c2", "s2", "out", "ws"):
            assert call(**{key: None}) == moe.MOE_ERR_NULL, key
        for key in ("x", "c13", "c2", "out", "ws"):
            assert call(**{key: ODD}) == moe.MOE_ERR_ALIGNMENT, key
        for key in ("ids", "w", "s13", "s2"):
            assert call(**{key: BAD}) == moe.MOE_ERR_ALIGNMENT, key
        assert call(n=need - 1) == moe.MOE_ERR_WORKSPACE
        assert call(pp=None) == moe.MOE_ERR_NULL
    assert call(x=None, ids=None, ws=None, n=0, pp=experts(T=0)) == moe.MOE_OK
    assert moe.fp8_experts_workspace_size(0, 256, 128, 8, 2) == 0
    # a batch's workspace: its quantised x, h and y at least
    assert moe.fp8_experts_workspace_size(4096, 7168, 2048, 48, 8) > 4096 * 7168 + 32768 * (2048 + 4 * 7168)


def balance(T=100, S=8, k=2, B=1, kind=2):
    return moe.BalanceProblem(T, S, k, B, kind)


@pytest.mark.parametrize("changes,status", [
    (dict(T=-1), "SHAPE"), (dict(S=0), "SHAPE"), (dict(S=1025), "SHAPE"), (dict(k=0), "SHAPE"), (dict(k=9), "SHAPE"),
    (dict(B=0), "SHAPE"), (dict(B=8193), "SHAPE"), (dict(T=1 << 30), "SHAPE"), (dict(kind=3), "UNSUPPORTED"), (dict(kind=-1), "UNSUPPORTED")])
def test_bad_balance(lib, changes, status):
    p, n = balance(**changes), ctypes.c_size_t(0)
    want = getattr(moe, "MOE_ERR_" + status)
    assert lib.moe_balance_workspace_size(ctypes.byref(p), ctypes.byref(n)) == want
    assert lib.moe_balance_loss(A, B, C, D, E, F, G, ctypes.byref(p), W, BIG, None) == want
    assert lib.moe_balance_loss_backward(A, B, C, D, E, F, G, ctypes.byref(p), None) == want


def test_balance_errors(lib):
    for p in (balance(T=100), balance(T=1000), balance(T=1000, B=3)):
        need = moe.balance_workspace_size(p.num_tokens, 8, 2, p.num_sequences)

        def loss(scores=A, ids=B, mask=None, off=C, out=D, counts=E, tokens=F, pp=p, ws=W, n=need):
            return lib.moe_balance_loss(scores, ids, mask, off, out, counts, tokens,
                                        ctypes.byref(pp) if pp else None, ws, n, None)

        def grad(d=A, scores=B, counts=C, tokens=D, mask=None, off=E, out=F, pp=p):
            return lib.moe_balance_loss_backward(d, scores, counts, tokens, mask, off, out,
                                                 ctypes.byref(pp) if pp else None, None)

        for key in ("scores", "ids", "out", "counts", "tokens", "pp"):
            assert loss(**{key: None}) == moe.MOE_ERR_NULL, key
        for key in ("ids", "off", "out", "counts", "tokens"):
            assert loss(**{key: BAD}) == moe.MOE_ERR_ALIGNMENT, key
        assert loss(scores=ODD) == moe.MOE_ERR_ALIGNMENT
        if need:
            assert loss(ws=None) == moe.MOE_ERR_NULL and loss(ws=ODD) == moe.MOE_ERR_ALIGNMENT
            assert loss(n=need - 1) == moe.MOE_ERR_WORKSPACE
        for key in ("d", "scores", "counts", "tokens", "out", "pp"):
            assert grad(**{key: None}) == moe.MOE_ERR_NULL, key
        for key in ("d", "counts", "tokens", "off"):
            assert grad(**{key: BAD}) == moe.MOE_ERR_ALIGNMENT, key
        for key in ("scores", "out"):
            assert grad(**{key: ODD}) == moe.MOE_ERR_ALIGNMENT, key
        if p.num_sequences > 1:
            assert loss(off=None) == moe.MOE_ERR_NULL and grad(off=None) == moe.MOE_ERR_NULL
    assert grad(d=None, scores=None, pp=balance(T=0)) == moe.MOE_OK
    assert moe.balance_workspace_size(128, 1024, 8) == 0 and moe.balance_workspace_size(129, 8, 1) > 0


def test_size_queries_refuse_integers_that_c_would_wrap():
    for call in (lambda: moe.fp8_matmul_workspace_size(1 << 64, 8, 128, True),
                 lambda: moe.fp8_matmul_workspace_size(4, (1 << 32) + 8, 128, True),
                 lambda: moe.fp8_matmul_backward_workspace_size(4, 8, (1 << 32) + 128),
                 lambda: moe.fp8_experts_workspace_size(4, 256, 128, (1 << 32) + 8, 2),
                 lambda: moe.balance_workspace_size(4, 8, (1 << 32) + 2),
                 lambda: moe.balance_workspace_size(4, 8, 2, (1 << 32) + 1)):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_what_is_no_gpu_tensor(lib):
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    for call in (lambda: moe.fp8_quantize(x), lambda: moe.fp8_matmul(x, x), lambda: moe.Fp8(x, x, 1),
                 lambda: moe.fp8_matmul_backward(x, x, x), lambda: moe.fp8_experts_forward(x, x, x, x, x),
                 lambda: moe.balance_loss(x, x), lambda: moe.balance_loss_backward(x, x, x, x, 2)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    for call in (lambda: moe.fp8_quantize([1.0]), lambda: moe.fp8_dequantize(x), lambda: moe.balance_loss(None, x)):
        with pytest.raises(TypeError):
            call()
