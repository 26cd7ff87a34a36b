"""include/moe_ffn.h without a GPU: the library exports what the header declares and every argument
error comes back as its status before any launch; the binding refuses what is no GPU tensor."""
import ctypes
import os
import re

import pytest
import torch

import w4a16_int4_grouped_moe_amd as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
A, B, C, D, E, F, G, W = (P(0x10000 * (i + 1)) for i in range(8))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        from w4a16_int4_grouped_moe_amd import build

        build.build()
    from w4a16_int4_grouped_moe_amd import _ffn

    return _ffn._library()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_ffn.h")).read(),
                  flags=re.S)
    return sorted(set(re.findall(r"\b(moe_(?:ffn|mxfp4)_\w+)\s*\(", text)))


def test_declared_entry_points_are_exported(lib):
    assert declared() == sorted([
        "moe_ffn_workspace_size", "moe_ffn_forward", "moe_ffn_backward", "moe_mxfp4_quantize",
        "moe_mxfp4_dequantize", "moe_mxfp4_matmul", "moe_mxfp4_matmul_workspace_size",
        "moe_mxfp4_ffn_forward"])
    for name in declared():
        assert hasattr(lib, name), name


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "moe_ffn.h")).read()
    for name in ("MOE_TYPE_BF16", "MOE_TYPE_FP16", "MOE_TYPE_FP32", "MOE_FFN_FORWARD",
                 "MOE_FFN_BACKWARD", "MOE_FFN_FORWARD_MXFP4"):
        assert int(re.search(r"#define %s (\d+)" % name, text).group(1)) == getattr(moe, name)


def problem(T=4, H=64, I=32):
    return moe.FfnProblem(T, H, I)


@pytest.mark.parametrize("T,H,I,multiple", [
    (-1, 64, 32, 8), (1 << 31, 64, 32, 8), (4, 0, 32, 8), (4, 64, 0, 8), (4, 60, 32, 8),
    (4, 64, 36, 8), (4, (1 << 20) + 8, 32, 8), (4, 64, (1 << 20) + 8, 8), (4, 40, 32, 32),
    (4, 64, 40, 32)])
def test_bad_sizes(lib, T, H, I, multiple):
    p = problem(T, H, I)
    n = ctypes.c_size_t(0)
    kinds = [moe.MOE_FFN_FORWARD_MXFP4] + ([0, 1] if multiple == 8 else [])
    for kind in kinds:
        assert lib.moe_ffn_workspace_size(ctypes.byref(p), kind, ctypes.byref(n)) == \
            moe.MOE_ERR_SHAPE
    big = 1 << 40
    assert lib.moe_mxfp4_ffn_forward(A, B, C, D, E, F, ctypes.byref(p), W, big, None) == \
        moe.MOE_ERR_SHAPE
    if multiple == 8:
        assert lib.moe_ffn_forward(A, B, C, D, None, ctypes.byref(p), W, big, None) == \
            moe.MOE_ERR_SHAPE
        assert lib.moe_ffn_backward(A, B, C, D, E, F, G, W, ctypes.byref(p), W, big, None) == \
            moe.MOE_ERR_SHAPE


def test_the_largest_token_count(lib):
    n = ctypes.c_size_t(0)
    for kind, width in ((moe.MOE_FFN_FORWARD, 8), (moe.MOE_FFN_BACKWARD, 8),
                        (moe.MOE_FFN_FORWARD_MXFP4, 32)):
        for T, status in (((1 << 31) - 256, moe.MOE_OK), ((1 << 31) - 255, moe.MOE_ERR_SHAPE)):
            p = problem(T, width, width)
            assert lib.moe_ffn_workspace_size(ctypes.byref(p), kind, ctypes.byref(n)) == status
    for rows, status in (((1 << 31) - 256, moe.MOE_OK), ((1 << 31) - 255, moe.MOE_ERR_SHAPE)):
        assert lib.moe_mxfp4_matmul_workspace_size(rows, 8, 32, 1, ctypes.byref(n)) == status


def test_workspace_size_arguments(lib):
    n = ctypes.c_size_t(0)
    p = problem()
    assert lib.moe_ffn_workspace_size(None, 0, ctypes.byref(n)) == moe.MOE_ERR_NULL
    assert lib.moe_ffn_workspace_size(ctypes.byref(p), 0, None) == moe.MOE_ERR_NULL
    for kind in (-1, 3):
        assert lib.moe_ffn_workspace_size(ctypes.byref(p), kind, ctypes.byref(n)) == \
            moe.MOE_ERR_UNSUPPORTED
    assert moe.ffn_workspace_size(0, 64, 32, moe.MOE_FFN_FORWARD) == 0
    # at least the bf16 h, and the bf16 gradients of g and u beside it
    assert moe.ffn_workspace_size(100, 64, 32, moe.MOE_FFN_FORWARD) >= 2 * 100 * 32
    assert moe.ffn_workspace_size(100, 64, 32, moe.MOE_FFN_BACKWARD) >= 6 * 100 * 32
    assert moe.ffn_workspace_size(100, 64, 32, moe.MOE_FFN_FORWARD_MXFP4) >= 100 * 96 * 17 // 32


def test_forward_errors(lib):
    p = problem()
    need = moe.ffn_workspace_size(4, 64, 32, moe.MOE_FFN_FORWARD)
    call = lambda x=A, a=B, b=C, o=D, gu=None, ws=W, n=need, pp=p: lib.moe_ffn_forward(  # noqa: E731
        x, a, b, o, gu, ctypes.byref(pp) if pp else None, ws, n, None)
    assert call(pp=None) == moe.MOE_ERR_NULL
    for key in ("x", "a", "b", "o", "ws"):
        assert call(**{key: None}) == moe.MOE_ERR_NULL, key
        assert call(**{key: P(0x10008)}) == moe.MOE_ERR_ALIGNMENT, key
    assert call(gu=P(0x10004)) == moe.MOE_ERR_ALIGNMENT
    assert call(n=need - 1) == moe.MOE_ERR_WORKSPACE
    assert call(x=None, pp=problem(T=0)) == moe.MOE_OK


def test_backward_errors(lib):
    p = problem()
    need = moe.ffn_workspace_size(4, 64, 32, moe.MOE_FFN_BACKWARD)

    def call(d=A, x=B, gu=C, a=D, b=E, dx=F, da=G, db=W, ws=P(0x200000), n=need, pp=p):
        return lib.moe_ffn_backward(d, x, gu, a, b, dx, da, db, ctypes.byref(pp), ws, n, None)

    for key in ("d", "x", "gu", "a", "b", "ws", "da", "db"):
        assert call(**{key: None}) == moe.MOE_ERR_NULL, key
    for key in ("d", "x", "gu", "a", "b", "ws", "dx", "da", "db"):
        assert call(**{key: P(0x10008)}) == moe.MOE_ERR_ALIGNMENT, key
    assert call(dx=None, da=None, db=None) == moe.MOE_ERR_NULL
    assert call(n=need - 1) == moe.MOE_ERR_WORKSPACE


def test_mxfp4_errors(lib):
    q = lambda x=A, t=0, r=4, w=64, c=B, s=C: lib.moe_mxfp4_quantize(x, t, r, w, c, s, None)  # noqa: E731
    d = lambda c=A, s=B, r=4, w=64, t=0, o=C: lib.moe_mxfp4_dequantize(c, s, r, w, t, o, None)  # noqa: E731
    for f in (q, d):
        for bad in (dict(r=-1), dict(r=1 << 31), dict(w=0), dict(w=48), dict(w=(1 << 20) + 32)):
            assert f(**bad) == moe.MOE_ERR_SHAPE, bad
        for t in (-1, 3):
            assert f(t=t) == moe.MOE_ERR_UNSUPPORTED
        assert f(r=0) == moe.MOE_OK
        assert f(c=None) == moe.MOE_ERR_NULL and f(s=None) == moe.MOE_ERR_NULL
        assert f(c=P(0x10008)) == moe.MOE_ERR_ALIGNMENT
    assert q(x=None) == moe.MOE_ERR_NULL and d(o=None) == moe.MOE_ERR_NULL


def test_matmul_errors(lib):
    need = moe.mxfp4_matmul_workspace_size(40, 8, 64, True)
    assert need >= 40 * 64 * 17 // 32
    assert moe.mxfp4_matmul_workspace_size(0, 8, 64, True) == 0

    def call(a=A, sa=None, b=B, sb=C, m=40, n=8, k=64, t=0, o=D, ws=W, nb=need):
        return lib.moe_mxfp4_matmul(a, sa, b, sb, m, n, k, t, o, ws, nb, None)

    for bad in (dict(m=-1), dict(n=0), dict(n=12), dict(k=16), dict(m=1 << 31)):
        assert call(**bad) == moe.MOE_ERR_SHAPE, bad
    assert call(t=1) == moe.MOE_ERR_UNSUPPORTED and call(t=7) == moe.MOE_ERR_UNSUPPORTED
    for key in ("a", "b", "sb", "o", "ws"):
        assert call(**{key: None}) == moe.MOE_ERR_NULL, key
    for key in ("a", "b", "o", "ws"):
        assert call(**{key: P(0x10008)}) == moe.MOE_ERR_ALIGNMENT, key
    assert call(nb=need - 1) == moe.MOE_ERR_WORKSPACE
    assert call(m=0, a=None) == moe.MOE_OK
    with pytest.raises(ValueError):
        moe.mxfp4_matmul_workspace_size(4, 9, 64, True)


def test_mxfp4_ffn_errors(lib):
    p = problem()
    need = moe.ffn_workspace_size(4, 64, 32, moe.MOE_FFN_FORWARD_MXFP4)

    def call(x=A, a=B, sa=C, b=D, sb=E, o=F, ws=W, n=need, pp=p):
        return lib.moe_mxfp4_ffn_forward(x, a, sa, b, sb, o, ctypes.byref(pp), ws, n, None)

    for key in ("x", "a", "sa", "b", "sb", "o", "ws"):
        assert call(**{key: None}) == moe.MOE_ERR_NULL, key
    for key in ("x", "a", "b", "o", "ws"):
        assert call(**{key: P(0x10008)}) == moe.MOE_ERR_ALIGNMENT, key
    assert call(n=need - 1) == moe.MOE_ERR_WORKSPACE
    assert call(x=None, pp=problem(T=0)) == moe.MOE_OK


def test_binding_refuses_sizes_past_a_c_int(lib):
    big = (1 << 32) + 64  # would be 64
    for args in ((4, big, 32), (4, 64, big)):
        with pytest.raises(ValueError):
            moe.ffn_workspace_size(*args, moe.MOE_FFN_FORWARD)
    for args in ((4, big, 64), (4, 64, big)):
        with pytest.raises(ValueError):
            moe.mxfp4_matmul_workspace_size(*args, True)


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.ffn_forward(x, torch.zeros(64, 64, dtype=torch.bfloat16), x)
    with pytest.raises(ValueError):
        moe.mxfp4_quantize(x)
    with pytest.raises(ValueError):
        moe.Mxfp4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(TypeError):
        moe.mxfp4_dequantize(x)
    with pytest.raises(TypeError):
        moe.ffn_forward(None, x, x)
