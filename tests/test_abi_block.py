"""C-ABI checks of the router's and the norm's calls that need no GPU: both
builds export every symbol of include/libmxmoe_block.h, and invalid arguments
are refused before anything is launched, by the entry points and by the
binding."""
import ctypes
import os
import re

import pytest
import torch

import mxfp8_block_scaled_04_amd as mx
from mxfp8_block_scaled_04_amd import block as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "libmxmoe_block.h")

# tests/test_sanitize_block.py runs this module against a sanitizer build of
# the entry points (kernel launchers stubbed out) named by MXMOE_BLOCK_LIB
SAN = os.environ.get("MXMOE_BLOCK_LIB")
if SAN:
    mx._lib = ctypes.CDLL(SAN)

P = ctypes.c_void_p
FAKE = P(0x100000)  # never dereferenced: every call below fails validation first
OK, NULL, SHAPE, ALIGN, CAPACITY, UNSUPPORTED = 0, 1, 2, 3, 4, 5


def _header_names():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(mx_[a-z_0-9]+)\s*\(", src)))


def test_every_header_symbol_is_exported():
    names = _header_names()
    assert sorted(mx.BLOCK_SYMBOLS) == names
    libs = [B._lib()] if SAN else [B._lib(), mx.open_library(mx.DEBUG_LIB_PATH)]
    for lib in libs:
        for n in names:
            assert hasattr(lib, n), n


def _variants(call, good):
    """Call with one argument (or several) replaced."""
    def f(**kw):
        args = list(good)
        for i, v in kw.items():
            args[int(i[1:])] = v
        return call(*args)
    return f


def test_router_refusals():
    # (logits, ldl, T, E, bias, groups, kept, top, k, scale, flags, experts, weights, scores, stream)
    f = _variants(B._lib().mx_router, (FAKE, 64, 5, 64, FAKE, 4, 2, 2, 8, 1.0, 0, FAKE, FAKE, FAKE, None))
    assert f(a1=63) == SHAPE and f(a2=-1) == SHAPE and f(a3=0) == SHAPE
    assert f(a1=5000, a3=4097, a5=1, a6=1) == SHAPE
    assert f(a5=0) == SHAPE and f(a5=3) == SHAPE and f(a5=128, a3=128, a1=128) == SHAPE
    assert f(a6=0) == SHAPE and f(a6=5) == SHAPE and f(a7=0) == SHAPE and f(a7=3) == SHAPE
    assert f(a8=0) == SHAPE and f(a8=65, a5=1, a6=1, a3=128, a1=128) == SHAPE
    assert f(a8=33) == SHAPE  # more than the experts of the groups kept
    assert f(a9=float("nan")) == SHAPE and f(a9=float("inf")) == SHAPE and f(a10=8) == SHAPE
    assert f(a2=1 << 24) == UNSUPPORTED and f(a1=1 << 32) == UNSUPPORTED
    assert f(a2=0, a3=3000, a1=3000, a5=60, a6=60) == OK  # 50 experts in each of 64 group places
    assert f(a3=4092, a1=4092, a5=33, a6=33) == UNSUPPORTED  # 124 experts in each of 64 group places
    for i in (0, 11, 12):
        assert f(**{f"a{i}": None}) == NULL
        assert f(**{f"a{i}": P(0x100002)}) == ALIGN
    for i in (4, 13):
        assert f(**{f"a{i}": P(0x100002)}) == ALIGN
    assert f(a0=P(0x100001), a10=4) == ALIGN
    assert f(a2=0, a0=None, a11=None, a12=None) == OK


def test_router_scores_in_the_place_of_logits_are_refused():
    """(The router reads logits again after it has written scores.)"""
    f = _variants(B._lib().mx_router, (FAKE, 64, 5, 64, FAKE, 4, 2, 2, 8, 1.0, 0, FAKE, FAKE, FAKE, None))
    assert f() == SHAPE


def test_router_backward_refusals():
    # (logits, ldl, T, E, experts, dweights, dscores, k, scale, flags, dlogits, ldd, stream)
    f = _variants(B._lib().mx_router_backward, (FAKE, 64, 5, 64, FAKE, FAKE, FAKE, 8, 1.0, 0, FAKE, 64, None))
    assert f(a1=63) == SHAPE and f(a11=63) == SHAPE and f(a2=-1) == SHAPE and f(a3=0) == SHAPE
    assert f(a7=0) == SHAPE and f(a7=65, a3=128, a1=128, a11=128) == SHAPE and f(a7=5, a3=4) == SHAPE
    assert f(a8=float("nan")) == SHAPE and f(a9=8) == SHAPE
    assert f(a2=1 << 24) == UNSUPPORTED and f(a1=1 << 32) == UNSUPPORTED and f(a11=1 << 32) == UNSUPPORTED
    for i in (0, 4, 5, 10):
        assert f(**{f"a{i}": None}) == NULL
        assert f(**{f"a{i}": P(0x100002)}) == ALIGN
    assert f(a6=P(0x100002)) == ALIGN and f(a10=P(0x100001), a9=4) == ALIGN
    assert f(a2=0, a0=None, a10=None) == OK


def test_combine_gradient_refusals():
    # (dout, ldd, y, M, ldy, slot_of, T, k, N, dweights, stream)
    f = _variants(B._lib().mx_combine_dweights, (FAKE, 64, FAKE, 10, 64, FAKE, 5, 2, 64, FAKE, None))
    assert f(a1=56) == SHAPE and f(a4=56) == SHAPE and f(a3=-1) == SHAPE and f(a6=-1) == SHAPE
    assert f(a7=0) == SHAPE and f(a8=-8) == SHAPE
    assert f(a1=68) == ALIGN and f(a4=68) == ALIGN
    assert f(a8=60) == UNSUPPORTED and f(a6=1 << 24) == UNSUPPORTED
    assert f(a6=1 << 20, a7=1 << 12) == UNSUPPORTED and f(a3=1 << 31) == UNSUPPORTED
    for i in (0, 2, 5, 9):
        assert f(**{f"a{i}": None}) == NULL
    for i in (0, 2):
        assert f(**{f"a{i}": P(0x100008)}) == ALIGN
    for i in (5, 9):
        assert f(**{f"a{i}": P(0x100002)}) == ALIGN
    assert f(a6=0, a0=None, a5=None, a9=None) == OK


def test_norm_refusals():
    # (x, ldx, residual, ldr, weight, M, N, eps, flags, h, ldh, y, ldy, q, s, rstd, stream)
    f = _variants(B._lib().mx_rms_norm,
                  (FAKE, 64, FAKE, 64, FAKE, 5, 64, 1e-6, 0, FAKE, 64, FAKE, 64, FAKE, FAKE, FAKE, None))
    assert f(a5=-1) == SHAPE and f(a6=60) == SHAPE and f(a6=0) == SHAPE
    for i in (1, 3, 10, 12):
        assert f(**{f"a{i}": 56}) == SHAPE
        assert f(**{f"a{i}": 68}) == ALIGN
        assert f(**{f"a{i}": 1 << 30}) == UNSUPPORTED
    assert f(a7=-1e-6) == SHAPE and f(a7=float("nan")) == SHAPE and f(a7=float("inf")) == SHAPE and f(a8=4) == SHAPE
    assert f(a6=40) == SHAPE  # codes in blocks of 32
    assert f(a2=None) == SHAPE  # h without a residual
    assert f(a9=None) == NULL and f(a0=None) == NULL and f(a4=None) == NULL
    assert f(a13=None) == NULL and f(a14=None) == NULL
    big = {f"a{i}": 40000 for i in (1, 3, 6, 10, 12)}
    assert f(**big) == UNSUPPORTED and f(a5=1 << 31) == UNSUPPORTED
    for i in (0, 2, 4, 9, 11, 13):
        assert f(**{f"a{i}": P(0x100008)}) == ALIGN
    for i in (14, 15):
        assert f(**{f"a{i}": P(0x100002)}) == ALIGN
    assert f(a5=0, a0=None, a4=None) == OK


def test_norm_backward_refusals():
    # (dy, ldy, dy2, ldy2, h, ldh, weight, rstd, dh_in, ldi, M, N, flags, dh, ldo, dx, lddx, dweight, fp32, accumulate,
    #  workspace, bytes, stream)
    lib = B._lib()
    M = 5000
    size = lib.mx_rms_norm_backward_workspace_bytes(M, 64)
    assert size > 0 and size % (4 * 64) == 0
    f = _variants(lib.mx_rms_norm_backward, (FAKE, 64, FAKE, 64, FAKE, 64, FAKE, FAKE, FAKE, 64, M, 64, 1, FAKE, 64,
                                             FAKE, 64, FAKE, 1, 0, FAKE, size, None))
    assert f(a10=-1) == SHAPE and f(a11=60) == SHAPE and f(a12=4) == SHAPE
    for i in (1, 3, 5, 9, 14, 16):
        assert f(**{f"a{i}": 56}) == SHAPE
        assert f(**{f"a{i}": 68}) == ALIGN
    assert f(a12=0) == SHAPE  # dx of a bf16 stream
    assert f(a18=2) == SHAPE and f(a19=-1) == SHAPE and f(a21=-1) == SHAPE
    assert f(a18=0, a19=1) == UNSUPPORTED  # added to bf16
    assert f(a21=size - 1) == CAPACITY and f(a20=None) == NULL
    for i in (0, 4, 6, 7, 13):
        assert f(**{f"a{i}": None}) == NULL
    for i in (0, 2, 4, 6, 8, 13, 15, 17, 20):
        assert f(**{f"a{i}": P(0x100008)}) == ALIGN
    assert f(a7=P(0x100002)) == ALIGN
    assert f(a10=1 << 31) == UNSUPPORTED
    assert f(a10=0, a0=None, a17=None) == OK


def test_norm_workspace():
    f = mx.mx_rms_norm_backward_workspace_bytes
    assert f(-1, 64) == -1 and f(5, 60) == -1 and f(5, 0) == -1 and f(5, 40000) == -1 and f(1 << 31, 64) == -1
    assert f(0, 64) == 0 and f(1, 64) == 0 and f(100000, 64) > 0


def test_the_binding_refuses():
    l, x = torch.zeros(3, 8), torch.zeros(3, 8, dtype=torch.bfloat16)
    w, i32 = torch.zeros(8), torch.zeros((3, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="one GPU"):
        mx.mx_router(l, 2)
    with pytest.raises(TypeError, match="logits"):
        mx.mx_router(l.double(), 2)
    with pytest.raises(ValueError, match="score"):
        mx.mx_router(l, 2, score="max")
    with pytest.raises(ValueError, match="contiguous rows"):
        mx.mx_router(torch.zeros(8, 3).t(), 2)
    with pytest.raises(ValueError, match="bias"):
        mx.mx_router(l, 2, bias=torch.zeros(7))
    with pytest.raises(TypeError, match="bias"):
        mx.mx_router(l, 2, bias=torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="experts"):
        mx.mx_router(l, 2, experts=torch.zeros((3, 3), dtype=torch.int32))
    with pytest.raises(ValueError, match="dweights"):
        mx.mx_router_backward(l, i32, torch.zeros(3, 3))
    with pytest.raises(TypeError, match="dlogits"):
        mx.mx_router_backward(l, i32, torch.zeros(3, 2), dlogits=x)
    with pytest.raises(ValueError, match="one GPU"):
        mx.mx_combine_dweights(x, x, i32)
    with pytest.raises(ValueError, match="y must"):
        mx.mx_combine_dweights(x, torch.zeros(3, 16, dtype=torch.bfloat16), i32)
    with pytest.raises(ValueError, match="one GPU"):
        mx.mx_rms_norm(x, w)
    with pytest.raises(TypeError, match="x must"):
        mx.mx_rms_norm(l, w, residual=l)  # x is bf16 beside a residual
    with pytest.raises(ValueError, match="h is written"):
        mx.mx_rms_norm(x, w, h=x)
    with pytest.raises(ValueError, match="s is written"):
        mx.mx_rms_norm(x, w, s=True)
    with pytest.raises(ValueError, match="weight"):
        mx.mx_rms_norm(x, torch.zeros(16))
    with pytest.raises(ValueError, match="accumulate"):
        mx.mx_rms_norm_backward(x, x, w, torch.zeros(3), accumulate=True)
    with pytest.raises(ValueError, match="dx"):
        mx.mx_rms_norm_backward(x, x, w, torch.zeros(3), dx=True)
    with pytest.raises(TypeError, match="dh_in"):
        mx.mx_rms_norm_backward(x, x, w, torch.zeros(3), dh_in=l)
