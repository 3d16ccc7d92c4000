"""C-ABI checks of the training-step calls that need no GPU: both builds
export every symbol of include/libmxmoe_train.h, invalid arguments are
refused before anything is launched, and plans are laid out as documented."""
import ctypes
import os
import re

import pytest
import torch

import mxfp8_block_scaled_04_amd as mx
from mxfp8_block_scaled_04_amd import training as T

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "libmxmoe_train.h")

# tests/test_sanitize_train.py runs this module against a sanitizer build of
# the entry points (kernel launchers stubbed out) named by MXMOE_TRAIN_LIB
SAN = os.environ.get("MXMOE_TRAIN_LIB")
if SAN:
    mx._lib = ctypes.CDLL(SAN)

P = ctypes.c_void_p
FAKE = P(0x100000)  # never dereferenced: every call below fails validation first
OK, NULL, SHAPE, ALIGN, UNSUPPORTED = 0, 1, 2, 3, 5


def _header_names():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(mx_[a-z_0-9]+)\s*\(", src)))


def test_every_header_symbol_is_exported():
    names = _header_names()
    assert sorted(mx.TRAIN_SYMBOLS) == names
    libs = [T._lib()] if SAN else [T._lib(), mx.open_library(mx.DEBUG_LIB_PATH)]
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


@pytest.mark.parametrize("name", ["mx_grouped_gemm_bf16", "mx_grouped_gemm_bf16_dgrad"])
def test_product_refusals(name):
    # (a, lda, w, offsets, G, M, N, K, out, ldo, stream); widths: forward a K, out N; dgrad a N, out K
    f = _variants(getattr(T._lib(), name), (FAKE, 64, FAKE, FAKE, 4, 100, 64, 64, FAKE, 64, None))
    a, o = (7, 6) if name == "mx_grouped_gemm_bf16" else (6, 7)
    assert f(a5=-1) == SHAPE and f(a6=60) == SHAPE and f(a7=60) == SHAPE
    assert f(a1=56) == SHAPE and f(a9=56) == SHAPE
    assert f(a4=0) == SHAPE and f(a4=4097) == SHAPE
    assert f(a1=68) == ALIGN and f(a9=68) == ALIGN
    for i in (0, 2, 3, 8):
        assert f(**{f"a{i}": None}) == NULL
    for i in (0, 2, 8):
        assert f(**{f"a{i}": P(0x100008)}) == ALIGN
    assert f(a3=P(0x100002)) == ALIGN
    assert f(a1=1 << 22) == UNSUPPORTED and f(a9=1 << 22) == UNSUPPORTED
    assert f(a5=1 << 31) == UNSUPPORTED
    assert f(a6=1 << 16, a7=1 << 15, a1=1 << 16, a9=1 << 16) == UNSUPPORTED  # N K = 2^31
    assert f(a5=0, a0=None, a8=None) == OK
    assert f(**{f"a{o}": 0, "a0": None, "a8": None}) == OK  # no columns
    assert f(**{f"a{a}": 0, "a8": None}) == NULL            # an empty contraction still writes


def test_weight_gradient_refusals():
    # (dy, ldy, x, ldx, offsets, G, M, N, K, dw, fp32, accumulate, workspace, bytes, stream)
    f = _variants(T._lib().mx_grouped_gemm_bf16_wgrad,
                  (FAKE, 64, FAKE, 72, FAKE, 4, 100, 64, 72, FAKE, 1, 1, FAKE, 64, None))
    assert f(a6=-1) == SHAPE and f(a7=60) == SHAPE and f(a8=70) == SHAPE
    assert f(a1=56) == SHAPE and f(a3=64) == SHAPE
    assert f(a10=2) == SHAPE and f(a11=-1) == SHAPE and f(a13=-1) == SHAPE
    assert f(a12=P(0x100008)) == ALIGN
    assert f(a10=0) == UNSUPPORTED  # added to bf16
    for i in (0, 2, 4, 9):
        assert f(**{f"a{i}": None}) == NULL
    for i in (0, 2, 9):
        assert f(**{f"a{i}": P(0x100004)}) == ALIGN
    assert f(a1=68) == ALIGN
    assert f(a7=0, a0=None, a9=None) == OK
    assert f(a6=0, a0=None, a2=None, a9=None) == NULL  # no rows: zeros are written


def test_weight_gradient_workspace():
    f = mx.mx_grouped_gemm_bf16_wgrad_workspace_bytes
    assert f(0, 64, 8, 8) == -1 and f(1, -1, 8, 8) == -1 and f(1, 64, 12, 8) == -1
    size = f(2, 65536, 256, 384)
    assert size > 0 and size % (4 * 2 * 256 * 384) == 0
    if not SAN:
        assert f(16, 32768, 7168, 2048) == 0 and f(1, 128, 128, 128) == 0


def _row(n=5, types=0, decay=0.0, w=0x1000, master=None, g=0x2000, m=0x3000, v=0x4000, ms=None, vs=None):
    return T.AdamwTensor(w, master, g, m, v, ms, vs, n, decay, types)


def _plan(*rows):
    lib = T._lib()
    table = (T.AdamwTensor * max(1, len(rows)))(*rows)
    size = lib.mx_adamw_plan_bytes(table, len(rows))
    image = ctypes.create_string_buffer(max(1, size))
    chunks = ctypes.c_int64(-7)
    return lib.mx_adamw_plan(table, len(rows), image, ctypes.byref(chunks)), size, chunks.value, image


def test_plan_refusals():
    assert _plan(_row())[0] == OK
    assert _plan(_row(types=8))[0] == SHAPE
    assert _plan(_row(decay=-0.1))[0] == SHAPE and _plan(_row(decay=float("nan")))[0] == SHAPE
    assert _plan(_row(decay=float("inf")))[0] == SHAPE
    assert _plan(_row(master=0x5000))[0] == SHAPE              # masters of float32 weights
    assert _plan(_row(master=0x5000, types=T.W_BF16))[0] == OK
    assert _plan(_row(ms=0x6000))[0] == SHAPE                  # scales of float32 states
    assert _plan(_row(types=T.STATE_8BIT))[0] == NULL          # 8-bit states without scales
    assert _plan(_row(types=T.STATE_8BIT, ms=0x6000, vs=0x7000, m=0x3001, v=0x4003))[0] == OK
    assert _plan(_row(types=T.STATE_8BIT, ms=0x6002, vs=0x7000))[0] == ALIGN
    for name in ("w", "g", "m", "v"):
        assert _plan(_row(**{name: None}))[0] == NULL
        assert _plan(_row(**{name: 0x1002}))[0] == ALIGN
    assert _plan(_row(w=0x1002, types=T.W_BF16))[0] == OK and _plan(_row(w=0x1001, types=T.W_BF16))[0] == ALIGN
    assert _plan(_row(n=0, w=None, g=None, m=None, v=None))[0] == OK
    lib, table = T._lib(), (T.AdamwTensor * 2)(_row(n=-1), _row())
    assert lib.mx_adamw_plan_bytes(table, 1) == -1 and lib.mx_adamw_plan_bytes(table, -1) == -1
    assert lib.mx_adamw_plan_bytes(None, 1) == -1
    chunks = ctypes.c_int64()
    assert lib.mx_adamw_plan(table, 2, FAKE, ctypes.byref(chunks)) == SHAPE
    assert lib.mx_adamw_plan(table, -1, FAKE, ctypes.byref(chunks)) == SHAPE
    assert lib.mx_adamw_plan(None, 1, FAKE, ctypes.byref(chunks)) == NULL
    assert lib.mx_adamw_plan(table, 1, None, ctypes.byref(chunks)) == NULL
    assert lib.mx_adamw_plan(table, 1, FAKE, None) == NULL
    big = (T.AdamwTensor * 1)(_row(n=1 << 44))  # 2^32 chunks
    assert lib.mx_adamw_plan_bytes(big, 1) == -1
    assert lib.mx_adamw_plan(big, 1, FAKE, ctypes.byref(chunks)) == UNSUPPORTED


def test_plan_shares_every_element_out_once():
    sizes = [1, 0, 4096, 4097, 100000, 255]
    rc, size, chunks, image = _plan(*(_row(n=n) for n in sizes))
    assert rc == OK and chunks == sum(-(-n // 4096) for n in sizes)
    entry = (size - 4 * chunks) // len(sizes)
    assert entry % 16 == 0 and entry >= ctypes.sizeof(T.AdamwTensor)
    owner = (ctypes.c_int32 * chunks).from_buffer_copy(image.raw[entry * len(sizes):size])
    assert list(owner) == [i for i, n in enumerate(sizes) for _ in range(-(-n // 4096))]


def test_step_and_norm_refusals():
    lib = T._lib()
    # (plan, count, chunks, steps, lr, lr_device, beta1, beta2, eps, grad_scale, stream)
    f = _variants(lib.mx_adamw, (FAKE, 1, 1, FAKE, 1e-3, None, 0.9, 0.99, 1e-8, None, None))
    assert f(a1=-1) == SHAPE and f(a2=-1) == SHAPE and f(a2=1 << 31) == SHAPE
    for i in (6, 7):
        assert f(**{f"a{i}": 1.0}) == SHAPE and f(**{f"a{i}": -0.1}) == SHAPE
        assert f(**{f"a{i}": float("nan")}) == SHAPE
    assert f(a8=-1e-8) == SHAPE and f(a8=float("inf")) == SHAPE and f(a4=float("nan")) == SHAPE
    assert f(a0=None) == NULL and f(a3=None) == NULL
    assert f(a0=P(0x100008)) == ALIGN and f(a3=P(0x100004)) == ALIGN
    assert f(a5=P(0x100002)) == ALIGN and f(a9=P(0x100002)) == ALIGN
    # (plan, count, chunks, max_norm, workspace, out, stream)
    g = _variants(lib.mx_grad_norm, (FAKE, 1, 1, 1.0, FAKE, FAKE, None))
    assert g(a1=-1) == SHAPE and g(a2=-1) == SHAPE
    for bad in (0.0, -1.0, float("nan")):
        assert g(a3=bad) == SHAPE
    assert g(a0=None) == NULL and g(a4=None) == NULL and g(a5=None) == NULL
    assert g(a4=P(0x100004)) == ALIGN and g(a5=P(0x100002)) == ALIGN
    assert lib.mx_grad_norm_workspace_bytes() >= 8


def test_the_binding_refuses_cpu_tensors():
    w, off = torch.zeros(1, 8, 8, dtype=torch.bfloat16), torch.tensor([0, 2], dtype=torch.int32)
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="one GPU"):
        mx.mx_grouped_gemm_bf16(x, w, off)
    with pytest.raises(ValueError, match="one GPU"):
        mx.mx_adamw_plan([torch.zeros(4)], [torch.zeros(4)], [torch.zeros(4)], [torch.zeros(4)])
    with pytest.raises(ValueError, match="K mismatch"):
        mx.mx_grouped_gemm_bf16(x[:, :4], w, off)
    with pytest.raises(ValueError, match="groups"):
        mx.mx_grouped_gemm_bf16(x, w, torch.tensor([0, 1, 2], dtype=torch.int32))
    with pytest.raises(ValueError, match="contiguous rows"):
        mx.mx_grouped_gemm_bf16(torch.zeros(8, 2, dtype=torch.bfloat16).t(), w, off)
