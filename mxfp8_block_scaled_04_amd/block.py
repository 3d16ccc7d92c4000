"""Python binding of what surrounds the experts: the router and its gradient,
the gradient of the routing weights through the combine, and the
root-mean-square norm with its gradient (see include/libmxmoe_block.h for the
contract of each call).

Argument marshalling only, as in the package's main module, which re-exports
everything here: every step runs in the HIP kernels, and there is no
fallback.  A call runs on the GPU of its tensors, on that GPU's current stream
unless it is given one.
"""
import ctypes

import torch

from . import _check, load
from .training import _empty as _empty_on

SIGMOID, RENORM, LOGITS_BF16 = 1, 2, 4
STREAM_FP32, WEIGHT_FP32 = 1, 2

# Exported C symbols of include/libmxmoe_block.h, in its order.
BLOCK_SYMBOLS = (
    "mx_router", "mx_router_backward", "mx_combine_dweights", "mx_rms_norm", "mx_rms_norm_backward",
    "mx_rms_norm_backward_workspace_bytes",
)

_BF16, _FP32, _INT32, _UINT8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8

_signed = None


def _lib():
    """The library, with the signatures of this module's calls set."""
    global _signed
    lib = load()  # (another one if a program opens a build of its own)
    if _signed is not lib:
        P, I64, I32, U32, F, ST = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_float,
                                   ctypes.c_int)
        for name, args, result in (
            ("mx_router", [P, I64, I64, I32, P, I32, I32, I32, I32, F, U32, P, P, P, P], ST),
            ("mx_router_backward", [P, I64, I64, I32, P, P, P, I32, F, U32, P, I64, P], ST),
            ("mx_combine_dweights", [P, I64, P, I64, I64, P, I64, I32, I64, P, P], ST),
            ("mx_rms_norm", [P, I64, P, I64, P, I64, I64, F, U32, P, I64, P, I64, P, P, P, P], ST),
            ("mx_rms_norm_backward", [P, I64, P, I64, P, I64, P, P, P, I64, I64, I64, U32, P, I64, P, I64, P, I32, I32,
                                      P, I64, P], ST),
            ("mx_rms_norm_backward_workspace_bytes", [I64, I64], I64),
        ):
            f = getattr(lib, name)
            f.argtypes, f.restype = args, result
        _signed = lib
    return lib


# Small calls are bound by the host's part (a launch is 3 us of it), so the
# checks below avoid what costs a microsecond: stream and device objects (the
# raw handles are read where this torch has them), sets and generators, tests
# of what a call has made itself.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name, at, stream, *args):
    """The call on GPU `at`, which need not be the current one."""
    if stream is not None:
        if stream.device.index != at:
            raise ValueError("the stream is of another GPU than the tensors")
        handle = stream.cuda_stream
    elif _raw_stream is not None:
        handle = _raw_stream(at)
    else:
        handle = torch.cuda.current_stream(at).cuda_stream
    if at == _current_device():
        rc = getattr(_lib(), name)(*args, handle)
    else:
        with torch.cuda.device(at):
            rc = getattr(_lib(), name)(*args, handle)
    if rc:
        _check(rc, name)


def _one_gpu(first, *others):
    """Its number."""
    at = first.get_device()  # -1: not on a GPU
    if at < 0:
        raise ValueError("all tensors must be on one GPU")
    for t in others:
        if t is not None and t.get_device() != at:
            raise ValueError("all tensors must be on one GPU")
    return at


def _empty(rows, columns, dtype, device, stream):
    if stream is None:
        return torch.empty(rows, columns, dtype=dtype, device=device)
    return _empty_on((rows, columns), dtype, device, stream)


def _vector(length, dtype, device, stream):
    return torch.empty(length, dtype=dtype, device=device) if stream is None else _empty_on(length, dtype, device, stream)


def _wrong_type(t, name, dtypes):
    return TypeError(f"{name} must be {' or '.join(str(d).removeprefix('torch.') for d in dtypes)}, not {t.dtype}")


def _matrix(t, name, dtypes, rows=None, columns=None):
    """The row stride of a matrix (of rows x columns, if given) whose rows are contiguous."""
    if t.dtype not in dtypes:
        raise _wrong_type(t, name, dtypes)
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a matrix")
    r, c = shape
    if rows is not None and (r != rows or c != columns):
        raise ValueError(f"{name} must be a matrix of {rows} x {columns}")
    ld, step = t.stride()
    if step != 1 and c > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return 8 * -(-c // 8) if r <= 1 or c == 0 else ld  # (not used)


def _whole(t, name, dtypes, *shape):
    if t.dtype not in dtypes:
        raise _wrong_type(t, name, dtypes)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {' x '.join(map(str, shape))}")


def _check_int32(bits):
    """bits: the bitwise or of numbers that the call takes as int32 (ctypes would drop what is above)."""
    if not -0x80000000 <= bits <= 0x7FFFFFFF:
        raise ValueError("the numbers of experts, choices and groups must be below 2^31")


def _at(t):
    return None if t is None else t.data_ptr()


def _flags(score, renorm, logits):
    if score not in ("softmax", "sigmoid"):
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    return (SIGMOID if score == "sigmoid" else 0) | (RENORM if renorm else 0) | (
        LOGITS_BF16 if logits.dtype is _BF16 else 0)


def mx_router(logits, k, bias=None, groups=1, groups_kept=None, group_top=2, score="softmax", renorm=True, scale=1.0,
              experts=None, weights=None, scores=None, stream=None):
    """logits float32 or bf16 [T, E] (row stride may exceed E) -> (experts int32
    [T, k], weights float32 [T, k], scores float32 [T, E] or None): the k
    experts of the largest score (+ bias float32 [E]) of each token, largest
    first, and their weights, as mx_route_plan and mx_combine take them (-1 and
    0 where a mask of -infinity leaves fewer).  score: "softmax" or "sigmoid";
    groups, groups_kept (default: all), group_top: choose among the experts of
    the groups_kept groups of the largest sums of group_top choices; renorm:
    weights are divided by their sum; scale: their factor.  scores: None, True
    (allocate) or a tensor that receives all scores."""
    ldl = _matrix(logits, "logits", (_FP32, _BF16))
    T, E = logits.shape
    flags = _flags(score, renorm, logits)
    if groups_kept is None:
        groups_kept = groups
    _check_int32(E | k | groups | groups_kept | group_top)
    dev = logits.device
    if experts is None:
        experts = _empty(T, k, _INT32, dev, stream)
    else:
        _whole(experts, "experts", (_INT32,), T, k)
    if weights is None:
        weights = _empty(T, k, _FP32, dev, stream)
    else:
        _whole(weights, "weights", (_FP32,), T, k)
    if scores is True:
        scores = _empty(T, E, _FP32, dev, stream)
    elif scores is not None:
        _whole(scores, "scores", (_FP32,), T, E)
    if bias is not None:
        _whole(bias, "bias", (_FP32,), E)
    at = _one_gpu(logits, bias, experts, weights, scores)
    _call("mx_router", at, stream, logits.data_ptr(), ldl, T, E, _at(bias), groups, groups_kept, group_top, k,
          scale, flags, experts.data_ptr(), weights.data_ptr(), _at(scores))
    return experts, weights, scores


def mx_router_backward(logits, experts, dweights, dscores=None, score="softmax", renorm=True, scale=1.0, dlogits=None,
                       stream=None):
    """Gradient of the logits [T, E] from that of the weights (dweights float32
    [T, k], of the experts int32 [T, k] that mx_router chose with the same
    score, renorm and scale) and, if given, of all scores (dscores float32
    [T, E]).  Returns dlogits of the logits' type."""
    ldl = _matrix(logits, "logits", (_FP32, _BF16))
    T, E = logits.shape
    k = experts.shape[1] if experts.dim() == 2 else 0
    _whole(experts, "experts", (_INT32,), T, k)
    _whole(dweights, "dweights", (_FP32,), T, k)
    if dscores is not None:
        _whole(dscores, "dscores", (_FP32,), T, E)
    flags = _flags(score, renorm, logits)
    _check_int32(E | k)
    ldd = E
    if dlogits is None:
        dlogits = _empty(T, E, logits.dtype, logits.device, stream)
    else:
        ldd = _matrix(dlogits, "dlogits", (logits.dtype,), T, E)
    at = _one_gpu(logits, experts, dweights, dscores, dlogits)
    _call("mx_router_backward", at, stream, logits.data_ptr(), ldl, T, E, experts.data_ptr(),
          dweights.data_ptr(), _at(dscores), k, scale, flags, dlogits.data_ptr(), ldd)
    return dlogits


def mx_combine_dweights(dout, y, slot_of, dweights=None, stream=None):
    """Gradient of mx_combine's weights: dout bf16 [T, N], y bf16 [M, N]
    expert-ordered rows, slot_of int32 [T, k] -> float32 [T, k], the products
    of each token's output gradient with its expert rows (0 where it has none)."""
    ldd = _matrix(dout, "dout", (_BF16,))
    T, N = dout.shape
    ldy = _matrix(y, "y", (_BF16,), y.shape[0], N)
    k = slot_of.shape[1] if slot_of.dim() == 2 else 0
    _whole(slot_of, "slot_of", (_INT32,), T, k)
    _check_int32(k)
    if dweights is None:
        dweights = _empty(T, k, _FP32, dout.device, stream)
    else:
        _whole(dweights, "dweights", (_FP32,), T, k)
    at = _one_gpu(dout, y, slot_of, dweights)
    _call("mx_combine_dweights", at, stream, dout.data_ptr(), ldd, y.data_ptr(), y.shape[0], ldy,
          slot_of.data_ptr(), T, k, N, dweights.data_ptr())
    return dweights


def mx_rms_norm(x, weight, residual=None, eps=1e-6, h=None, y=True, q=None, s=None, rstd=None, stream=None):
    """Root-mean-square norm of the rows of x + residual, and its MXFP8 rows.
    x bf16 [M, N]; residual None or bf16 or float32 [M, N] (without one x may
    be float32); weight bf16 or float32 [N].  y, q, s, rstd: None (not
    written), True (allocated) or a tensor: y bf16 [M, N], q uint8 [M, N] codes
    and s their packed scales (with q; as mx_quantize_rows of y writes them),
    rstd float32 [M] for the backward pass.  h: the sum, allocated with a
    residual if None; it may be the residual itself.  Returns (y, h, q, s, rstd);
    h is None without a residual."""
    M, N = x.shape if x.dim() == 2 else (0, 0)
    dev, ldh, ldy = x.device, N, N
    if residual is None:
        ldx, ldr, kind = _matrix(x, "x", (_BF16, _FP32)), 0, x.dtype
        if h is not None:
            raise ValueError("h is written with a residual only")
    else:
        ldx, ldr, kind = _matrix(x, "x", (_BF16,)), _matrix(residual, "residual", (_BF16, _FP32), M, N), residual.dtype
        if h is None:
            h = _empty(M, N, kind, dev, stream)
        else:
            ldh = _matrix(h, "h", (kind,), M, N)
    _whole(weight, "weight", (_BF16, _FP32), N)
    if y is True:
        y = _empty(M, N, _BF16, dev, stream)
    elif y is not None:
        ldy = _matrix(y, "y", (_BF16,), M, N)
    if q is not None:
        size = 32 * -(-M // 32) * 8 * -(-N // 256)  # mx_scale_bytes
        if q is True:
            q = _empty(M, N, _UINT8, dev, stream)
        else:
            _whole(q, "q", (_UINT8,), M, N)
        if s is None or s is True:
            s = _vector(size, _UINT8, dev, stream)
        else:
            _whole(s, "s", (_UINT8,), size)
    elif s is not None:
        raise ValueError("s is written with q only")
    if rstd is True:
        rstd = _vector(M, _FP32, dev, stream)
    elif rstd is not None:
        _whole(rstd, "rstd", (_FP32,), M)
    at = _one_gpu(x, residual, weight, h, y, q, s, rstd)
    flags = (STREAM_FP32 if kind is _FP32 else 0) | (WEIGHT_FP32 if weight.dtype is _FP32 else 0)
    _call("mx_rms_norm", at, stream, x.data_ptr(), ldx, _at(residual), ldr, weight.data_ptr(), M, N, eps,
          flags, _at(h), ldh, _at(y), ldy, _at(q), _at(s), _at(rstd))
    return y, h, q, s, rstd


def mx_rms_norm_backward(dy, h, weight, rstd, dy2=None, dh_in=None, dh=None, dx=None, dweight=True, accumulate=False,
                         workspace=None, stream=None):
    """Gradients of mx_rms_norm: dy (and dy2) bf16 [M, N] gradients of y, h and
    rstd of the forward pass (h = x without a residual), dh_in the gradient
    that reaches h from behind, of h's type.  Returns (dh, dx, dweight): dh of
    h's type, the gradient of x and of the residual; dx None, or its bf16
    rounding where h is float32 (True: allocated); dweight [N]: None (left
    out), True (allocated in the weight's type), a dtype, or a bf16 or float32
    tensor, which accumulate adds to (float32).  workspace: a uint8 tensor of
    mx_rms_norm_backward_workspace_bytes, allocated on the stream's behalf if
    None."""
    ldh = _matrix(h, "h", (_BF16, _FP32))
    M, N = h.shape
    kind, dev, ldo, lddx = h.dtype, h.device, N, N
    ldy = _matrix(dy, "dy", (_BF16,), M, N)
    ldy2 = 0 if dy2 is None else _matrix(dy2, "dy2", (_BF16,), M, N)
    ldi = 0 if dh_in is None else _matrix(dh_in, "dh_in", (kind,), M, N)
    _whole(weight, "weight", (_BF16, _FP32), N)
    _whole(rstd, "rstd", (_FP32,), M)
    if dh is None:
        dh = _empty(M, N, kind, dev, stream)
    else:
        ldo = _matrix(dh, "dh", (kind,), M, N)
    if dx is not None:
        if kind is not _FP32:
            raise ValueError("dx is written for a float32 stream only: dh is it")
        if dx is True:
            dx = _empty(M, N, _BF16, dev, stream)
        else:
            lddx = _matrix(dx, "dx", (_BF16,), M, N)
    size = 0
    if isinstance(dweight, torch.Tensor):
        _whole(dweight, "dweight", (_BF16, _FP32), N)
    elif accumulate:
        raise ValueError("accumulate needs dweight")
    elif dweight is not None:
        dweight = _vector(N, weight.dtype if dweight is True else dweight, dev, stream)
        if dweight.dtype is not _FP32 and dweight.dtype is not _BF16:
            raise _wrong_type(dweight, "dweight", (_BF16, _FP32))
    if dweight is not None:
        if workspace is None:
            size = _lib().mx_rms_norm_backward_workspace_bytes(M, N)
            if size > 0:
                workspace = _vector(size, _UINT8, dev, stream)
        elif workspace.dtype is not _UINT8 or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 tensor")
        else:
            size = workspace.numel()
    at = _one_gpu(h, dy, dy2, weight, rstd, dh_in, dh, dx, dweight, workspace)
    flags = (STREAM_FP32 if kind is _FP32 else 0) | (WEIGHT_FP32 if weight.dtype is _FP32 else 0)
    _call("mx_rms_norm_backward", at, stream, dy.data_ptr(), ldy, _at(dy2), ldy2, h.data_ptr(), ldh,
          weight.data_ptr(), rstd.data_ptr(), _at(dh_in), ldi, M, N, flags, dh.data_ptr(), ldo, _at(dx), lddx,
          _at(dweight), dweight is not None and dweight.dtype is _FP32, bool(accumulate), _at(workspace),
          max(size, 0))
    return dh, dx, dweight


def mx_rms_norm_backward_workspace_bytes(M, N):
    return int(_lib().mx_rms_norm_backward_workspace_bytes(int(M), int(N)))
