"""Python binding of the training-step calls of libmxmoe (products of
unquantized experts, gradient norm, AdamW; see include/libmxmoe_train.h for
the contract of each call).

Argument marshalling only, as in the package's main module, which re-exports
everything here: every step runs in the HIP kernels, and there is no
fallback.
"""
import ctypes

import torch

from . import _check, _ptr, load

BLOCK = 256  # elements per scale of an 8-bit optimizer state

W_BF16, G_BF16, STATE_8BIT, UNBIASED = 1, 2, 4, 16

# Exported C symbols of include/libmxmoe_train.h, in its order.
TRAIN_SYMBOLS = (
    "mx_grouped_gemm_bf16", "mx_grouped_gemm_bf16_dgrad", "mx_grouped_gemm_bf16_wgrad",
    "mx_grouped_gemm_bf16_wgrad_workspace_bytes", "mx_adamw_plan_bytes", "mx_adamw_plan",
    "mx_grad_norm_workspace_bytes", "mx_grad_norm", "mx_adamw",
)


class AdamwTensor(ctypes.Structure):
    """mx_adamw_tensor."""
    _fields_ = [("w", ctypes.c_void_p), ("master", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("weight_decay", ctypes.c_float), ("types", ctypes.c_uint32)]


_signed = None


def _lib():
    """The library, with the signatures of this module's calls set."""
    global _signed
    lib = load()  # (another one if a program opens a build of its own)
    if _signed is not lib:
        P, I64, I32, F, D, ST = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_double,
                                 ctypes.c_int)
        for name, args, result in (
            ("mx_grouped_gemm_bf16", [P, I64, P, P, I32, I64, I64, I64, P, I64, P], ST),
            ("mx_grouped_gemm_bf16_dgrad", [P, I64, P, P, I32, I64, I64, I64, P, I64, P], ST),
            ("mx_grouped_gemm_bf16_wgrad", [P, I64, P, I64, P, I32, I64, I64, I64, P, I32, I32, P, I64, P], ST),
            ("mx_grouped_gemm_bf16_wgrad_workspace_bytes", [I32, I64, I64, I64], I64),
            ("mx_adamw_plan_bytes", [P, I32], I64),
            ("mx_adamw_plan", [P, I32, P, P], ST),
            ("mx_grad_norm_workspace_bytes", [], I64),
            ("mx_grad_norm", [P, I32, I64, F, P, P, P], ST),
            ("mx_adamw", [P, I32, I64, P, D, P, D, D, D, P, P], ST),
        ):
            f = getattr(lib, name)
            f.argtypes, f.restype = args, result
        _signed = lib
    return lib


# Small calls are bound by the host's part, so the checks below avoid what
# costs a microsecond each (sets of devices, ctypes objects for addresses).
_BF16, _INT32 = torch.bfloat16, torch.int32


def _stream(stream):
    return torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream


def _rows(t, name):
    """(rows, columns, row stride) of a bf16 matrix whose rows are contiguous."""
    if t.dtype is not _BF16 or t.dim() != 2:
        raise TypeError(f"{name} must be a bf16 matrix")
    M, C = t.shape
    ld, step = t.stride()
    if C > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if M <= 1 or C == 0:  # a stride that is not used
        ld = 8 * -(-C // 8)
    return M, C, ld


def _offsets(t):
    if t.dtype is not _INT32 or t.dim() != 1 or not t.is_contiguous() or t.numel() < 2:
        raise ValueError("group_offsets must be a contiguous int32 [G + 1] tensor")
    return t.numel() - 1


def _weights(w, G):
    if w.dtype is not _BF16 or w.dim() != 3 or not w.is_contiguous():
        raise ValueError("w must be a contiguous bf16 [G, N, K] tensor")
    g, N, K = w.shape
    if g != G:
        raise ValueError("w and group_offsets differ in the number of groups")
    return N, K


def _same_device(first, *others):
    at = first.get_device()  # -1: not on a GPU
    if at < 0 or any(t is not None and t.get_device() != at for t in others):
        raise ValueError("all tensors must be on one GPU")


def _empty(shape, dtype, device, stream):
    """A buffer of a call's own, from the pool of the stream that writes it:
    memory of another pool can still be in use on that pool's stream, and can
    be given back there before the call has run."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def mx_grouped_gemm_bf16(x, w, group_offsets, out=None, stream=None):
    """out[r] = x[r] w[g]^T for the rows r of group g: x bf16 [M, K] (row
    stride may exceed K), w bf16 [G, N, K], group_offsets int32 [G+1].
    Returns out bf16 [M, N]."""
    G = _offsets(group_offsets)
    N, K = _weights(w, G)
    M, Kx, ldx = _rows(x, "x")
    if Kx != K:
        raise ValueError("K mismatch")
    if out is None:
        out = _empty((M, N), _BF16, x.device, stream)
    Mo, No, ldo = _rows(out, "out")
    if Mo != M or No != N:
        raise ValueError("out shape")
    _same_device(x, w, group_offsets, out)
    rc = _lib().mx_grouped_gemm_bf16(x.data_ptr(), ldx, w.data_ptr(), group_offsets.data_ptr(), G, M, N, K,
                                     out.data_ptr(), ldo, _stream(stream))
    _check(rc, "mx_grouped_gemm_bf16")
    return out


def mx_grouped_gemm_bf16_dgrad(dy, w, group_offsets, dx=None, stream=None):
    """dx[r] = dy[r] w[g] for the rows r of group g: dy bf16 [M, N], w bf16
    [G, N, K].  Returns dx bf16 [M, K]."""
    G = _offsets(group_offsets)
    N, K = _weights(w, G)
    M, Ny, ldy = _rows(dy, "dy")
    if Ny != N:
        raise ValueError("N mismatch")
    if dx is None:
        dx = _empty((M, K), _BF16, dy.device, stream)
    Mx, Kx, ldx = _rows(dx, "dx")
    if Mx != M or Kx != K:
        raise ValueError("dx shape")
    _same_device(dy, w, group_offsets, dx)
    rc = _lib().mx_grouped_gemm_bf16_dgrad(dy.data_ptr(), ldy, w.data_ptr(), group_offsets.data_ptr(), G, M, N, K,
                                           dx.data_ptr(), ldx, _stream(stream))
    _check(rc, "mx_grouped_gemm_bf16_dgrad")
    return dx


def mx_grouped_gemm_bf16_wgrad(dy, x, group_offsets, dw=None, accumulate=False, workspace=None, stream=None):
    """dw[g] = sum over the rows r of group g of dy[r]^T x[r]: dy bf16 [M, N],
    x bf16 [M, K].  dw: a bf16 or float32 [G, N, K] tensor, or None (bf16 is
    allocated); accumulate adds to the float32 dw given.  workspace: a uint8
    tensor of mx_grouped_gemm_bf16_wgrad_workspace_bytes, allocated on the
    stream's behalf if None.  Returns dw."""
    G = _offsets(group_offsets)
    M, N, ldy = _rows(dy, "dy")
    Mx, K, ldx = _rows(x, "x")
    if Mx != M:
        raise ValueError("dy and x differ in their rows")
    if dw is None:
        if accumulate:
            raise ValueError("accumulate needs dw")
        dw = _empty((G, N, K), _BF16, x.device, stream)
    fp32 = dw.dtype is torch.float32
    if tuple(dw.shape) != (G, N, K) or not dw.is_contiguous() or not (fp32 or dw.dtype is _BF16):
        raise ValueError("dw must be a contiguous bf16 or float32 [G, N, K] tensor")
    _same_device(dy, x, group_offsets, dw, workspace)
    lib = _lib()
    size = 0
    if workspace is None:
        size = lib.mx_grouped_gemm_bf16_wgrad_workspace_bytes(G, M, N, K)
        if size > 0:
            workspace = _empty(size, torch.uint8, dy.device, stream)
    elif workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    else:
        size = workspace.numel()
    rc = lib.mx_grouped_gemm_bf16_wgrad(dy.data_ptr(), ldy, x.data_ptr(), ldx, group_offsets.data_ptr(), G, M, N, K,
                                        dw.data_ptr(), fp32, bool(accumulate),
                                        None if workspace is None else workspace.data_ptr(), max(size, 0),
                                        _stream(stream))
    _check(rc, "mx_grouped_gemm_bf16_wgrad")
    return dw


def mx_grouped_gemm_bf16_wgrad_workspace_bytes(G, M, N, K):
    return int(_lib().mx_grouped_gemm_bf16_wgrad_workspace_bytes(int(G), int(M), int(N), int(K)))


class AdamWPlan:
    """A list of tensors as mx_grad_norm and mx_adamw take it: the device copy
    of the plan and, behind it, the workspace of the norm.  Keeps the tensors
    alive; to be kept itself until the calls that use it have run.  Calls of
    mx_grad_norm on one plan share its workspace: on several streams, each
    has to wait for the one before."""

    def __init__(self, device, count, chunks, image, workspace_at, tensors):
        self.device, self.count, self.chunks, self.tensors = device, count, chunks, tensors
        self.image, self.workspace = image, image[workspace_at:]
        self.address, self.workspace_address = image.data_ptr(), self.workspace.data_ptr()


def mx_adamw_plan(weights, grads, ms, vs, masters=None, m_scales=None, v_scales=None, weight_decay=0.0,
                  unbiased=False):
    """Plan of the tensors (lists of contiguous GPU tensors of the same
    lengths): weights and gradients float32 or bf16; states float32, or E4M3
    codes (uint8 or float8_e4m3fn) with float32 scales, one per 256 elements;
    masters float32, or None in the list or for all; weight_decay a number or
    one per tensor.  unbiased: 8-bit states are rounded at random, so that they
    are right on average (to be set for training: to nearest, which is the
    default of mx_adamw_tensor, a slowly falling v stays where it is; see
    include/libmxmoe_train.h).  Copies the plan and the zeroed workspace of mx_grad_norm
    to the GPU (synchronously: any stream can use them then): made once, while
    the tensors stay where they are."""
    count = len(weights)

    def column(values, name):
        if values is None:
            return [None] * count
        values = list(values)
        if len(values) != count:
            raise ValueError(f"{name}: {len(values)} values for {count} tensors")
        return values

    grads, ms, vs = column(grads, "grads"), column(ms, "ms"), column(vs, "vs")
    masters, m_scales, v_scales = (column(masters, "masters"), column(m_scales, "m_scales"),
                                   column(v_scales, "v_scales"))
    decay = [weight_decay] * count if isinstance(weight_decay, (int, float)) else column(weight_decay, "weight_decay")
    wide, narrow = (torch.float32, torch.bfloat16), (torch.uint8, torch.float8_e4m3fn)
    rows = (AdamwTensor * max(count, 1))()
    for i, (w, g, m, v, master, msc, vsc) in enumerate(zip(weights, grads, ms, vs, masters, m_scales, v_scales)):
        n = w.numel()
        if w.dtype not in wide or g.dtype not in wide:
            raise TypeError(f"tensor {i}: weights and gradients must be float32 or bf16")
        eight = m.dtype in narrow
        if (v.dtype in narrow) != eight or (not eight and (m.dtype != torch.float32 or v.dtype != torch.float32)):
            raise TypeError(f"tensor {i}: states must both be float32 or both E4M3 codes")
        if any(t.numel() != n for t in (g, m, v) + (() if master is None else (master,))):
            raise ValueError(f"tensor {i}: lengths differ")
        if master is not None and master.dtype != torch.float32:
            raise TypeError(f"tensor {i}: masters must be float32")
        for s in (msc, vsc):
            if s is not None and (s.dtype != torch.float32 or s.numel() != -(-n // BLOCK)):
                raise ValueError(f"tensor {i}: scales must be float32, one per {BLOCK} elements")
        given = [t for t in (w, g, m, v, master, msc, vsc) if t is not None]
        if not all(t.is_contiguous() for t in given):
            raise ValueError(f"tensor {i}: contiguous tensors required")
        _same_device(weights[0], *given)
        address = [None if t is None or t.numel() == 0 else t.data_ptr() for t in (w, master, g, m, v, msc, vsc)]
        rows[i] = AdamwTensor(*address, n, float(decay[i]), (W_BF16 if w.dtype == torch.bfloat16 else 0)
                              | (G_BF16 if g.dtype == torch.bfloat16 else 0) | (STATE_8BIT if eight else 0)
                              | (UNBIASED if eight and unbiased else 0))
    lib = _lib()
    at = max(16 * -(-int(lib.mx_adamw_plan_bytes(rows, count)) // 16), 0)  # (a list that is refused: below)
    image = torch.zeros(at + int(lib.mx_grad_norm_workspace_bytes()), dtype=torch.uint8)
    chunks = ctypes.c_int64(0)
    _check(lib.mx_adamw_plan(rows, count, _ptr(image), ctypes.byref(chunks)), "mx_adamw_plan")
    device = weights[0].device if count else torch.device("cuda", torch.cuda.current_device())
    return AdamWPlan(device, count, chunks.value, image.to(device), at,
                     [list(weights), grads, ms, vs, masters, m_scales, v_scales])


def mx_grad_norm(plan, max_norm=float("inf"), out=None, stream=None):
    """Global norm of the plan's gradients and the factor that clips them to
    max_norm.  Returns out float32 [2]: the norm and the factor (NaN when the
    norm is not finite)."""
    if out is None:
        out = _empty(2, torch.float32, plan.device, stream)
    if out.dtype != torch.float32 or out.numel() != 2 or not out.is_contiguous():
        raise ValueError("out must be a contiguous float32 [2] tensor")
    _same_device(plan.image, out)
    rc = _lib().mx_grad_norm(plan.address, plan.count, plan.chunks, max_norm, plan.workspace_address, out.data_ptr(),
                             _stream(stream))
    _check(rc, "mx_grad_norm")
    return out


def mx_adamw(plan, steps, lr, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=None, stream=None):
    """One AdamW step of the plan's tensors.  steps: int64 [2] on the GPU, the
    number of steps done (raised by the call) and a zero.  lr: a number, or a
    float32 tensor of one value on the GPU.  grad_scale: a float32 tensor of
    one value on the GPU (mx_grad_norm's second result); where it is not a
    finite non-negative number, the call changes nothing."""
    if steps.dtype != torch.int64 or steps.numel() != 2 or not steps.is_contiguous():
        raise ValueError("steps must be a contiguous int64 [2] tensor")
    on_device = lr if isinstance(lr, torch.Tensor) else None
    for t, name in ((on_device, "lr"), (grad_scale, "grad_scale")):
        if t is not None and (t.dtype != torch.float32 or t.numel() != 1):
            raise ValueError(f"{name} must be a float32 tensor of one value")
    _same_device(plan.image, steps, on_device, grad_scale)
    rc = _lib().mx_adamw(plan.address, plan.count, plan.chunks, steps.data_ptr(), 0.0 if on_device is not None else lr,
                         None if on_device is None else on_device.data_ptr(), beta1, beta2, eps,
                         None if grad_scale is None else grad_scale.data_ptr(), _stream(stream))
    _check(rc, "mx_adamw")
