"""Python binding of the training step's C ABI (include/moe_train.h): token
rows sorted by expert and back, the router's gradient, and the experts'
grouped products, each with its gradient.

Argument marshalling only, like the package's other calls: every function
checks dtype, device, layout and size, then calls the C function of the same
name.  Outputs are the caller's buffers.  Tensors of token rows ([T, d]: x,
dx, out, dout, add) may have any row stride with contiguous columns; all
others are contiguous.  A call runs on the current CUDA device, where all its
tensors (and the stream, where one is given) have to be; others are refused.
The tensors belong to the stream the call is queued on: order other streams'
work on them with events, as for any kernel.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import (MOE_DTYPE_BF16, MOE_DTYPE_F32, _DIMS, _PROTOS, _check, _stream, lib, moe_dims)

_P, _I, _I64, _F, _SZ = C.c_void_p, C.c_int, C.c_int64, C.c_float, C.c_size_t
_PROTOS.update({
    "moe_train_workspace_size": ([_DIMS, C.POINTER(C.c_size_t)], _I),
    "moe_dispatch_rows": ([_DIMS, _P, _I64, _P, _I, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "moe_dispatch_rows_grad": ([_DIMS, _P, _P, _P, _I64, _P, _I64, _P], _I),
    "moe_combine_rows": ([_DIMS, _P, _P, _P, _P, _I64, _P, _I64, _P], _I),
    "moe_combine_rows_grad": ([_DIMS, _P, _I64, _P, _P, _P, _P, _P, _P], _I),
    "moe_gate_grad": ([_DIMS, _P, _P, _P, _F, _P, _P, _P, _SZ, _P], _I),
    "moe_experts_up": ([_DIMS, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "moe_experts_up_grad": ([_DIMS, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _SZ, _P], _I),
    "moe_experts_down": ([_DIMS, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "moe_experts_down_grad": ([_DIMS, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _SZ, _P], _I),
    "moe_experts_path": ([_DIMS], C.c_char_p),
})

__all__ = ["moe_train_workspace_size", "moe_dispatch_rows", "moe_dispatch_rows_grad", "moe_combine_rows",
           "moe_combine_rows_grad", "moe_gate_grad", "moe_experts_up", "moe_experts_up_grad", "moe_experts_down",
           "moe_experts_down_grad", "moe_experts_path"]

_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8
_WTYPE = {MOE_DTYPE_F32: torch.float32, MOE_DTYPE_BF16: torch.bfloat16}


def _here():
    """The current CUDA device's index (-2: there is none)."""
    try:
        return torch._C._cuda_getDevice()
    except RuntimeError:
        return -2


def _refuse(dev, t, dtype, numel, name):
    if t is None:
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, but the call runs on the current device, cuda:{dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")


def _buf(dev, t, dtype, numel, name, optional=False):
    """Address of a contiguous tensor of at least numel elements on device dev (None -> None if optional)."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.numel() >= numel:
            return t.data_ptr()
    except AttributeError:
        if t is None and optional:
            return None
    _refuse(dev, t, dtype, numel, name)


def _rows(dev, t, dtype, T, d, name, optional=False):
    """Address and row stride of token rows [T, d] (contiguous columns)."""
    if t is None and optional:
        return None, 0
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not dtype:
        _refuse(dev, t, dtype, T * d, name)
    shape = t.shape
    if len(shape) != 2 or shape[0] < T or shape[1] != d:
        raise ValueError(f"{name} has shape {tuple(shape)}, needs [{T}, {d}]")
    ld, inner = t.stride()
    if inner != 1 and d > 1:
        raise ValueError(f"{name} must have contiguous columns")
    if T <= 1:
        ld = d
    if ld < d:
        raise ValueError(f"{name} has a row stride of {ld}, below its {d} columns")
    return t.data_ptr(), ld


def _queue(dev, stream):
    """The stream of a call: the given one, or the device's current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise ValueError(f"the stream is of cuda:{stream.device_index}, but the current device is cuda:{dev}")
    return _stream(stream)


def _grad_type(dev, dims, a, b, names, numel):
    """Addresses of the weight gradients and their type code (both of wtype or both float32)."""
    given = [t for t in (a, b) if t is not None]
    if not given:
        return None, None, dims.wtype
    dtype = given[0].dtype
    if dtype not in (_F32, _WTYPE[dims.wtype]):
        raise TypeError(f"{names[0]} has dtype {dtype}, expected {_WTYPE[dims.wtype]} or {_F32}")
    pa, pb = (_buf(dev, t, dtype, numel, n, True) for t, n in zip((a, b), names))
    return pa, pb, MOE_DTYPE_F32 if dtype is _F32 else MOE_DTYPE_BF16


def moe_train_workspace_size(dims: moe_dims) -> int:
    """Bytes of the workspace of these calls (zero-fill it once)."""
    n = C.c_size_t()
    _check(lib().moe_train_workspace_size(C.byref(dims), C.byref(n)), "moe_train_workspace_size")
    return n.value


def moe_experts_path(dims: moe_dims) -> str:
    """Which kernels the experts' products run for these dimensions (no device work)."""
    return lib().moe_experts_path(C.byref(dims)).decode()


def moe_dispatch_rows(dims, x, expert_idx, capacity, x_perm, expert_offsets, perm, inv_perm, ws, stream=None):
    """Sort the slots by expert and copy the token rows: x [T, d] -> x_perm [T*k, d]."""
    dev = _here()
    T, d, wt = dims.T, dims.d, _WTYPE[dims.wtype]
    slots = T * dims.k
    px, ldx = _rows(dev, x, wt, T, d, "x")
    _check(lib().moe_dispatch_rows(
        dims, px, ldx, _buf(dev, expert_idx, _I32, slots, "expert_idx"), int(capacity),
        _buf(dev, x_perm, wt, slots * d, "x_perm"), _buf(dev, expert_offsets, _I32, dims.N + 1, "expert_offsets"),
        _buf(dev, perm, _I32, slots, "perm"), _buf(dev, inv_perm, _I32, slots, "inv_perm"),
        _buf(dev, ws, _U8, 0, "ws"), ws.numel(), _queue(dev, stream)), "moe_dispatch_rows")


def moe_dispatch_rows_grad(dims, dx_perm, inv_perm, add, dx, stream=None):
    """dx [T, d] = add + the sum of every token's rows of dx_perm [T*k, d]."""
    dev = _here()
    T, d, wt = dims.T, dims.d, _WTYPE[dims.wtype]
    slots = T * dims.k
    padd, ldadd = _rows(dev, add, wt, T, d, "add", True)
    pdx, lddx = _rows(dev, dx, wt, T, d, "dx")
    _check(lib().moe_dispatch_rows_grad(
        dims, _buf(dev, dx_perm, wt, slots * d, "dx_perm"), _buf(dev, inv_perm, _I32, slots, "inv_perm"), padd,
        ldadd, pdx, lddx, _queue(dev, stream)), "moe_dispatch_rows_grad")


def moe_combine_rows(dims, y_perm, gate, inv_perm, add, out, stream=None):
    """out [T, d] = add + the gate-weighted sum of every token's rows of y_perm [T*k, d]."""
    dev = _here()
    T, d, wt = dims.T, dims.d, _WTYPE[dims.wtype]
    slots = T * dims.k
    padd, ldadd = _rows(dev, add, wt, T, d, "add", True)
    pout, ldout = _rows(dev, out, wt, T, d, "out")
    _check(lib().moe_combine_rows(
        dims, _buf(dev, y_perm, wt, slots * d, "y_perm"), _buf(dev, gate, _F32, slots, "gate", True),
        _buf(dev, inv_perm, _I32, slots, "inv_perm"), padd, ldadd, pout, ldout, _queue(dev, stream)), "moe_combine_rows")


def moe_combine_rows_grad(dims, dout, y_perm, gate, inv_perm, dy_perm, dgate, stream=None):
    """dy_perm [T*k, d] and dgate [T, k] (either may be None) from dout [T, d]."""
    dev = _here()
    T, d, wt = dims.T, dims.d, _WTYPE[dims.wtype]
    slots = T * dims.k
    pd, ldd = _rows(dev, dout, wt, T, d, "dout")
    _check(lib().moe_combine_rows_grad(
        dims, pd, ldd, _buf(dev, y_perm, wt, slots * d, "y_perm", dgate is None),
        _buf(dev, gate, _F32, slots, "gate", True), _buf(dev, inv_perm, _I32, slots, "inv_perm"),
        _buf(dev, dy_perm, wt, slots * d, "dy_perm", True), _buf(dev, dgate, _F32, slots, "dgate", True),
        _queue(dev, stream)), "moe_combine_rows_grad")


def moe_gate_grad(dims, router_prob, topk_idx, dgate, balance, dlogits, balance_loss, ws, stream=None):
    """dlogits [T, N] from dgate [T, k]; balance_loss [1] may be None."""
    dev = _here()
    T, N = dims.T, dims.N
    slots = T * dims.k
    _check(lib().moe_gate_grad(
        dims, _buf(dev, router_prob, _F32, T * N, "router_prob"), _buf(dev, topk_idx, _I32, slots, "topk_idx"),
        _buf(dev, dgate, _F32, slots, "dgate"), float(balance), _buf(dev, dlogits, _F32, T * N, "dlogits"),
        _buf(dev, balance_loss, _F32, 1, "balance_loss", True), _buf(dev, ws, _U8, 0, "ws"), ws.numel(),
        _queue(dev, stream)), "moe_gate_grad")


def moe_experts_up(dims, x_perm, expert_offsets, w_gate, w_up, g, u, h, ws, stream=None):
    """g = x Wg^T, u = x Wu^T (both may be None), h = SiLU(g) u per expert's rows."""
    dev = _here()
    d, I, wt, slots = dims.d, dims.I, _WTYPE[dims.wtype], dims.T * dims.k
    nw = dims.N * I * d
    _check(lib().moe_experts_up(
        dims, _buf(dev, x_perm, wt, slots * d, "x_perm"), _buf(dev, expert_offsets, _I32, dims.N + 1, "expert_offsets"),
        _buf(dev, w_gate, wt, nw, "w_gate"), _buf(dev, w_up, wt, nw, "w_up"), _buf(dev, g, wt, slots * I, "g", True),
        _buf(dev, u, wt, slots * I, "u", True), _buf(dev, h, wt, slots * I, "h"), _buf(dev, ws, _U8, 0, "ws"), ws.numel(),
        _queue(dev, stream)), "moe_experts_up")


def moe_experts_up_grad(dims, dg, du, x_perm, expert_offsets, w_gate, w_up, dx_perm, dw_gate, dw_up, accumulate, ws,
                        stream=None):
    """dx_perm = dg Wg + du Wu (may be None); dw_gate = dg^T x, dw_up = du^T x
    [N, I, d] in the layer's type or float32 (both may be None).  accumulate
    adds to the float32 buffers."""
    dev = _here()
    d, I, wt, slots = dims.d, dims.I, _WTYPE[dims.wtype], dims.T * dims.k
    nw = dims.N * I * d
    pg, pu, gtype = _grad_type(dev, dims, dw_gate, dw_up, ("dw_gate", "dw_up"), nw)
    _check(lib().moe_experts_up_grad(
        dims, _buf(dev, dg, wt, slots * I, "dg"), _buf(dev, du, wt, slots * I, "du"),
        _buf(dev, x_perm, wt, slots * d, "x_perm", pg is None), _buf(dev, expert_offsets, _I32, dims.N + 1, "expert_offsets"),
        _buf(dev, w_gate, wt, nw, "w_gate", dx_perm is None), _buf(dev, w_up, wt, nw, "w_up", dx_perm is None),
        _buf(dev, dx_perm, wt, slots * d, "dx_perm", True), pg, pu, gtype, int(bool(accumulate)),
        _buf(dev, ws, _U8, 0, "ws"), ws.numel(), _queue(dev, stream)), "moe_experts_up_grad")


def moe_experts_down(dims, h, expert_offsets, w_down, y_perm, ws, stream=None):
    """y_perm = h Wd per expert's rows."""
    dev = _here()
    d, I, wt, slots = dims.d, dims.I, _WTYPE[dims.wtype], dims.T * dims.k
    _check(lib().moe_experts_down(
        dims, _buf(dev, h, wt, slots * I, "h"), _buf(dev, expert_offsets, _I32, dims.N + 1, "expert_offsets"),
        _buf(dev, w_down, wt, dims.N * I * d, "w_down"), _buf(dev, y_perm, wt, slots * d, "y_perm"),
        _buf(dev, ws, _U8, 0, "ws"), ws.numel(), _queue(dev, stream)), "moe_experts_down")


def moe_experts_down_grad(dims, dy_perm, h, g, u, expert_offsets, w_down, dg, du, dw_down, accumulate, ws, stream=None):
    """dg, du through h = SiLU(g) u (both may be None); dw_down = h^T dy
    [N, I, d] in the layer's type or float32 (may be None).  accumulate adds
    to the float32 buffer."""
    dev = _here()
    d, I, wt, slots = dims.d, dims.I, _WTYPE[dims.wtype], dims.T * dims.k
    nw, skip = dims.N * I * d, dg is None and du is None
    pw, _, gtype = _grad_type(dev, dims, dw_down, None, ("dw_down", ""), nw)
    _check(lib().moe_experts_down_grad(
        dims, _buf(dev, dy_perm, wt, slots * d, "dy_perm"), _buf(dev, h, wt, slots * I, "h", pw is None),
        _buf(dev, g, wt, slots * I, "g", skip), _buf(dev, u, wt, slots * I, "u", skip),
        _buf(dev, expert_offsets, _I32, dims.N + 1, "expert_offsets"), _buf(dev, w_down, wt, nw, "w_down", skip),
        _buf(dev, dg, wt, slots * I, "dg", True), _buf(dev, du, wt, slots * I, "du", True), pw, gtype, int(bool(accumulate)),
        _buf(dev, ws, _U8, 0, "ws"), ws.numel(), _queue(dev, stream)), "moe_experts_down_grad")
