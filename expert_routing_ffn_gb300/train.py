"""Python binding of the training step's C ABI (include/moe_train.h): token
rows sorted by expert and back, the router's gradient, the experts' grouped
products, and the norms, gate and residual of the block around the layer, each
with its gradient; activations kept for the backward pass in 8 bits.

Argument marshalling only, like the package's other calls: every function
checks dtype, device, layout and size, then calls the C function of the same
name.  Outputs are the caller's buffers.  Tensors of token rows ([T, d]: x,
dx, n, dn, y, dy, residual, out, dout, next, add; [rows, cols] of the calls
that pack and unpack) may have any row stride with contiguous columns; all
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


class moe_block(C.Structure):
    """The end of a block (include/moe_train.h); make_block fills it in."""
    _fields_ = [("eps", _F), ("weight_offset", _F), ("residual_scale", _F), ("post_norm", _I), ("gate", _I)]


_BLOCK = C.POINTER(moe_block)
_PROTOS.update({
    "moe_norm_rows": ([_DIMS, _P, _I64, _P, _F, _F, _P, _I64, _P, _P], _I),
    "moe_norm_rows_grad": ([_DIMS, _P, _I64, _P, _I64, _P, _P, _F, _P, _I64, _P, _I64, _P, _I, _I, _P, _SZ, _P], _I),
    "moe_block_out": ([_DIMS, _BLOCK, _P, _I64, _I, _P, _I64, _P, _P, _P, _P, _I64, _P, _I64, _P, _P, _P], _I),
    "moe_block_out_grad": ([_DIMS, _BLOCK, _P, _I64, _P, _I64, _P, _I64, _I, _P, _I64, _P, _P, _P, _P, _P, _P, _I64,
                            _P, _I64, _P, _P, _P, _I, _I, _P, _SZ, _P], _I),
    "moe_packed_size": ([_I64, _I, C.POINTER(_SZ), C.POINTER(_SZ)], _I),
    "moe_pack_rows": ([_I64, _I, _P, _I64, _I, _P, _P, _P], _I),
    "moe_unpack_rows": ([_I64, _I, _P, _P, _P, _I, _I64, _P, _I64, _I, _P], _I),
    "moe_experts_up_packed": ([_DIMS, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P], _I),
    "moe_experts_down_grad_packed": ([_DIMS, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _SZ, _P], _I),
    "moe_combine_rows_grad_packed": ([_DIMS, _P, _I64, _P, _P, _P, _P, _P, _P, _P], _I),
})

__all__ = ["moe_train_workspace_size", "moe_dispatch_rows", "moe_dispatch_rows_grad", "moe_combine_rows",
           "moe_combine_rows_grad", "moe_gate_grad", "moe_experts_up", "moe_experts_up_grad", "moe_experts_down",
           "moe_experts_down_grad", "moe_experts_path", "moe_block", "make_block", "moe_norm_rows", "moe_norm_rows_grad",
           "moe_block_out", "moe_block_out_grad", "moe_packed_size", "packed_rows", "moe_pack_rows", "moe_unpack_rows",
           "moe_experts_up_packed", "moe_experts_down_grad_packed", "moe_combine_rows_grad_packed",
           "MOE_GATE_NONE", "MOE_GATE_TOKEN", "MOE_GATE_CHANNEL", "MOE_GATE_FULL"]

MOE_GATE_NONE, MOE_GATE_TOKEN, MOE_GATE_CHANNEL, MOE_GATE_FULL = range(4)

_F32, _I32, _U8, _I8 = torch.float32, torch.int32, torch.uint8, torch.int8
_WTYPE = {MOE_DTYPE_F32: torch.float32, MOE_DTYPE_BF16: torch.bfloat16}
_CODE = {t: c for c, t in _WTYPE.items()}


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
    if t is None and optional:
        return None
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.numel() >= numel:
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(dev, t, dtype, numel, name)


def _rows(dev, t, dtype, T, d, name, optional=False):
    """Address and row stride of token rows [T, d] (contiguous columns); a single row's stride says
    nothing, and d keeps its loads wide."""
    if t is None and optional:
        return None, 0
    try:  # the common case first: a call's host time is its checks
        if t.dtype is dtype and t.get_device() == dev:
            rows, cols = t.shape
            ld, inner = t.stride()
            if cols == d and rows >= T and inner == 1 and ld >= d:
                return t.data_ptr(), ld if T > 1 else d
    except (AttributeError, ValueError):
        pass
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


# ---------------------------------------------------------------- the block around the layer


def make_block(eps=1e-6, weight_offset=0.0, residual_scale=1.0, post_norm=True, gate=MOE_GATE_NONE) -> moe_block:
    """How a block ends: out = residual + residual_scale gate p, p the block's
    output, normed with post_norm; norms multiply by weight_offset + weight."""
    return moe_block(eps, weight_offset, residual_scale, int(bool(post_norm)), int(gate))


def _branch_type(dims, t, name):
    """The type of a block's output (and of its gradient): the layer's, or float32."""
    if t is None:
        return _WTYPE[dims.wtype]
    dtype = getattr(t, "dtype", None)
    if dtype is not _F32 and dtype is not _WTYPE[dims.wtype]:
        raise TypeError(f"{name} has dtype {dtype}, expected {_WTYPE[dims.wtype]} or {_F32}")
    return dtype


def _gate_buf(dev, dims, block, t, name, channel_type, optional):
    """Address of a gate (or its gradient) of the block's kind."""
    wt, T, d = _WTYPE[dims.wtype], dims.T, dims.d
    if block.gate == MOE_GATE_TOKEN:
        return _buf(dev, t, _F32, T, name, optional)
    if block.gate == MOE_GATE_CHANNEL:
        return _buf(dev, t, channel_type, d, name, optional)
    if block.gate == MOE_GATE_FULL:
        return _buf(dev, t, wt, T * d, name, optional)
    if t is not None:
        raise ValueError(f"{name} is given, but the block has no gate")
    return None


def moe_norm_rows(dims, x, weight, eps, weight_offset, n, rstd, stream=None):
    """n [T, d] = x rstd (weight_offset + weight); weight [d] and rstd [T] may be None."""
    dev = _here()
    T, d, wt = dims.T, dims.d, _WTYPE[dims.wtype]
    px, ldx = _rows(dev, x, wt, T, d, "x")
    pn, ldn = _rows(dev, n, wt, T, d, "n")
    _check(lib().moe_norm_rows(dims, px, ldx, _buf(dev, weight, wt, d, "weight", True), float(eps), float(weight_offset),
                               pn, ldn, _buf(dev, rstd, _F32, T, "rstd", True), _queue(dev, stream)), "moe_norm_rows")


def moe_norm_rows_grad(dims, dn, x, rstd, weight, weight_offset, add, dx, dweight, accumulate, ws, stream=None):
    """dx [T, d] = add + the gradient of moe_norm_rows' x; dweight [d] in the
    layer's type or float32 (may be None, as add).  accumulate adds to the
    float32 dweight."""
    dev = _here()
    T, d, wt = dims.T, dims.d, _WTYPE[dims.wtype]
    pdn, lddn = _rows(dev, dn, wt, T, d, "dn")
    px, ldx = _rows(dev, x, wt, T, d, "x")
    padd, ldadd = _rows(dev, add, wt, T, d, "add", True)
    pdx, lddx = _rows(dev, dx, wt, T, d, "dx")
    pw, _, gtype = _grad_type(dev, dims, dweight, None, ("dweight", ""), d)
    _check(lib().moe_norm_rows_grad(
        dims, pdn, lddn, px, ldx, _buf(dev, rstd, _F32, T, "rstd"), _buf(dev, weight, wt, d, "weight", True),
        float(weight_offset), padd, ldadd, pdx, lddx, pw, gtype, int(bool(accumulate)), _buf(dev, ws, _U8, 0, "ws"),
        ws.numel(), _queue(dev, stream)), "moe_norm_rows_grad")


def moe_block_out(dims, block, y, residual, gate, w_post, w_next, out, next, rstd_post, rstd_next, stream=None):
    """out [T, d] = residual + residual_scale gate p, and next [T, d] = out's norm
    (may be None); y in the layer's type or float32; gate as block.gate says;
    w_post, w_next, rstd_post, rstd_next may be None."""
    dev = _here()
    T, d, wt = dims.T, dims.d, _WTYPE[dims.wtype]
    yt = _branch_type(dims, y, "y")
    py, ldy = _rows(dev, y, yt, T, d, "y")
    pr, ldr = _rows(dev, residual, wt, T, d, "residual")
    po, ldo = _rows(dev, out, wt, T, d, "out")
    pn, ldn = _rows(dev, next, wt, T, d, "next", True)
    _check(lib().moe_block_out(
        dims, block, py, ldy, MOE_DTYPE_F32 if yt is _F32 else MOE_DTYPE_BF16, pr, ldr,
        _gate_buf(dev, dims, block, gate, "gate", wt, False), _buf(dev, w_post, wt, d, "w_post", True),
        _buf(dev, w_next, wt, d, "w_next", True), po, ldo, pn, ldn, _buf(dev, rstd_post, _F32, T, "rstd_post", True),
        _buf(dev, rstd_next, _F32, T, "rstd_next", True), _queue(dev, stream)), "moe_block_out")


def moe_block_out_grad(dims, block, dout, dnext, y, out, gate, w_post, w_next, rstd_post, rstd_next, dresidual, dy, dgate,
                       dw_post, dw_next, accumulate, ws, stream=None):
    """Gradients of moe_block_out from dout and dnext (one of them may be None):
    dresidual, dy (y's type), dgate, dw_post, dw_next, each None where it is not
    wanted.  dw_post, dw_next and a channel's dgate share a type, the layer's or
    float32; accumulate adds to them in float32."""
    dev = _here()
    T, d, wt = dims.T, dims.d, _WTYPE[dims.wtype]
    yt = _branch_type(dims, dy if y is None else y, "dy" if y is None else "y")
    branch = dy is not None or dgate is not None or dw_post is not None
    # the sums over the tokens share the first one's type
    first, name = (dw_post, "dw_post") if dw_post is not None else (dw_next, "dw_next") if dw_next is not None else \
        (dgate if block.gate == MOE_GATE_CHANNEL else None, "dgate")
    gdtype = wt if first is None else getattr(first, "dtype", None)
    if gdtype is not _F32 and gdtype is not wt:
        raise TypeError(f"{name} has dtype {gdtype}, expected {wt} or {_F32}")
    pdo, lddo = _rows(dev, dout, wt, T, d, "dout", dnext is not None)
    pdn, lddn = _rows(dev, dnext, wt, T, d, "dnext", True)
    py, ldy = _rows(dev, y, yt, T, d, "y", not branch)
    po, ldo = _rows(dev, out, wt, T, d, "out", dnext is None)
    pdr, lddr = _rows(dev, dresidual, wt, T, d, "dresidual", True)
    pdy, lddy = _rows(dev, dy, yt, T, d, "dy", True)
    _check(lib().moe_block_out_grad(
        dims, block, pdo, lddo, pdn, lddn, py, ldy, MOE_DTYPE_F32 if yt is _F32 else MOE_DTYPE_BF16, po, ldo,
        _gate_buf(dev, dims, block, gate, "gate", wt, not branch), _buf(dev, w_post, wt, d, "w_post", True),
        _buf(dev, w_next, wt, d, "w_next", True),
        _buf(dev, rstd_post, _F32, T, "rstd_post", not (branch and block.post_norm)),
        _buf(dev, rstd_next, _F32, T, "rstd_next", dnext is None), pdr, lddr, pdy, lddy,
        _gate_buf(dev, dims, block, dgate, "dgate", gdtype, True), _buf(dev, dw_post, gdtype, d, "dw_post", True),
        _buf(dev, dw_next, gdtype, d, "dw_next", True), MOE_DTYPE_F32 if gdtype is _F32 else MOE_DTYPE_BF16,
        int(bool(accumulate)), _buf(dev, ws, _U8, 0, "ws"), ws.numel(), _queue(dev, stream)), "moe_block_out_grad")


# ---------------------------------------------------------------- activations in 8 bits


def moe_packed_size(rows: int, cols: int):
    """(bytes of q, bytes of scale) of packed rows."""
    q, e = C.c_size_t(), C.c_size_t()
    _check(lib().moe_packed_size(int(rows), int(cols), C.byref(q), C.byref(e)), "moe_packed_size")
    return q.value, e.value


def packed_rows(rows: int, cols: int, device="cuda"):
    """Buffers for packed rows: q int8 [rows, 32 nb] and scale uint8 [rows, nb]."""
    _, e = moe_packed_size(max(rows, 1), cols)
    nb = e // max(rows, 1)
    return (torch.empty((rows, 32 * nb), dtype=_I8, device=device), torch.empty((rows, nb), dtype=_U8, device=device))


def _packed(dev, q, scale, rows, cols, name, optional=False):
    nb = (cols + 31) // 32
    return (_buf(dev, q, _I8, rows * nb * 32, name + "_q", optional),
            _buf(dev, scale, _U8, rows * nb, name + "_scale", optional))


def _plain_rows(dev, t, name):
    """rows, cols, address, row stride and type code of a tensor [rows, cols]."""
    try:
        code = _CODE[t.dtype]
        rows, cols = t.shape
        ld, inner = t.stride()
        if inner == 1 and ld >= cols and t.get_device() == dev:
            return rows, cols, t.data_ptr(), ld if rows > 1 else cols, code
    except (AttributeError, KeyError, ValueError):
        pass
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise TypeError(f"{name} must be a tensor [rows, cols]")
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {torch.bfloat16} or {torch.float32}")
    rows, cols = t.shape
    p, ld = _rows(dev, t, t.dtype, rows, cols, name)
    return rows, cols, p, ld, MOE_DTYPE_F32 if t.dtype is _F32 else MOE_DTYPE_BF16


def moe_pack_rows(x, q, scale, stream=None):
    """x [rows, cols] (bfloat16 or float32) to 8 bits: q int8, scale uint8 (packed_rows makes them)."""
    dev = _here()
    rows, cols, px, ldx, xtype = _plain_rows(dev, x, "x")
    if getattr(scale, "shape", (0,))[-1] != (cols + 31) // 32:
        raise ValueError(f"scale must be [rows, {(cols + 31) // 32}] for {cols} columns")
    pq, ps = _packed(dev, q, scale, rows, cols, "x")
    _check(lib().moe_pack_rows(rows, cols, px, ldx, xtype, pq, ps, _queue(dev, stream)), "moe_pack_rows")


def moe_unpack_rows(q, scale, index, divisor, out, stream=None):
    """out [rows, cols] (bfloat16 or float32) from packed rows: row index[i] // divisor
    (index None: row i); a negative index, or a row that is not there, gives zeros."""
    dev = _here()
    rows, cols, po, ldo, otype = _plain_rows(dev, out, "out")
    nb = (cols + 31) // 32
    if not isinstance(scale, torch.Tensor) or scale.dim() != 2 or scale.shape[1] != nb:
        raise ValueError(f"scale must be [source rows, {nb}] for {cols} columns")
    src = scale.shape[0]
    pq, ps = _packed(dev, q, scale, src, cols, "x")
    _check(lib().moe_unpack_rows(src, cols, pq, ps, _buf(dev, index, _I32, rows, "index", True), int(divisor), rows, po, ldo,
                                 otype, _queue(dev, stream)), "moe_unpack_rows")


def moe_experts_up_packed(dims, x_perm, expert_offsets, w_gate, w_up, g_q, g_scale, u_q, u_scale, h, ws, stream=None):
    """moe_experts_up with g and u [T*k, I] kept in 8 bits."""
    dev = _here()
    d, I, wt, slots = dims.d, dims.I, _WTYPE[dims.wtype], dims.T * dims.k
    nw = dims.N * I * d
    _check(lib().moe_experts_up_packed(
        dims, _buf(dev, x_perm, wt, slots * d, "x_perm"), _buf(dev, expert_offsets, _I32, dims.N + 1, "expert_offsets"),
        _buf(dev, w_gate, wt, nw, "w_gate"), _buf(dev, w_up, wt, nw, "w_up"), *_packed(dev, g_q, g_scale, slots, I, "g"),
        *_packed(dev, u_q, u_scale, slots, I, "u"), _buf(dev, h, wt, slots * I, "h"), _buf(dev, ws, _U8, 0, "ws"), ws.numel(),
        _queue(dev, stream)), "moe_experts_up_packed")


def moe_experts_down_grad_packed(dims, dy_perm, g_q, g_scale, u_q, u_scale, expert_offsets, w_down, h, dg, du, dw_down,
                                 accumulate, ws, stream=None):
    """dg, du through h = SiLU(g) u from g and u in 8 bits, h [T*k, I] formed anew,
    and dw_down = h^T dy [N, I, d] in the layer's type or float32 (may be None).
    accumulate adds to the float32 buffer."""
    dev = _here()
    d, I, wt, slots = dims.d, dims.I, _WTYPE[dims.wtype], dims.T * dims.k
    nw = dims.N * I * d
    pw, _, gtype = _grad_type(dev, dims, dw_down, None, ("dw_down", ""), nw)
    _check(lib().moe_experts_down_grad_packed(
        dims, _buf(dev, dy_perm, wt, slots * d, "dy_perm"), *_packed(dev, g_q, g_scale, slots, I, "g"),
        *_packed(dev, u_q, u_scale, slots, I, "u"), _buf(dev, expert_offsets, _I32, dims.N + 1, "expert_offsets"),
        _buf(dev, w_down, wt, nw, "w_down"), _buf(dev, h, wt, slots * I, "h"), _buf(dev, dg, wt, slots * I, "dg"),
        _buf(dev, du, wt, slots * I, "du"), pw, gtype, int(bool(accumulate)), _buf(dev, ws, _U8, 0, "ws"), ws.numel(),
        _queue(dev, stream)), "moe_experts_down_grad_packed")


def moe_combine_rows_grad_packed(dims, dout, y_q, y_scale, gate, inv_perm, dy_perm, dgate, stream=None):
    """moe_combine_rows_grad with y_perm [T*k, d] in 8 bits (either output may be None)."""
    dev = _here()
    T, d, wt = dims.T, dims.d, _WTYPE[dims.wtype]
    slots = T * dims.k
    pd, ldd = _rows(dev, dout, wt, T, d, "dout")
    _check(lib().moe_combine_rows_grad_packed(
        dims, pd, ldd, *_packed(dev, y_q, y_scale, slots, d, "y", dgate is None),
        _buf(dev, gate, _F32, slots, "gate", True), _buf(dev, inv_perm, _I32, slots, "inv_perm"),
        _buf(dev, dy_perm, wt, slots * d, "dy_perm", True), _buf(dev, dgate, _F32, slots, "dgate", True),
        _queue(dev, stream)), "moe_combine_rows_grad_packed")
