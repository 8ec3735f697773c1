"""The operators between the layers: block norm with 8-bit checkpoints, and
microscaled 4-bit quantisation and products (include/ssd.h, ssd_block_norm_*,
ssd_mx4_*).  Marshalling only; arguments, streams and outputs as in layer.py.
"""
from __future__ import annotations

import ctypes
from typing import Tuple

import ssd_chunked_scan_amd as ssd
from . import layer
from .layer import _dense, _io, _like, _On, _outputs, _ptr, _tokens, _workspace

_I64, _VP = ctypes.c_int64, ctypes.c_void_p


class BlockShape(ctypes.Structure):
    _fields_ = [("rows", _I64), ("columns", _I64), ("x_stride", _I64), ("z_stride", _I64), ("residual_stride", _I64),
                ("dy_stride", _I64), ("dresidual_stride", _I64), ("eps", ctypes.c_float), ("alpha", ctypes.c_float),
                ("reserved", _I64 * 4)]


class BlockCheckpoint(ctypes.Structure):
    _fields_ = [("x", _VP), ("x_scales", _VP), ("z", _VP), ("z_scales", _VP), ("residual", _VP), ("residual_scales", _VP)]


class Mx4Shape(ctypes.Structure):
    _fields_ = [("rows", _I64), ("columns", _I64), ("outputs", _I64), ("x_stride", _I64), ("reserved", _I64 * 4)]


def declare(lib) -> None:
    """Argument types of these operators' entry points."""
    i32, sz = ctypes.c_int, ctypes.c_size_t
    block, mx4, kept = ctypes.POINTER(BlockShape), ctypes.POINTER(Mx4Shape), ctypes.POINTER(BlockCheckpoint)
    for name, argtypes in (
            ("ssd_block_norm_fwd", [block, i32] + [_VP] * 8 + [kept, _VP]),
            ("ssd_block_norm_bwd", [block, i32] + [_VP] * 8 + [kept] + [_VP] * 7 + [sz, _VP]),
            ("ssd_mx4_quant", [mx4, i32] + [_VP] * 4), ("ssd_mx4_dequant", [mx4, i32] + [_VP] * 4),
            ("ssd_mx4_matmul", [mx4, i32] + [_VP] * 7), ("ssd_mx4_linear", [mx4, i32] + [_VP] * 6 + [sz, _VP])):
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = i32
    for name, shape in (("ssd_block_norm_bwd", block), ("ssd_mx4_linear", mx4)):
        size = getattr(lib, name + "_workspace_bytes")
        size.argtypes = [shape, i32]
        size.restype = sz


# -------------------------------------------------------------- block norm


def _block_common(name, x, z, post_weight, pre_weight, scale, alpha, eps):
    """x: whichever activation gives the shape and the type."""
    io = _io(x, name)
    if x.dim() < 1:
        raise ValueError(f"{name}: x must be [..., D]")
    dev, dt, f32 = x.device, x.dtype, layer.torch.float32
    D = x.shape[-1]
    shape = BlockShape(x.numel() // D if D else 0, D, 0, 0 if z is None else _tokens(z, "z", x.shape, dt, dev), 0, 0, 0, eps,
                       alpha)
    _dense(post_weight, "post_weight", (D,), f32, dev)
    _dense(pre_weight, "pre_weight", (D,), f32, dev)
    _dense(scale, "scale", (D,), f32, dev)
    return io, shape


_KEPT = ("x", "z", "residual")


def _has_gate(checkpoint):
    return checkpoint.get("z_q") is not None or checkpoint.get("z_scales") is not None


def _checkpoint(given, like, gate):
    """The dict of a checkpoint's tensors, new or checked, and its structure."""
    torch = layer.torch
    dev, shape = like.device, like.shape
    scales = (*shape[:-1], -(-shape[-1] // 128))
    fields, out = {}, {}
    for name in _KEPT:
        q, s = name + "_q", name + "_scales"
        if name == "z" and not gate:
            if given is not None and _has_gate(given):
                raise ValueError("checkpoint: z_q and z_scales are given without a gate")
            continue
        if given is None:
            out[q] = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
            out[s] = torch.empty(scales, dtype=torch.float32, device=dev)
        else:
            if given.get(q) is None or given.get(s) is None:
                raise ValueError(f"checkpoint: {q} or {s} is missing")
            _dense(given[q], q, shape, torch.float8_e4m3fn, dev)
            _dense(given[s], s, scales, torch.float32, dev)
            out[q], out[s] = given[q], given[s]
        fields[name], fields[s] = out[q].data_ptr(), out[s].data_ptr()
    return out, BlockCheckpoint(**fields)


def ssd_block_norm_fwd(x, residual, post_weight=None, pre_weight=None, z=None, scale=None, alpha: float = 1.0,
                       eps: float = 1e-5, checkpoint=False, y=None, residual_out=None, stream=None):
    """The seam between two blocks: x [..., D], a block's output, is normed
    (post_weight [D]), gated by silu(z), scaled (scale [D]) and added to alpha
    residual; the sum, rounded to x's dtype, is the residual stream, and its norm
    (pre_weight [D]) the next block's input.  Root-mean-square norms; weights
    and scale fp32, None: 1; z None: no gate.  Returns (y, the residual stream,
    the checkpoint or None).  ``residual_out`` may be ``residual`` itself.

    ``checkpoint`` True (or a dict to write into): 8-bit copies of x, z and
    the stream for ssd_block_norm_bwd, a dict of x_q, z_q, residual_q
    (float8_e4m3fn, x's shape) and x_scales, z_scales, residual_scales (fp32
    [..., ceil(D / 128)]); z's only with z."""
    lib = layer._library()
    io, shape = _block_common("ssd_block_norm_fwd", x, z, post_weight, pre_weight, scale, alpha, eps)
    if not x.is_contiguous():
        shape.x_stride = _tokens(x, "x", x.shape, x.dtype, x.device)
    shape.residual_stride = _tokens(residual, "residual", x.shape, x.dtype, x.device)
    with _On(x.device, stream) as st:
        y = _like(y, "y", x)
        residual_out = _like(residual_out, "residual_out", x)
        kept = struct = None
        if checkpoint is not False and checkpoint is not None:
            kept, struct = _checkpoint(None if checkpoint is True else checkpoint, x, z is not None)
            struct = ctypes.byref(struct)
        status = lib.ssd_block_norm_fwd(ctypes.byref(shape), io, x.data_ptr(), residual.data_ptr(), _ptr(post_weight),
                                        _ptr(pre_weight), _ptr(z), _ptr(scale), y.data_ptr(), residual_out.data_ptr(),
                                        struct, st)
    ssd._check(status)
    return y, residual_out, kept


def ssd_block_norm_bwd(x, residual_out, post_weight, pre_weight, dy, z=None, scale=None, dresidual_out=None,
                       alpha: float = 1.0, eps: float = 1e-5, checkpoint=None, stream=None, workspace=None, out=None):
    """Gradients of ssd_block_norm_fwd from dy and dresidual_out [..., D] (the
    gradient of the residual stream from its other uses, or None): a dict of dx,
    dresidual, dz (dy's dtype; dz None without a gate) and dpost_weight,
    dpre_weight, dscale [D] (fp32; None without the argument).  x and z as the
    forward call saw them and residual_out as it returned it; or None for
    all three, with the ``checkpoint`` that it returned: the gradients at the
    values that the checkpoint holds.  ``out``: the outputs to write, every one
    that is returned."""
    lib = layer._library()
    name = "ssd_block_norm_bwd"
    io, shape = _block_common(name, dy, z, post_weight, pre_weight, scale, alpha, eps)
    dev, dt = dy.device, dy.dtype
    if not dy.is_contiguous():
        shape.dy_stride = _tokens(dy, "dy", dy.shape, dt, dev)
    struct, gate = None, z is not None
    if checkpoint is not None:
        if x is not None or residual_out is not None or z is not None:
            raise ValueError(f"{name}: a checkpoint stands for x, residual_out and z")
        gate = _has_gate(checkpoint)
        _, struct = _checkpoint(checkpoint, dy, gate)
        struct = ctypes.byref(struct)
    else:
        if x is None or residual_out is None:
            raise ValueError(f"{name}: x and residual_out are needed without a checkpoint")
        shape.x_stride = _tokens(x, "x", dy.shape, dt, dev)
        shape.residual_stride = _tokens(residual_out, "residual_out", dy.shape, dt, dev)
    if dresidual_out is not None:
        shape.dresidual_stride = _tokens(dresidual_out, "dresidual_out", dy.shape, dt, dev)
    with _On(dev, stream) as st:
        out = _outputs(out, {"dx": dy, "dresidual": dy, "dz": dy if gate else None, "dpost_weight": post_weight,
                             "dpre_weight": pre_weight, "dscale": scale})
        sums = post_weight is not None or pre_weight is not None or scale is not None
        need = int(lib.ssd_block_norm_bwd_workspace_bytes(ctypes.byref(shape), io)) if sums else 0
        ws = _workspace(workspace, need, dev)
        status = lib.ssd_block_norm_bwd(ctypes.byref(shape), io, _ptr(x), _ptr(residual_out), _ptr(post_weight),
                                        _ptr(pre_weight), _ptr(z), _ptr(scale), dy.data_ptr(), _ptr(dresidual_out), struct,
                                        _ptr(out["dx"]), _ptr(out["dresidual"]), _ptr(out["dz"]),
                                        _ptr(out["dpost_weight"]), _ptr(out["dpre_weight"]), _ptr(out["dscale"]), _ptr(ws),
                                        0 if ws is None else ws.numel(), st)
    ssd._check(status)
    return out


# --------------------------------------------------------- 4-bit operands


def _mx4_rows(name, x):
    if x.dim() < 1:
        raise ValueError(f"{name}: expected [..., columns]")
    D = x.shape[-1]
    return (x.numel() // D if D else 0), D


def _mx4_operand(q, scales, name, scales_name, device):
    """Checks codes and scales; the rows and the padded columns they hold."""
    u8 = layer.torch.uint8
    half = q.shape[-1] if q.dim() else 0
    if half == 0 or half % 64 != 0:
        raise ValueError(f"{name}: expected [..., columns / 2], columns padded to a multiple of 128, got {tuple(q.shape)}")
    rows = q.numel() // half
    _dense(q, name, q.shape, u8, device)
    _dense(scales, scales_name, (half // 64, rows, 4), u8, device)
    return rows, 2 * half


def _mx4_device(name, q):
    if not q.is_cuda:
        raise ValueError(f"{name} runs on the GPU only (on {q.device})")
    return q.device


def _mx4_io(name, dtype) -> int:
    if dtype is layer.torch.bfloat16:
        return 1
    if dtype is layer.torch.float32:
        return 0
    raise TypeError(f"{name}: dtype must be bfloat16 or float32, got {dtype}")


def _mx4_output(given, name, like, shape, dtype):
    """An output on like's device."""
    if given is None:
        return like.new_empty(shape, dtype=dtype)
    _dense(given, name, shape, dtype, like.device)
    return given


def ssd_mx4_quant(x, q=None, scales=None, stream=None) -> Tuple["torch.Tensor", "torch.Tensor"]:
    """x [..., K] in microscaled 4-bit floating point: e2m1 codes with a
    power-of-two scale for each 32 columns.  Returns (q, scales), uint8: q
    [..., kp / 2], two codes a byte, kp = K padded with zeros to a multiple of
    128, and scales [kp / 128, rows, 4], rows the product of x's other dimensions.
    A block with an infinity or a NaN stands for NaN."""
    lib = layer._library()
    io = _io(x, "ssd_mx4_quant")
    rows, K = _mx4_rows("ssd_mx4_quant", x)
    dev, u8 = x.device, layer.torch.uint8
    kb = -(-K // 128)
    shape = Mx4Shape(rows, K, 0, 0 if x.is_contiguous() else _tokens(x, "x", x.shape, x.dtype, dev))
    with _On(dev, stream) as st:
        q = _mx4_output(q, "q", x, (*x.shape[:-1], 64 * kb), u8)
        scales = _mx4_output(scales, "scales", x, (kb, rows, 4), u8)
        status = lib.ssd_mx4_quant(ctypes.byref(shape), io, x.data_ptr(), q.data_ptr(), scales.data_ptr(), st)
    ssd._check(status)
    return q, scales


def ssd_mx4_dequant(q, scales, columns: int, dtype=None, y=None, stream=None) -> "torch.Tensor":
    """The values of ssd_mx4_quant's codes: [..., columns] in ``dtype``, bfloat16
    (the default) or float32, either of which holds them exactly.  (Codes from
    elsewhere may have scale bytes 253 and 254: values past the largest number
    become infinities.)"""
    lib = layer._library()
    name = "ssd_mx4_dequant"
    dev = _mx4_device(name, q)
    dtype = layer.torch.bfloat16 if dtype is None else dtype
    io = _mx4_io(name, dtype)
    rows, kp = _mx4_operand(q, scales, "q", "scales", dev)
    if not kp - 128 < columns <= kp:
        raise ValueError(f"{name}: columns {columns} does not match codes of {kp} padded columns")
    shape = Mx4Shape(rows, columns, 0, 0)
    with _On(dev, stream) as st:
        y = _mx4_output(y, "y", q, (*q.shape[:-1], columns), dtype)
        status = lib.ssd_mx4_dequant(ctypes.byref(shape), io, q.data_ptr(), scales.data_ptr(), y.data_ptr(), st)
    ssd._check(status)
    return y


def _mx4_weights(name, wq, wscales, bias, dev):
    if wq.dim() != 2:
        raise ValueError(f"{name}: wq must be [N, columns / 2], got {tuple(wq.shape)}")
    N, kp = _mx4_operand(wq, wscales, "wq", "wscales", dev)
    if bias is not None:
        _dense(bias, "bias", (N,), layer.torch.float32, dev)
    return N, kp


def ssd_mx4_matmul(q, scales, wq, wscales, bias=None, dtype=None, y=None, stream=None) -> "torch.Tensor":
    """y [..., N] = a w^T + bias of 4-bit operands: a from q and scales, w [N, K]
    from wq and wscales (ssd_mx4_quant of either); sums in fp32, bias [N] fp32,
    y in ``dtype``, bfloat16 (the default) or float32."""
    lib = layer._library()
    name = "ssd_mx4_matmul"
    dev = _mx4_device(name, q)
    dtype = layer.torch.bfloat16 if dtype is None else dtype
    io = _mx4_io(name, dtype)
    rows, kp = _mx4_operand(q, scales, "q", "scales", dev)
    N, wkp = _mx4_weights(name, wq, wscales, bias, dev)
    if wkp != kp:
        raise ValueError(f"{name}: q has {kp} padded columns, wq {wkp}")
    shape = Mx4Shape(rows, kp, N, 0)
    with _On(dev, stream) as st:
        y = _mx4_output(y, "y", q, (*q.shape[:-1], N), dtype)
        status = lib.ssd_mx4_matmul(ctypes.byref(shape), io, q.data_ptr(), scales.data_ptr(), wq.data_ptr(),
                                    wscales.data_ptr(), _ptr(bias), y.data_ptr(), st)
    ssd._check(status)
    return y


def ssd_mx4_linear(x, wq, wscales, bias=None, y=None, workspace=None, stream=None) -> "torch.Tensor":
    """y [..., N] = x w^T + bias with w [N, K] from ssd_mx4_quant and x [..., K]
    quantised the same way as it is read; y in x's dtype.  For activations that
    several products share, ssd_mx4_quant and ssd_mx4_matmul."""
    lib = layer._library()
    name = "ssd_mx4_linear"
    io = _io(x, name)
    rows, K = _mx4_rows(name, x)
    dev = x.device
    N, kp = _mx4_weights(name, wq, wscales, bias, dev)
    if not kp - 128 < K <= kp:
        raise ValueError(f"{name}: x has {K} columns, wq {kp} padded ones")
    shape = Mx4Shape(rows, K, N, 0 if x.is_contiguous() else _tokens(x, "x", x.shape, x.dtype, dev))
    with _On(dev, stream) as st:
        y = _mx4_output(y, "y", x, (*x.shape[:-1], N), x.dtype)
        ws = _workspace(workspace, int(lib.ssd_mx4_linear_workspace_bytes(ctypes.byref(shape), io)), dev)
        status = lib.ssd_mx4_linear(ctypes.byref(shape), io, x.data_ptr(), wq.data_ptr(), wscales.data_ptr(), _ptr(bias),
                                    y.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel(), st)
    ssd._check(status)
    return y
