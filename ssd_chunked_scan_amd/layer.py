"""The layer operators around the scan: gated linear recurrence, causal
depthwise convolution and root-mean-square norm (include/ssd.h, ssd_glr_*,
ssd_conv_*, ssd_norm_*).  Marshalling only, like the rest of the binding: every
step runs in the HIP kernels, on x's device and its current stream (or the raw
stream handle given as ``stream``).

Activations are [b, L, D] ([b, D] for a step, [..., D] for the norm) with the
last dimension contiguous and the tokens evenly spaced, so column slices of a
projection's output are taken as they are; everything else is contiguous.
Outputs are new tensors unless given, and must not overlap inputs.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import ssd_chunked_scan_amd as ssd

torch = None   # from the first call on (_library): the package and the C interface do without it

_I64, _VP = ctypes.c_int64, ctypes.c_void_p


class GlrShape(ctypes.Structure):
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("channels", _I64), ("x_stride", _I64), ("g_stride", _I64),
                ("z_stride", _I64), ("dy_stride", _I64), ("normalize", _I64), ("reserved", _I64 * 4)]


class ConvShape(ctypes.Structure):
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("channels", _I64), ("width", _I64), ("x_stride", _I64),
                ("dy_stride", _I64), ("silu", _I64), ("reserved", _I64 * 4)]


class NormShape(ctypes.Structure):
    _fields_ = [("rows", _I64), ("columns", _I64), ("ngroups", _I64), ("x_stride", _I64), ("z_stride", _I64),
                ("residual_stride", _I64), ("dy_stride", _I64), ("dresidual_stride", _I64),
                ("eps", ctypes.c_float), ("quant_block", ctypes.c_int32), ("reserved", _I64 * 4)]


def declare(lib) -> None:
    """Argument types of the layer operators' entry points."""
    i32, sz = ctypes.c_int, ctypes.c_size_t
    for name, shape, pointers, workspace in (
            ("ssd_glr_fwd", GlrShape, 9, True), ("ssd_glr_bwd", GlrShape, 15, True), ("ssd_glr_step", GlrShape, 7, False),
            ("ssd_conv_fwd", ConvShape, 7, False), ("ssd_conv_bwd", ConvShape, 11, True),
            ("ssd_conv_step", ConvShape, 5, False), ("ssd_norm_fwd", NormShape, 6, False),
            ("ssd_norm_quant_fwd", NormShape, 7, False), ("ssd_norm_bwd", NormShape, 8, True)):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.POINTER(shape), i32] + [_VP] * pointers + ([_VP, sz] if workspace else []) + [_VP]
        fn.restype = i32
        if workspace:
            size = getattr(lib, name + "_workspace_bytes")
            size.argtypes = [ctypes.POINTER(shape), i32]
            size.restype = sz


def _io(x, name: str) -> int:
    if not x.is_cuda:
        raise ValueError(f"{name} runs on the GPU only (x is on {x.device})")
    if x.dtype is torch.bfloat16:
        return 1
    if x.dtype is torch.float32:
        return 0
    raise TypeError(f"x must be bfloat16 or float32, got {x.dtype}")


def _refuse(t, name, shape, dtype, device):
    """Says which of an argument's properties is wrong."""
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _tokens(t, name, shape, dtype, device) -> int:
    """Checks an activation and returns its token stride in elements: the last
    dimension contiguous, all others collapsible to one (size-1 ones aside)."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        _refuse(t, name, shape, dtype, device)
    if t.is_contiguous():
        return 0
    st, stride, span = t.stride(), None, 0
    if shape[-1] != 1 and st[-1] != 1:
        raise ValueError(f"{name}: its last dimension must be contiguous")
    for n, s in zip(reversed(shape[:-1]), reversed(st[:-1])):
        if n == 1:
            continue
        if stride is None:
            stride, span = s, s * n
        elif s != span:
            raise ValueError(f"{name}: its tokens must be evenly spaced (strides {st} of shape {tuple(shape)})")
        else:
            span *= n
    if stride is None:
        return 0   # a single token
    if stride < shape[-1]:
        raise ValueError(f"{name}: tokens must not overlap (token stride {stride})")
    return stride


def _dense(t, name, shape, dtype, device):
    if t is None:
        return
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        _refuse(t, name, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle of a device, without the Stream object around it
# (2 us of a 10 us call), and the current device, where torch offers that.
_raw_stream = _current_device = None


def _library():
    """libssd.so, and torch with the first call."""
    global torch, _raw_stream, _current_device
    if torch is None:
        import torch as module
        _current_device = getattr(module._C, "_cuda_getDevice", module.cuda.current_device)
        _raw_stream = getattr(module._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: module.cuda.current_stream(index).cuda_stream)
        torch = module
    return ssd.load_library()


class _On:
    """The device made current and, with a stream handle given, that stream
    too: what is allocated inside belongs to the stream the kernels run on.
    Does nothing for the usual call, x's device current and no stream given."""
    __slots__ = ("index", "stack", "stream")

    def __init__(self, device, stream):
        self.index, self.stream = device.index, stream
        self.stack = None if stream is None and device.index == _current_device() else contextlib.ExitStack()

    def __enter__(self):
        if self.stack is not None:
            self.stack.enter_context(torch.cuda.device(self.index))
            if self.stream is not None:
                self.stack.enter_context(torch.cuda.stream(
                    torch.cuda.ExternalStream(self.stream, device=self.index) if self.stream
                    else torch.cuda.default_stream(self.index)))
                return self.stream
        return _raw_stream(self.index)

    def __exit__(self, *exc):
        if self.stack is not None:
            self.stack.close()


def _like(given, name, x):
    """An output of x's shape and type."""
    if given is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    _dense(given, name, x.shape, x.dtype, x.device)
    return given


def _output(given, name, shape, dtype, device):
    if given is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _dense(given, name, shape, dtype, device)
    return given


def _workspace(given, need: int, device):
    if given is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    if given.dtype is not torch.uint8 or given.device != device or not given.is_contiguous():
        raise ValueError(f"workspace: a contiguous uint8 tensor on {device}")
    if given.numel() < need:
        raise ValueError(f"workspace: {given.numel()} bytes, {need} needed")
    return given


def _outputs(given, wanted, dinit_type=None):
    """The dict of a backward pass's outputs, each of the shape and type of the
    tensor named for it (dinit of dinit_type): new ones, or those given; None
    where that is None."""
    out = {}
    for name, like in wanted.items():
        if like is None:
            out[name] = None
            continue
        dtype = dinit_type if name == "dinit" and dinit_type is not None else like.dtype
        if given is None:
            out[name] = torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
        else:
            if given.get(name) is None:
                raise ValueError(f"out: {name} is missing")
            _dense(given[name], name, like.shape, dtype, like.device)
            out[name] = given[name]
    return out


def _sequence(x, name):
    if x.dim() != 3:
        raise ValueError(f"{name}: x must be [b, L, D], got {tuple(x.shape)}")
    return x.shape


# ------------------------------------------------- gated linear recurrence


def _glr_common(name, x, g, A, bias, z, seq_idx, init_states, normalize):
    io = _io(x, name)
    dev, dt, f32 = x.device, x.dtype, torch.float32
    b, L, D = _sequence(x, name)
    shape = GlrShape(b, L, D, _tokens(x, "x", x.shape, dt, dev), _tokens(g, "g", x.shape, dt, dev),
                     0 if z is None else _tokens(z, "z", x.shape, dt, dev), 0, 1 if normalize else 0)
    _dense(A, "A", (D,), f32, dev)
    _dense(bias, "bias", (D,), f32, dev)
    _dense(seq_idx, "seq_idx", (b, L), torch.int32, dev)
    _dense(init_states, "init_states", (b, D), f32, dev)
    return io, shape


def ssd_glr_fwd(x, g, A, bias=None, z=None, seq_idx=None, init_states=None, normalize: bool = True,
                return_final_states: bool = True, y=None, final_states=None, workspace=None,
                stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gated linear recurrence h_t = r_t a_t h_{t-1} + k_t x_t over the channels
    of x [b, L, D], a = exp(A softplus(g + bias)), k = sqrt(1 - a^2) with
    ``normalize`` and 1 without, r = 0 where seq_idx [b, L] (int32) changes;
    returns (y, final_states): y = h, or h silu(z) with z, in x's dtype, and the
    fp32 state [b, D] after the last token (None without
    ``return_final_states``).  g, z as x; A (<= 0), bias [D], init_states
    [b, D]: fp32."""
    lib = _library()
    io, shape = _glr_common("ssd_glr_fwd", x, g, A, bias, z, seq_idx, init_states, normalize)
    dev, b, D = x.device, shape.batch, shape.channels
    with _On(dev, stream) as st:
        y = _like(y, "y", x)
        if return_final_states or final_states is not None:
            final_states = _output(final_states, "final_states", (b, D), torch.float32, dev)
        need = int(lib.ssd_glr_fwd_workspace_bytes(ctypes.byref(shape), io))
        ws = _workspace(workspace, need, dev)
        status = lib.ssd_glr_fwd(ctypes.byref(shape), io, x.data_ptr(), g.data_ptr(), A.data_ptr(), _ptr(bias), _ptr(z),
                                 _ptr(seq_idx), _ptr(init_states), y.data_ptr(), _ptr(final_states), _ptr(ws),
                                 0 if ws is None else ws.numel(), st)
    ssd._check(status)
    return y, (final_states if return_final_states else None)


def ssd_glr_bwd(x, g, A, bias, dy, z=None, seq_idx=None, init_states=None, dfinal=None, normalize: bool = True,
                stream=None, workspace=None, out=None):
    """Gradients of J = <dy, y> + <dfinal, final_states> for y, final_states =
    ssd_glr_fwd(x, g, A, bias, z, seq_idx, init_states, normalize): a dict of
    dx, dg, dz (x's dtype), dA, dbias [D] and dinit [b, D] (fp32); dz, dbias and
    dinit are None without z, bias and init_states.  dy as x; dfinal [b, D]
    fp32 or None.  ``out``: the outputs to write, every one that is returned."""
    lib = _library()
    io, shape = _glr_common("ssd_glr_bwd", x, g, A, bias, z, seq_idx, init_states, normalize)
    dev, b, D, f32 = x.device, shape.batch, shape.channels, torch.float32
    shape.dy_stride = _tokens(dy, "dy", x.shape, x.dtype, dev)
    _dense(dfinal, "dfinal", (b, D), f32, dev)
    with _On(dev, stream) as st:
        out = _outputs(out, {"dx": x, "dg": x, "dz": z, "dA": A, "dbias": bias, "dinit": init_states})
        need = int(lib.ssd_glr_bwd_workspace_bytes(ctypes.byref(shape), io))
        ws = _workspace(workspace, need, dev)
        status = lib.ssd_glr_bwd(ctypes.byref(shape), io, x.data_ptr(), g.data_ptr(), A.data_ptr(), _ptr(bias), _ptr(z),
                                 _ptr(seq_idx), _ptr(init_states), dy.data_ptr(), _ptr(dfinal), _ptr(out["dx"]),
                                 _ptr(out["dg"]), _ptr(out["dz"]), _ptr(out["dA"]), _ptr(out["dbias"]),
                                 _ptr(out["dinit"]), _ptr(ws), 0 if ws is None else ws.numel(), st)
    ssd._check(status)
    return out


def ssd_glr_step(x, g, A, state, bias=None, z=None, normalize: bool = True, y=None, stream=None) -> torch.Tensor:
    """One token of ssd_glr_fwd: x, g, z [b, D]; state [b, D] fp32 updated in
    place.  Returns y [b, D]."""
    lib = _library()
    io = _io(x, "ssd_glr_step")
    if x.dim() != 2:
        raise ValueError(f"ssd_glr_step: x must be [b, D], got {tuple(x.shape)}")
    dev, dt, f32 = x.device, x.dtype, torch.float32
    b, D = x.shape
    shape = GlrShape(b, 1, D, _tokens(x, "x", x.shape, dt, dev), _tokens(g, "g", x.shape, dt, dev),
                     0 if z is None else _tokens(z, "z", x.shape, dt, dev), 0, 1 if normalize else 0)
    _dense(A, "A", (D,), f32, dev)
    _dense(bias, "bias", (D,), f32, dev)
    _dense(state, "state", (b, D), f32, dev)
    with _On(dev, stream) as st:
        y = _like(y, "y", x)
        status = lib.ssd_glr_step(ctypes.byref(shape), io, x.data_ptr(), g.data_ptr(), A.data_ptr(), _ptr(bias), _ptr(z),
                                  state.data_ptr(), y.data_ptr(), st)
    ssd._check(status)
    return y


# ------------------------------------------------------------- convolution


def _conv_common(name, x, weight, bias, seq_idx, init_states, silu):
    io = _io(x, name)
    dev, dt, f32 = x.device, x.dtype, torch.float32
    b, L, D = _sequence(x, name)
    if weight.dim() != 2:
        raise ValueError(f"{name}: weight must be [D, W], got {tuple(weight.shape)}")
    W = weight.shape[1]
    shape = ConvShape(b, L, D, W, _tokens(x, "x", x.shape, dt, dev), 0, 1 if silu else 0)
    _dense(weight, "weight", (D, W), f32, dev)
    _dense(bias, "bias", (D,), f32, dev)
    _dense(seq_idx, "seq_idx", (b, L), torch.int32, dev)
    _dense(init_states, "init_states", (b, W - 1, D), dt, dev)
    return io, shape


def ssd_conv_fwd(x, weight, bias=None, seq_idx=None, init_states=None, silu: bool = True,
                 return_final_states: bool = True, y=None, final_states=None,
                 stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal depthwise convolution of x [b, L, D] with weight [D, W] (fp32, W =
    2, 3 or 4; weight[:, W-1] meets the current token) and bias [D], then silu
    unless ``silu`` is False; a document (seq_idx [b, L] int32) does not see the
    one before it.  init_states [b, W-1, D] (x's dtype) are the inputs before
    the row.  Returns (y, final_states): the window [b, W-1, D] the next token
    sees (None without ``return_final_states``)."""
    lib = _library()
    io, shape = _conv_common("ssd_conv_fwd", x, weight, bias, seq_idx, init_states, silu)
    dev = x.device
    with _On(dev, stream) as st:
        y = _like(y, "y", x)
        if return_final_states or final_states is not None:
            final_states = _output(final_states, "final_states", (shape.batch, shape.width - 1, shape.channels), x.dtype,
                                   dev)
        status = lib.ssd_conv_fwd(ctypes.byref(shape), io, x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(seq_idx),
                                  _ptr(init_states), y.data_ptr(), _ptr(final_states), st)
    ssd._check(status)
    return y, (final_states if return_final_states else None)


def ssd_conv_bwd(x, weight, bias, dy, seq_idx=None, init_states=None, dfinal=None, silu: bool = True, stream=None,
                 workspace=None, out=None):
    """Gradients of J = <dy, y> + <dfinal, final_states> for ssd_conv_fwd: a dict
    of dx (x's dtype), dweight [D, W], dbias [D] (None without bias) and dinit
    [b, W-1, D] (None without init_states), fp32.  dy as x; dfinal [b, W-1, D]
    fp32 or None.  ``out``: the outputs to write, every one that is returned."""
    lib = _library()
    io, shape = _conv_common("ssd_conv_bwd", x, weight, bias, seq_idx, init_states, silu)
    dev, f32 = x.device, torch.float32
    b, D, W = shape.batch, shape.channels, shape.width
    shape.dy_stride = _tokens(dy, "dy", x.shape, x.dtype, dev)
    _dense(dfinal, "dfinal", (b, W - 1, D), f32, dev)
    with _On(dev, stream) as st:
        out = _outputs(out, {"dx": x, "dweight": weight, "dbias": bias, "dinit": init_states}, f32)
        need = int(lib.ssd_conv_bwd_workspace_bytes(ctypes.byref(shape), io))
        ws = _workspace(workspace, need, dev)
        status = lib.ssd_conv_bwd(ctypes.byref(shape), io, x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(seq_idx),
                                  _ptr(init_states), dy.data_ptr(), _ptr(dfinal), _ptr(out["dx"]), _ptr(out["dweight"]),
                                  _ptr(out["dbias"]), _ptr(out["dinit"]), _ptr(ws), 0 if ws is None else ws.numel(), st)
    ssd._check(status)
    return out


def ssd_conv_step(x, weight, state, bias=None, silu: bool = True, y=None, stream=None) -> torch.Tensor:
    """One token of ssd_conv_fwd: x [b, D]; state [b, W-1, D] (x's dtype), the
    last W-1 inputs, shifted in place.  Returns y [b, D]."""
    lib = _library()
    io = _io(x, "ssd_conv_step")
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError(f"ssd_conv_step: x must be [b, D] and weight [D, W], got {tuple(x.shape)}, {tuple(weight.shape)}")
    dev, dt, f32 = x.device, x.dtype, torch.float32
    b, D = x.shape
    W = weight.shape[1]
    shape = ConvShape(b, 1, D, W, _tokens(x, "x", x.shape, dt, dev), 0, 1 if silu else 0)
    _dense(weight, "weight", (D, W), f32, dev)
    _dense(bias, "bias", (D,), f32, dev)
    _dense(state, "state", (b, W - 1, D), dt, dev)
    with _On(dev, stream) as st:
        y = _like(y, "y", x)
        status = lib.ssd_conv_step(ctypes.byref(shape), io, x.data_ptr(), weight.data_ptr(), _ptr(bias),
                                   state.data_ptr(), y.data_ptr(), st)
    ssd._check(status)
    return y


# -------------------------------------------------------------------- norm


def _fits(name, value, bits):
    """ctypes drops the bits that a structure's field has no room for."""
    if not -(1 << (bits - 1)) <= value < 1 << (bits - 1):
        raise ValueError(f"{name}: {value} does not fit {bits} bits")


def _norm_common(name, x, weight, z, eps, ngroups):
    _fits("ngroups", ngroups, 64)
    io = _io(x, name)
    if x.dim() < 1:
        raise ValueError(f"{name}: x must be [..., D]")
    dev, dt = x.device, x.dtype
    D = x.shape[-1]
    rows = x.numel() // D if D else 0
    shape = NormShape(rows, D, ngroups, _tokens(x, "x", x.shape, dt, dev),
                      0 if z is None else _tokens(z, "z", x.shape, dt, dev), 0, 0, 0, eps, 0)
    _dense(weight, "weight", (D,), torch.float32, dev)
    return io, shape


def _norm_fwd(name, x, weight, residual, z, eps, ngroups, residual_out):
    io, shape = _norm_common(name, x, weight, z, eps, ngroups)
    if residual is not None:
        shape.residual_stride = _tokens(residual, "residual", x.shape, x.dtype, x.device)
    elif residual_out is not None:
        raise ValueError("residual_out needs residual")
    return io, shape


def ssd_norm_fwd(x, weight=None, residual=None, z=None, eps: float = 1e-5, ngroups: int = 1, y=None, residual_out=None,
                 stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Root-mean-square norm of each row of x [..., D] in ``ngroups`` column
    groups, times weight [D] (fp32, None: 1): of x, of x + residual (rounded to
    x's dtype, the residual stream), or of x silu(z).  Returns (y, the residual
    stream or None).  ``residual_out`` may be ``residual`` itself."""
    lib = _library()
    io, shape = _norm_fwd("ssd_norm_fwd", x, weight, residual, z, eps, ngroups, residual_out)
    with _On(x.device, stream) as st:
        y = _like(y, "y", x)
        if residual is not None:
            residual_out = _like(residual_out, "residual_out", x)
        status = lib.ssd_norm_fwd(ctypes.byref(shape), io, x.data_ptr(), _ptr(weight), _ptr(residual), _ptr(z),
                                  y.data_ptr(), _ptr(residual_out), st)
    ssd._check(status)
    return y, residual_out


def ssd_norm_quant_fwd(x, weight=None, residual=None, z=None, eps: float = 1e-5, ngroups: int = 1, block: int = 128,
                       q=None, scales=None, residual_out=None,
                       stream=None) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """ssd_norm_fwd with an 8-bit output: returns (q, scales, the residual stream
    or None) with y = q * scale, q [..., D] float8_e4m3fn and one fp32 scale =
    max|y| / 448 for each ``block`` = 128 columns of a norm group, or for each
    norm group with ``block`` = 0: scales [..., ngroups * blocks]."""
    lib = _library()
    _fits("block", block, 32)
    io, shape = _norm_fwd("ssd_norm_quant_fwd", x, weight, residual, z, eps, ngroups, residual_out)
    shape.quant_block = block
    per = shape.columns // ngroups if ngroups > 0 else 0
    blocks = -(-per // block) if block > 0 else 1
    with _On(x.device, stream) as st:
        if q is None:
            q = torch.empty_like(x, dtype=torch.float8_e4m3fn, memory_format=torch.contiguous_format)
        else:
            _dense(q, "q", x.shape, torch.float8_e4m3fn, x.device)
        scales = _output(scales, "scales", (*x.shape[:-1], max(ngroups, 0) * blocks), torch.float32, x.device)
        if residual is not None:
            residual_out = _like(residual_out, "residual_out", x)
        status = lib.ssd_norm_quant_fwd(ctypes.byref(shape), io, x.data_ptr(), _ptr(weight), _ptr(residual), _ptr(z),
                                        q.data_ptr(), scales.data_ptr(), _ptr(residual_out), st)
    ssd._check(status)
    return q, scales, residual_out


def ssd_norm_bwd(x, weight, dy, z=None, dresidual=None, eps: float = 1e-5, ngroups: int = 1, stream=None, workspace=None,
                 out=None):
    """Gradients of ssd_norm_fwd from dy [..., D]: a dict of dx, dz (x's dtype; dz
    None without z) and dweight [D] (fp32; None without weight).  x is what the
    norm saw: the forward call's x, or with a residual the stream it returned;
    dresidual, the stream's gradient from its other uses, is added to dx, which
    is the gradient of x and of the residual alike.  ``out``: the outputs to
    write, every one that is returned."""
    lib = _library()
    io, shape = _norm_common("ssd_norm_bwd", x, weight, z, eps, ngroups)
    dev = x.device
    shape.dy_stride = _tokens(dy, "dy", x.shape, x.dtype, dev)
    if dresidual is not None:
        shape.dresidual_stride = _tokens(dresidual, "dresidual", x.shape, x.dtype, dev)
    with _On(dev, stream) as st:
        out = _outputs(out, {"dx": x, "dz": z, "dweight": weight})
        need = int(lib.ssd_norm_bwd_workspace_bytes(ctypes.byref(shape), io)) if weight is not None else 0
        ws = _workspace(workspace, need, dev)
        status = lib.ssd_norm_bwd(ctypes.byref(shape), io, x.data_ptr(), _ptr(weight), _ptr(z), dy.data_ptr(),
                                  _ptr(dresidual), _ptr(out["dx"]), _ptr(out["dz"]), _ptr(out["dweight"]), _ptr(ws),
                                  0 if ws is None else ws.numel(), st)
    ssd._check(status)
    return out
