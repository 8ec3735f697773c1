"""The operators between the layers on the host: their fp64 definitions against
autograd, differences and small tables, every refusal of their C entry points
and of the binding, made before any launch (CPU only: no kernel is started)."""
import ctypes

import pytest
import torch

import block_reference as ref

import ssd_chunked_scan_amd as ssd

F = FAKE = 0x100000   # aligned, never dereferenced: every call below fails validation
OK, NULL, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 5
BIG = (F, 1 << 40)


# ------------------------------------------------------------- definitions


@pytest.mark.parametrize("gate", [True, False])
def test_block_reference_gradients(gate):
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen).double()
    x, res, z, post, pre, scale = r(5, 12), r(5, 12), r(5, 12), r(12), r(12), r(12)
    dy, dst = r(5, 12), r(5, 12)
    alpha, eps = 0.7, 1e-5
    t = [q.clone().requires_grad_() for q in (x, res, z, post, pre, scale)]
    s, _ = ref.block_stream(t[0], t[1], t[2] if gate else None, t[3], t[5], alpha, eps)
    y, _ = ref.block_out(s, t[4], eps)
    ((y * dy).sum() + (s * dst).sum()).backward()
    got = ref.block_backward(x, s.detach(), z if gate else None, post, pre, scale, dy, dst, alpha, eps)
    for name, q in zip(("dx", "dresidual", "dz", "dpost_weight", "dpre_weight", "dscale"), t):
        if name == "dz" and not gate:
            assert got[name] is None
        else:
            assert torch.allclose(got[name][0], q.grad, rtol=1e-10, atol=1e-11), name
    # and against a central difference along one direction of x
    d, h = r(5, 12), 1e-5

    def J(e):
        s, _ = ref.block_stream(x + e * d, res, z if gate else None, post, scale, alpha, eps)
        return float((ref.block_out(s, pre, eps)[0] * dy).sum() + (s * dst).sum())

    assert abs((J(h) - J(-h)) / (2 * h) - float((got["dx"][0] * d).sum())) < 1e-6 * float((got["dx"][0] * d).abs().sum())


def test_mx4_reference_on_a_table():
    """One block with maximum 4 (scale 1): the borders between the values go to
    the even code, above 6 everything is 6."""
    v = [4.0, 0.0, 0.25, 0.26, 0.5, 0.75, 0.74, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 3.49, -0.25, -0.75, -3.5]
    want = [6, 0, 0, 1, 1, 2, 1, 2, 3, 4, 4, 5, 6, 5, 8, 10, 14]
    code, byte = ref.mx4(torch.tensor([v]).double())
    assert code[0, :len(v)].tolist() == want and byte[0].tolist() == [127, 0, 0, 0]
    code, byte = ref.mx4(torch.tensor([[7.99, 5.0, 5.01, -7.0, 4.99]]).double())
    assert code[0, :5].tolist() == [7, 6, 7, 15, 6] and byte[0, 0] == 127
    back = ref.unpack(*ref.pack(code, byte))
    assert back[0, :5].tolist() == [6, 4, 6, -6, 4]


# -------------------------------------------------------------- refusals


def call(name, shape, *pointers, io=1, ws=None):
    lib = ssd.load_library()
    args = [None if shape is None else ctypes.byref(shape), io, *pointers]
    if ws is not None:
        args += list(ws)
    return getattr(lib, name)(*args, None)


def block(**kw):
    s = ssd.BlockShape(10, 256, 0, 0, 0, 0, 0, 1e-5, 1.0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def mx4(**kw):
    s = ssd.Mx4Shape(10, 256, 0, 0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def kept(**kw):
    c = ssd.BlockCheckpoint(F, F, F, F, F, F)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


FWD = [F, F, F, F, F, F, F, F, None]                              # x residual post pre z scale y residual_out ckpt
BWD = [F, F, F, F, F, F, F, F, None, F, F, F, F, F, F]            # x s post pre z scale dy ds ckpt dx dr dz dpost dpre dscale
QUANT, DEQUANT = [F, F, F], [F, F, F]                             # x q scales; q scales y
MATMUL, LINEAR = [F] * 6, [F] * 5                                 # q scales wq wscales bias y; x wq wscales bias y


def put(args, **kw):
    out = list(args)
    for i, v in kw.items():
        out[int(i[1:])] = v
    return out


RESERVED = (ctypes.c_int64 * 4)(0, 0, 1, 0)


@pytest.mark.parametrize("change,status", [
    (dict(rows=0), SHAPE), (dict(columns=0), SHAPE), (dict(rows=-1), SHAPE), (dict(columns=16385), UNSUPPORTED),
    (dict(rows=1 << 30), UNSUPPORTED), (dict(x_stride=255), SHAPE), (dict(z_stride=-256), SHAPE),
    (dict(residual_stride=1), SHAPE), (dict(dy_stride=1), SHAPE), (dict(dresidual_stride=1), SHAPE),
    (dict(x_stride=(1 << 40) + 1), UNSUPPORTED), (dict(eps=0.0), UNSUPPORTED), (dict(eps=float("nan")), UNSUPPORTED),
    (dict(alpha=float("inf")), UNSUPPORTED), (dict(alpha=float("nan")), UNSUPPORTED), (dict(reserved=RESERVED), UNSUPPORTED),
])
def test_block_shapes(change, status):
    s = block(**change)
    assert call("ssd_block_norm_fwd", s, *FWD) == status
    assert call("ssd_block_norm_bwd", s, *BWD, ws=BIG) == status
    lib = ssd.load_library()
    assert lib.ssd_block_norm_bwd_workspace_bytes(ctypes.byref(s), 1) == 0
    assert lib.ssd_last_error()


@pytest.mark.parametrize("args,status", [
    (put(FWD, _0=None), NULL), (put(FWD, _1=None), NULL), (put(FWD, _6=None), NULL), (put(FWD, _7=None), NULL),
    (put(FWD, _0=F + 1), ALIGN), (put(FWD, _2=F + 2), ALIGN), (put(FWD, _3=F + 2), ALIGN), (put(FWD, _4=F + 1), ALIGN),
    (put(FWD, _5=F + 1), ALIGN), (put(FWD, _7=F + 1), ALIGN),
    (put(FWD, _8=kept(x=None)), NULL), (put(FWD, _8=kept(x_scales=None)), NULL), (put(FWD, _8=kept(residual=None)), NULL),
    (put(FWD, _8=kept(z=None)), NULL), (put(FWD, _8=kept(z=None, z_scales=None)), NULL),
    (put(FWD, _4=None, _8=kept()), NULL), (put(FWD, _8=kept(x_scales=F + 2)), ALIGN),
    (put(FWD, _8=kept(z_scales=F + 2)), ALIGN),
])
def test_block_fwd_pointers(args, status):
    assert call("ssd_block_norm_fwd", block(), *args) == status


def test_block_fwd_in_place_is_dense():
    """Rows of residual_out lie elsewhere than a strided residual's."""
    assert call("ssd_block_norm_fwd", block(residual_stride=512), *put(FWD, _7=FWD[1])) == UNSUPPORTED


@pytest.mark.parametrize("args,ws,status", [
    (put(BWD, _0=None), BIG, NULL), (put(BWD, _1=None), BIG, NULL), (put(BWD, _6=None), BIG, NULL),
    (put(BWD, _9=None), BIG, NULL), (put(BWD, _10=None), BIG, NULL), (put(BWD, _11=None), BIG, NULL),
    (put(BWD, _4=None), BIG, NULL), (put(BWD, _2=None), BIG, NULL), (put(BWD, _12=None), BIG, NULL),
    (put(BWD, _3=None), BIG, NULL), (put(BWD, _14=None), BIG, NULL), (put(BWD, _5=None), BIG, NULL),
    (put(BWD, _7=F + 1), BIG, ALIGN), (put(BWD, _13=F + 2), BIG, ALIGN),
    (put(BWD, _8=kept()), BIG, UNSUPPORTED), (put(BWD, _0=None, _1=None, _8=kept()), BIG, UNSUPPORTED),
    (put(BWD, _0=None, _1=None, _4=None, _8=kept(residual_scales=None)), BIG, NULL),
    (put(BWD, _0=None, _1=None, _4=None, _8=kept(z=None)), BIG, NULL),
    (put(BWD, _0=None, _1=None, _4=None, _8=kept(z=None, z_scales=None)), BIG, NULL),     # dz without a gate
    (put(BWD, _0=None, _1=None, _4=None, _11=None, _8=kept()), BIG, NULL),                # a gate without dz
    (BWD, (None, 0), WORKSPACE), (BWD, (F, 100), WORKSPACE), (BWD, (F + 8, 1 << 40), ALIGN),
])
def test_block_bwd_pointers(args, ws, status):
    assert call("ssd_block_norm_bwd", block(), *args, ws=ws) == status


@pytest.mark.parametrize("change,status", [
    (dict(rows=0), SHAPE), (dict(columns=0), SHAPE), (dict(columns=(1 << 20) + 1), UNSUPPORTED),
    (dict(rows=1 << 30), UNSUPPORTED), (dict(x_stride=255), SHAPE), (dict(reserved=RESERVED), UNSUPPORTED),
    (dict(rows=(1 << 28) + 1, columns=1), UNSUPPORTED), (dict(rows=1 << 20, columns=1 << 20), UNSUPPORTED),
])
def test_mx4_shapes(change, status):
    s = mx4(**change)
    assert call("ssd_mx4_quant", s, *QUANT) == status
    assert call("ssd_mx4_dequant", s, *DEQUANT) == status
    s.outputs = 64
    assert call("ssd_mx4_matmul", s, *MATMUL) == status
    assert call("ssd_mx4_linear", s, *LINEAR, ws=BIG) == status
    assert ssd.load_library().ssd_mx4_linear_workspace_bytes(ctypes.byref(s), 1) == 0


def test_mx4_outputs():
    for outputs, status in ((0, SHAPE), (-1, SHAPE), ((1 << 20) + 1, UNSUPPORTED)):
        assert call("ssd_mx4_matmul", mx4(outputs=outputs), *MATMUL) == status
        assert call("ssd_mx4_linear", mx4(outputs=outputs), *LINEAR, ws=BIG) == status
    assert call("ssd_mx4_matmul", mx4(outputs=1 << 20, rows=1 << 18), *MATMUL) == UNSUPPORTED
    assert call("ssd_mx4_quant", mx4(outputs=1), *QUANT) == UNSUPPORTED
    assert call("ssd_mx4_dequant", mx4(outputs=1), *DEQUANT) == UNSUPPORTED
    assert call("ssd_mx4_dequant", mx4(x_stride=256), *DEQUANT) == UNSUPPORTED
    assert call("ssd_mx4_matmul", mx4(outputs=1, x_stride=256), *MATMUL) == UNSUPPORTED


def test_mx4_limits():
    """Fewer than 2^24 workgroups of 16 rows x 512 columns and of 64 x 64 outputs:
    the size beyond is refused, the last one is not (by its next check)."""
    for rows, status in ((1 << 28, UNSUPPORTED), ((1 << 28) - 16, NULL)):
        assert call("ssd_mx4_quant", mx4(rows=rows, columns=512), *put(QUANT, _0=None)) == status
    for rows, status in ((1 << 16, UNSUPPORTED), ((1 << 16) - 64, NULL)):
        assert call("ssd_mx4_matmul", mx4(rows=rows, columns=1, outputs=1 << 20), *put(MATMUL, _0=None)) == status


@pytest.mark.parametrize("name,args,ws,status", [
    ("ssd_mx4_quant", put(QUANT, _0=None), None, NULL), ("ssd_mx4_quant", put(QUANT, _1=None), None, NULL),
    ("ssd_mx4_quant", put(QUANT, _2=None), None, NULL), ("ssd_mx4_quant", put(QUANT, _0=F + 1), None, ALIGN),
    ("ssd_mx4_quant", put(QUANT, _1=F + 8), None, ALIGN), ("ssd_mx4_quant", put(QUANT, _2=F + 2), None, ALIGN),
    ("ssd_mx4_dequant", put(DEQUANT, _0=None), None, NULL), ("ssd_mx4_dequant", put(DEQUANT, _2=None), None, NULL),
    ("ssd_mx4_dequant", put(DEQUANT, _0=F + 4), None, ALIGN), ("ssd_mx4_dequant", put(DEQUANT, _2=F + 1), None, ALIGN),
    ("ssd_mx4_matmul", put(MATMUL, _0=None), None, NULL), ("ssd_mx4_matmul", put(MATMUL, _3=None), None, NULL),
    ("ssd_mx4_matmul", put(MATMUL, _5=None), None, NULL), ("ssd_mx4_matmul", put(MATMUL, _2=F + 8), None, ALIGN),
    ("ssd_mx4_matmul", put(MATMUL, _4=F + 2), None, ALIGN), ("ssd_mx4_matmul", put(MATMUL, _5=F + 1), None, ALIGN),
    ("ssd_mx4_linear", put(LINEAR, _0=None), BIG, NULL), ("ssd_mx4_linear", put(LINEAR, _1=None), BIG, NULL),
    ("ssd_mx4_linear", put(LINEAR, _4=None), BIG, NULL), ("ssd_mx4_linear", put(LINEAR, _2=F + 2), BIG, ALIGN),
])
def test_mx4_pointers(name, args, ws, status):
    assert call(name, mx4(outputs=64 if len(args) > 3 else 0), *args, ws=ws) == status


def test_mx4_linear_workspace():
    lib = ssd.load_library()
    size = lambda rows, columns: lib.ssd_mx4_linear_workspace_bytes(ctypes.byref(mx4(rows=rows, columns=columns, outputs=64)), 1)
    assert size(1, 2560) == size(16, 2560) == 0
    assert size(17, 2560) == 17 * 20 * 64 + 1536      # codes (85 x 256), scales rounded up to 256
    s = mx4(rows=100, outputs=64)
    need = size(100, 256)
    assert need > 0
    for ws, status in (((None, 0), WORKSPACE), ((F, need - 1), WORKSPACE), ((F + 8, need), ALIGN)):
        assert call("ssd_mx4_linear", s, *LINEAR, ws=ws) == status


def test_shape_and_type():
    for name, shape, args, ws in (("ssd_block_norm_fwd", block(), FWD, None), ("ssd_block_norm_bwd", block(), BWD, BIG),
                                  ("ssd_mx4_quant", mx4(), QUANT, None), ("ssd_mx4_dequant", mx4(), DEQUANT, None),
                                  ("ssd_mx4_matmul", mx4(outputs=8), MATMUL, None), ("ssd_mx4_linear", mx4(outputs=8), LINEAR, BIG)):
        assert call(name, None, *args, ws=ws) == NULL
        assert call(name, shape, *args, io=2, ws=ws) == UNSUPPORTED


def test_cpu_tensors_are_refused():
    x, q, s = torch.zeros(4, 128), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8)
    for f in (lambda: ssd.ssd_block_norm_fwd(x, x), lambda: ssd.ssd_block_norm_bwd(x, x, None, None, x),
              lambda: ssd.ssd_mx4_quant(x), lambda: ssd.ssd_mx4_dequant(q, s, 128),
              lambda: ssd.ssd_mx4_matmul(q, s, q, s), lambda: ssd.ssd_mx4_linear(x, q, s)):
        with pytest.raises(ValueError, match="GPU only"):
            f()
