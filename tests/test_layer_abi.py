"""The layer operators' fp64 definitions against autograd and differences, and
every refusal of their C entry points, made on the host before any launch (CPU
only: no kernel is started here)."""
import ctypes

import pytest
import torch

import layer_reference as ref

import ssd_chunked_scan_amd as ssd

FAKE = 0x100000   # aligned, never dereferenced: every call below fails validation
OK, NULL, SHAPE, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 5


def draw(seed):
    gen = torch.Generator().manual_seed(seed)
    return gen, lambda *s: torch.randn(*s, generator=gen).double()


def agree(got, tensors):
    for name, t in tensors.items():
        assert torch.allclose(got[name][0], t.grad, rtol=1e-10, atol=1e-11), name


@pytest.mark.parametrize("normalize", [True, False])
def test_glr_reference_gradients(normalize):
    gen, r = draw(0)
    b, L, D = 2, 40, 6
    x, g, z, A, bias, init = r(b, L, D), r(b, L, D), r(b, L, D), -r(D).abs() - 0.1, r(D), r(b, D)
    seq = (torch.rand(b, L, generator=gen) < 0.1).cumsum(1).int()
    dy, df = r(b, L, D), r(b, D)
    t = [q.clone().requires_grad_() for q in (x, g, z, A, bias, init)]
    m = ref.Glr(t[0], t[1], t[3], t[4], t[2], seq, t[5], normalize)
    (y, _), (f, _) = m.outputs()
    ((y * dy).sum() + (f * df).sum()).backward()
    want = ref.Glr(x, g, A, bias, z, seq, init, normalize).backward(dy, df)
    agree(want, dict(zip(("dx", "dg", "dz", "dA", "dbias", "dinit"), t)))
    # and against a central difference of the definition along one direction
    d = r(b, L, D)
    J = lambda s: sum((o * w).sum() for (o, _), w in
                      zip(ref.Glr(x, g + s * d, A, bias, z, seq, init, normalize).outputs(), (dy, df)))
    h = 1e-5
    diff = float(J(h) - J(-h)) / (2 * h)
    assert abs(diff - float((want["dg"][0] * d).sum())) < 1e-6 * float((want["dg"][0] * d).abs().sum())


@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_reference_gradients(W):
    gen, r = draw(1)
    b, L, D = 2, 23, 5
    x, w, bias, init = r(b, L, D), r(D, W), r(D), r(b, W - 1, D)
    seq = (torch.rand(b, L, generator=gen) < 0.2).cumsum(1).int()
    dy, df = r(b, L, D), r(b, W - 1, D)
    t = [q.clone().requires_grad_() for q in (x, w, bias, init)]
    (y, _), f = ref.conv(t[0], t[1], t[2], seq, t[3], True)
    ((y * dy).sum() + (f * df).sum()).backward()
    agree(ref.conv(x, w, bias, seq, init, True, dy, df), dict(zip(("dx", "dweight", "dbias", "dinit"), t)))


def test_norm_reference_gradients():
    _, r = draw(2)
    x, z, w, dy = r(5, 12), r(5, 12), r(12), r(5, 12)
    t = [q.clone().requires_grad_() for q in (x, z, w)]
    v, _ = ref.norm_input(t[0], None, t[1], None)
    y, *_ = ref.norm(v, 0.0, t[2], 1e-5, 3)
    (y * dy).sum().backward()
    agree(ref.norm_backward(x, z, w, dy, None, 1e-5, 3), dict(zip(("dx", "dz", "dweight"), t)))


# -------------------------------------------------------------- refusals


def call(name, shape, *pointers, io=1, ws=None):
    lib = ssd.load_library()
    args = [None if shape is None else ctypes.byref(shape), io, *pointers]
    if ws is not None:
        args += list(ws)
    return getattr(lib, name)(*args, None)


def glr(**kw):
    s = ssd.GlrShape(2, 300, 64, 0, 0, 0, 0, 1)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def conv(**kw):
    s = ssd.ConvShape(2, 300, 64, 4, 0, 0, 1)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def norm(**kw):
    s = ssd.NormShape(10, 256, 2, 0, 0, 0, 0, 0, 1e-5, 0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


F = FAKE
GLR_FWD = [F, F, F, F, F, F, F, F, F]                 # x g A bias z seq init y final
GLR_BWD = [F, F, F, F, F, F, F, F, F, F, F, F, F, F, F]   # .. dy dfinal dx dg dz dA dbias dinit
GLR_STEP = [F] * 7                                     # x g A bias z state y
CONV_FWD, CONV_BWD, CONV_STEP = [F] * 7, [F] * 11, [F] * 5
NORM_FWD, NORM_QUANT, NORM_BWD = [F, F, F, None, F, F], [F, F, F, None, F, F, F], [F, F, F, F, None, F, F, F]
BIG = (F, 1 << 40)


def put(args, **kw):
    out = list(args)
    for i, v in kw.items():
        out[int(i[1:])] = v
    return out


@pytest.mark.parametrize("change,status", [
    (dict(batch=0), SHAPE), (dict(seqlen=0), SHAPE), (dict(channels=-1), SHAPE),
    (dict(channels=(1 << 20) + 1), UNSUPPORTED), (dict(seqlen=1 << 30), UNSUPPORTED),
    (dict(batch=1 << 20, seqlen=1 << 20), UNSUPPORTED), (dict(batch=1 << 62), UNSUPPORTED),
    (dict(x_stride=63), SHAPE), (dict(g_stride=-64), SHAPE), (dict(z_stride=(1 << 22) + 1), UNSUPPORTED),
    (dict(dy_stride=1), SHAPE), (dict(normalize=2), UNSUPPORTED), (dict(reserved=(ctypes.c_int64 * 4)(0, 0, 0, 1)), UNSUPPORTED),
    (dict(batch=(1 << 30) - 1, seqlen=1, channels=1 << 20), UNSUPPORTED),
])
def test_glr_shapes(change, status):
    s = glr(**change)
    assert call("ssd_glr_fwd", s, *GLR_FWD, ws=BIG) == status
    assert call("ssd_glr_bwd", s, *GLR_BWD, ws=BIG) == status
    lib = ssd.load_library()
    assert lib.ssd_glr_fwd_workspace_bytes(ctypes.byref(s), 1) == 0
    assert lib.ssd_glr_bwd_workspace_bytes(ctypes.byref(s), 1) == 0
    assert lib.ssd_last_error()


@pytest.mark.parametrize("name,args,ws,status", [
    ("ssd_glr_fwd", put(GLR_FWD, _0=None), BIG, NULL), ("ssd_glr_fwd", put(GLR_FWD, _1=None), BIG, NULL),
    ("ssd_glr_fwd", put(GLR_FWD, _2=None), BIG, NULL), ("ssd_glr_fwd", put(GLR_FWD, _7=None), BIG, NULL),
    ("ssd_glr_fwd", put(GLR_FWD, _0=F + 1), BIG, ALIGN), ("ssd_glr_fwd", put(GLR_FWD, _3=F + 2), BIG, ALIGN),
    ("ssd_glr_fwd", put(GLR_FWD, _4=F + 1), BIG, ALIGN), ("ssd_glr_fwd", put(GLR_FWD, _8=F + 2), BIG, ALIGN),
    ("ssd_glr_bwd", GLR_BWD, (None, 0), WORKSPACE), ("ssd_glr_bwd", GLR_BWD, (F, 1000), WORKSPACE),
    ("ssd_glr_bwd", GLR_BWD, (F + 8, 1 << 40), ALIGN),
    ("ssd_glr_bwd", put(GLR_BWD, _11=None), BIG, NULL), ("ssd_glr_bwd", put(GLR_BWD, _4=None), BIG, NULL),
    ("ssd_glr_bwd", put(GLR_BWD, _13=None), BIG, NULL), ("ssd_glr_bwd", put(GLR_BWD, _3=None), BIG, NULL),
    ("ssd_glr_bwd", put(GLR_BWD, _6=None), BIG, NULL), ("ssd_glr_bwd", put(GLR_BWD, _12=None), BIG, NULL),
    ("ssd_glr_bwd", put(GLR_BWD, _7=None), BIG, NULL), ("ssd_glr_bwd", put(GLR_BWD, _9=F + 1), BIG, ALIGN),
])
def test_glr_pointers(name, args, ws, status):
    assert call(name, glr(), *args, ws=ws) == status


def test_strides_of_single_tokens():
    """A step reads one token of each row of a long buffer: its stride may be
    anything that 64 bits address."""
    far = 1 << 40
    assert call("ssd_glr_step", glr(seqlen=1, x_stride=far, g_stride=far), *put(GLR_STEP, _0=None)) == NULL
    assert call("ssd_glr_step", glr(seqlen=1, x_stride=far + 1), *GLR_STEP) == UNSUPPORTED
    assert call("ssd_glr_step", glr(seqlen=1, batch=1 << 24, x_stride=far), *GLR_STEP) == UNSUPPORTED
    assert call("ssd_conv_step", conv(seqlen=1, x_stride=far), *put(CONV_STEP, _0=None)) == NULL
    assert call("ssd_norm_fwd", norm(x_stride=far), *put(NORM_FWD, _0=None)) == NULL
    assert call("ssd_norm_fwd", norm(rows=1 << 21, x_stride=far), *NORM_FWD) == UNSUPPORTED


def test_glr_split_needs_its_workspace():
    s = glr(batch=1, seqlen=4096)
    lib = ssd.load_library()
    need = lib.ssd_glr_fwd_workspace_bytes(ctypes.byref(s), 1)
    assert need > 0
    assert call("ssd_glr_fwd", s, *GLR_FWD, ws=(None, 0)) == WORKSPACE
    assert call("ssd_glr_fwd", s, *GLR_FWD, ws=(F, need - 1)) == WORKSPACE
    assert call("ssd_glr_fwd", s, *GLR_FWD, ws=(F + 4, need)) == ALIGN


@pytest.mark.parametrize("change,status", [
    (dict(batch=0), SHAPE), (dict(channels=0), SHAPE), (dict(width=1), UNSUPPORTED), (dict(width=5), UNSUPPORTED),
    (dict(silu=-1), UNSUPPORTED), (dict(x_stride=10), SHAPE), (dict(dy_stride=(1 << 22) + 1), UNSUPPORTED),
    (dict(seqlen=1 << 31), UNSUPPORTED), (dict(reserved=(ctypes.c_int64 * 4)(1, 0, 0, 0)), UNSUPPORTED),
])
def test_conv_shapes(change, status):
    s = conv(**change)
    assert call("ssd_conv_fwd", s, *CONV_FWD) == status
    assert call("ssd_conv_bwd", s, *CONV_BWD, ws=BIG) == status
    assert ssd.load_library().ssd_conv_bwd_workspace_bytes(ctypes.byref(s), 1) == 0


@pytest.mark.parametrize("name,args,ws,status", [
    ("ssd_conv_fwd", put(CONV_FWD, _0=None), None, NULL), ("ssd_conv_fwd", put(CONV_FWD, _1=None), None, NULL),
    ("ssd_conv_fwd", put(CONV_FWD, _5=None), None, NULL), ("ssd_conv_fwd", put(CONV_FWD, _4=F + 1), None, ALIGN),
    ("ssd_conv_fwd", put(CONV_FWD, _2=F + 1), None, ALIGN),
    ("ssd_conv_bwd", put(CONV_BWD, _5=None), BIG, NULL), ("ssd_conv_bwd", put(CONV_BWD, _7=None), BIG, NULL),
    ("ssd_conv_bwd", put(CONV_BWD, _9=None), BIG, NULL), ("ssd_conv_bwd", put(CONV_BWD, _4=None), BIG, NULL),
    ("ssd_conv_bwd", CONV_BWD, (F, 100), WORKSPACE), ("ssd_conv_bwd", CONV_BWD, (F + 1, 1 << 40), ALIGN),
])
def test_conv_pointers(name, args, ws, status):
    assert call(name, conv(), *args, ws=ws) == status


@pytest.mark.parametrize("change,status", [
    (dict(rows=0), SHAPE), (dict(columns=0), SHAPE), (dict(ngroups=0), SHAPE), (dict(ngroups=3), SHAPE),
    (dict(columns=16385, ngroups=1), UNSUPPORTED), (dict(columns=1 << 20, ngroups=1 << 19), UNSUPPORTED),
    (dict(eps=0.0), UNSUPPORTED), (dict(eps=float("nan")), UNSUPPORTED), (dict(eps=float("inf")), UNSUPPORTED),
    (dict(residual_stride=5), SHAPE), (dict(dresidual_stride=5), SHAPE), (dict(quant_block=64), UNSUPPORTED),
    (dict(reserved=(ctypes.c_int64 * 4)(0, 1, 0, 0)), UNSUPPORTED),
])
def test_norm_shapes(change, status):
    s = norm(**change)
    assert call("ssd_norm_fwd", s, *NORM_FWD) == status
    assert call("ssd_norm_quant_fwd", s, *NORM_QUANT) == status
    assert call("ssd_norm_bwd", s, *NORM_BWD, ws=BIG) == status
    assert ssd.load_library().ssd_norm_bwd_workspace_bytes(ctypes.byref(s), 1) == 0


def test_norm_quant_block_belongs_to_the_8_bit_output():
    assert call("ssd_norm_fwd", norm(quant_block=128), *NORM_FWD) == UNSUPPORTED
    assert call("ssd_norm_bwd", norm(quant_block=128), *NORM_BWD, ws=BIG) == UNSUPPORTED


@pytest.mark.parametrize("name,args,ws,status", [
    ("ssd_norm_fwd", put(NORM_FWD, _0=None), None, NULL), ("ssd_norm_fwd", put(NORM_FWD, _4=None), None, NULL),
    ("ssd_norm_fwd", put(NORM_FWD, _5=None), None, NULL), ("ssd_norm_fwd", put(NORM_FWD, _2=None), None, NULL),
    ("ssd_norm_fwd", put(NORM_FWD, _3=F), None, UNSUPPORTED), ("ssd_norm_fwd", put(NORM_FWD, _1=F + 2), None, ALIGN),
    ("ssd_norm_quant_fwd", put(NORM_QUANT, _5=None), None, NULL), ("ssd_norm_quant_fwd", put(NORM_QUANT, _5=F + 2), None, ALIGN),
    ("ssd_norm_bwd", put(NORM_BWD, _2=F, _4=F), BIG, UNSUPPORTED), ("ssd_norm_bwd", put(NORM_BWD, _6=None), BIG, NULL),
    ("ssd_norm_bwd", put(NORM_BWD, _7=None), BIG, NULL), ("ssd_norm_bwd", put(NORM_BWD, _3=None), BIG, NULL),
    ("ssd_norm_bwd", NORM_BWD, (F, 100), WORKSPACE), ("ssd_norm_bwd", NORM_BWD, (None, 0), WORKSPACE),
])
def test_norm_pointers(name, args, ws, status):
    assert call(name, norm(), *args, ws=ws) == status


def test_shape_and_type():
    for name, args, ws in (("ssd_glr_fwd", GLR_FWD, BIG), ("ssd_glr_bwd", GLR_BWD, BIG), ("ssd_glr_step", GLR_STEP, None),
                           ("ssd_conv_fwd", CONV_FWD, None), ("ssd_conv_bwd", CONV_BWD, BIG), ("ssd_conv_step", CONV_STEP, None),
                           ("ssd_norm_fwd", NORM_FWD, None), ("ssd_norm_quant_fwd", NORM_QUANT, None),
                           ("ssd_norm_bwd", NORM_BWD, BIG)):
        assert call(name, None, *args, ws=ws) == NULL
        shape = {"g": glr, "c": conv, "n": norm}[name[4]]()
        assert call(name, shape, *args, io=2, ws=ws) == UNSUPPORTED
        if name.endswith("step"):
            assert call(name, shape, *args) == SHAPE       # 300 tokens


def test_cpu_tensors_are_refused():
    x, A = torch.zeros(1, 4, 8), -torch.ones(8)
    for f in (lambda: ssd.ssd_glr_fwd(x, x, A), lambda: ssd.ssd_glr_bwd(x, x, A, None, x),
              lambda: ssd.ssd_glr_step(x[0], x[0], A, x[0]), lambda: ssd.ssd_conv_fwd(x, torch.zeros(8, 4)),
              lambda: ssd.ssd_conv_bwd(x, torch.zeros(8, 4), None, x), lambda: ssd.ssd_norm_fwd(x),
              lambda: ssd.ssd_conv_step(x[0], torch.zeros(8, 4), torch.zeros(4, 3, 8)),
              lambda: ssd.ssd_norm_quant_fwd(x), lambda: ssd.ssd_norm_bwd(x, None, x)):
        with pytest.raises(ValueError, match="GPU only"):
            f()
