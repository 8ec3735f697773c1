"""The layer operators on the GPU against their fp64 definitions
(layer_reference.py): every element within a bound that counts the roundings of
the evaluation, at the sizes, strides, masks and types where the kernels take
another path."""
import math

import pytest
import torch

import layer_reference as ref

import ssd_chunked_scan_amd as ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def within(name, got, pair, io=None):
    want, err = pair if io is None else ref.rounded(pair, io)
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= err)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / err).max()):.2f} times the "
                           f"bound, first at {torch.nonzero(bad)[0].tolist()}: {got[bad][0]} for {want[bad][0]}")


def rand(gen, *shape, dtype=torch.float32, scale=1.0):
    """On the GPU, drawn on the CPU; poisoned memory is not an input."""
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).to(DEV)


def cpu(t):
    return None if t is None else t.detach().double().cpu()


def documents(gen, b, L, mean):
    cuts = torch.rand(b, L, generator=gen) < 1.0 / mean
    # document numbers fall and repeat: only a change starts one
    return (cuts.cumsum(1) % 3).to(torch.int32).to(DEV)


def sliced(gen, parts, lead, D, dtype, pad):
    """`parts` column slices of one projection's rows, `pad` columns of NaN in
    front of each."""
    wide = torch.full((*lead, parts * (D + pad)), math.nan)
    for i in range(parts):
        at = i * (D + pad) + pad
        wide[..., at:at + D] = torch.randn(*lead, D, generator=gen)
    wide = wide.to(dtype).to(DEV)
    return [wide[..., i * (D + pad) + pad:(i + 1) * (D + pad)] for i in range(parts)]


# ------------------------------------------------- gated linear recurrence

GLR_CASES = [
    # b, L, D, dtype, gate, normalize, mean document (0: none), init, pad (None: dense)
    (1, 1, 1, "f32", False, True, 0, False, None),
    (1, 1, 2, "bf16", True, True, 0, True, None),
    (3, 2, 34, "bf16", False, False, 1, True, None),
    (2, 7, 33, "bf16", True, True, 2, True, None),
    (2, 127, 32, "f32", True, True, 0, False, None),
    (1, 128, 64, "bf16", False, True, 30, False, 8),
    (1, 129, 66, "f32", False, False, 30, True, None),
    (2, 300, 31, "f32", True, False, 0, True, 3),
    (2, 511, 130, "bf16", True, True, 40, True, 2),
    (1, 513, 96, "bf16", True, True, 0, True, 1),
    (2, 1030, 98, "f32", True, True, 100, True, None),
    (1, 4099, 40, "bf16", False, True, 700, True, None),
    (16, 260, 1056, "bf16", True, True, 90, True, None),      # one split, three rounds
    (3, 901, 1001, "f32", False, True, 0, False, None),
    (4, 140, 4130, "bf16", True, True, 50, True, None),       # 260 strips: on 256 compute units the last 4 in halves
]


def glr_inputs(case, seed=0):
    b, L, D, dtype, gate, normalize, mean, init, pad = case
    gen = torch.Generator().manual_seed(seed)
    io = TYPES[dtype]
    parts = 2 + gate
    cols = sliced(gen, parts, (b, L), D, io, pad) if pad is not None else [rand(gen, b, L, D, dtype=io) for _ in range(parts)]
    dt = torch.exp(torch.rand(D, generator=gen) * math.log(100.0) + math.log(1e-3))
    s = dict(x=cols[0], g=cols[1], z=cols[2] if gate else None,
             bias=torch.log(torch.expm1(dt)).to(DEV), A=-torch.exp(torch.rand(D, generator=gen) * math.log(16.0)).to(DEV),
             seq_idx=documents(gen, b, L, mean) if mean else None, init_states=rand(gen, b, D) if init else None,
             normalize=normalize)
    grad = dict(dy=rand(gen, b, L, D, dtype=io), dfinal=rand(gen, b, D) if init else None)
    return io, s, grad


def glr_reference(s):
    seq = None if s["seq_idx"] is None else s["seq_idx"].cpu()
    return ref.Glr(cpu(s["x"]), cpu(s["g"]), cpu(s["A"]), cpu(s["bias"]), cpu(s["z"]), seq, cpu(s["init_states"]),
                   s["normalize"])


@pytest.mark.parametrize("case", GLR_CASES, ids=str)
def test_glr_fwd(case):
    io, s, _ = glr_inputs(case)
    y, final = ssd.ssd_glr_fwd(**s)
    r = glr_reference(s)
    ry, rf = r.outputs()
    within("y", y, ry, io)
    within("final", final, rf, torch.float32)


@pytest.mark.parametrize("case", GLR_CASES, ids=str)
def test_glr_bwd(case):
    io, s, grad = glr_inputs(case, seed=1)
    got = ssd.ssd_glr_bwd(**s, **grad)
    want = glr_reference(s).backward(cpu(grad["dy"]), cpu(grad["dfinal"]))
    for k in ("dx", "dg", "dz"):
        if want[k] is None:
            assert got[k] is None
        else:
            within(k, got[k], want[k], io)
    within("dA", got["dA"], want["dA"], torch.float32)
    within("dbias", got["dbias"], want["dbias"], torch.float32)
    if s["init_states"] is None:
        assert got["dinit"] is None
    else:
        within("dinit", got["dinit"], want["dinit"], torch.float32)


@pytest.mark.parametrize("case", [GLR_CASES[3], GLR_CASES[9], GLR_CASES[11]], ids=str)
def test_glr_without_bias(case):
    io, s, grad = glr_inputs(case, seed=2)
    s["bias"] = None
    y, final = ssd.ssd_glr_fwd(**s)
    r = glr_reference(s)
    within("y", y, r.outputs()[0], io)
    got = ssd.ssd_glr_bwd(**s, **grad)
    want = r.backward(cpu(grad["dy"]), cpu(grad["dfinal"]))
    assert got["dbias"] is None
    within("dg", got["dg"], want["dg"], io)
    within("dA", got["dA"], want["dA"], torch.float32)


@pytest.mark.parametrize("normalize", [True, False])
def test_glr_extreme_gates(normalize):
    """Gates from decay 0 to decay 1: softplus from 80 to e^-80."""
    v = torch.tensor([-80.0, -40.0, -17.0, -16.0, -8.0, -1.0, -1e-3, 0.0, 1e-3, 1.0, 8.0, 20.0, 40.0, 80.0])
    gen = torch.Generator().manual_seed(5)
    D = v.numel()
    s = dict(x=rand(gen, 2, 150, D), g=v.expand(2, 150, D).contiguous().to(DEV), A=torch.linspace(-0.5, -4.0, D).to(DEV),
             bias=torch.zeros(D, device=DEV), z=None, seq_idx=None, init_states=rand(gen, 2, D), normalize=normalize)
    grad = dict(dy=rand(gen, 2, 150, D), dfinal=rand(gen, 2, D))
    r = glr_reference(s)
    y, final = ssd.ssd_glr_fwd(**s)
    within("y", y, r.outputs()[0], torch.float32)
    within("final", final, r.outputs()[1], torch.float32)
    got = ssd.ssd_glr_bwd(**s, **grad)
    want = r.backward(cpu(grad["dy"]), cpu(grad["dfinal"]))
    for k in want:
        if want[k] is not None:
            within(k, got[k], want[k], torch.float32)


@pytest.mark.parametrize("L", [40, 1500])
def test_glr_nonfinite_values_stay_in_their_document(L):
    """A document with NaN and infinities beside finite ones: the others' values
    and gradients are the ones they have alone."""
    gen = torch.Generator().manual_seed(3)
    D = 34
    seq = torch.zeros(1, L, dtype=torch.int32, device=DEV)
    a, b = L // 3, 2 * L // 3
    seq[:, a:b] = 1
    io, s, grad = glr_inputs((1, L, D, "f32", True, True, 0, True, None), seed=3)
    s["seq_idx"] = seq
    bad = torch.zeros(1, L, D, dtype=torch.bool, device=DEV)
    bad[:, a:b] = True
    dirty = dict(s)
    for k in ("x", "g"):
        dirty[k] = torch.where(bad & (torch.arange(D, device=DEV) % 2 == 0), torch.full_like(s[k], math.nan), s[k])
    dirty["x"] = torch.where(bad & (torch.arange(D, device=DEV) % 2 == 1), torch.full_like(s["x"], math.inf), dirty["x"])
    dy = torch.where(bad, torch.full_like(grad["dy"], -math.nan), grad["dy"])
    y, f = ssd.ssd_glr_fwd(**s)
    yd, fd = ssd.ssd_glr_fwd(**dirty)
    ok = ~bad
    assert torch.equal(yd[ok], y[ok]) and torch.equal(fd, f)
    assert not torch.isfinite(yd[bad]).any()
    g = ssd.ssd_glr_bwd(**s, **grad)
    gd = ssd.ssd_glr_bwd(**dirty, dy=dy, dfinal=grad["dfinal"])
    for k in ("dx", "dg", "dz"):
        assert torch.equal(gd[k][ok], g[k][ok]), k
    assert torch.equal(gd["dinit"], g["dinit"])


@pytest.mark.parametrize("L", [3, 200])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_glr_bwd_outputs_at_any_address(dtype, L):
    """The gradients do not depend on where the outputs lie (from 64-byte
    boundaries to those of one element), and nothing beside them is written."""
    D = 160
    io, s, grad = glr_inputs((2, L, D, dtype, True, True, 40, True, None), seed=9)
    want = ssd.ssd_glr_bwd(**s, **grad)
    exact = glr_reference(s).backward(cpu(grad["dy"]), cpu(grad["dfinal"]))
    for shift in (0, 1, 2, 64 // torch.tensor([], dtype=io).element_size()):
        bufs = {k: torch.full((2 * L * D + 256,), 7., dtype=io, device=DEV) for k in ("dx", "dg", "dz")}
        out = {k: b[64 + shift:64 + shift + 2 * L * D].view(2, L, D) for k, b in bufs.items()}
        out.update({k: torch.empty_like(want[k]) for k in ("dA", "dbias", "dinit")})
        got = ssd.ssd_glr_bwd(**s, **grad, out=out)
        for k in ("dx", "dg", "dz"):
            within(k, got[k], exact[k], io)
            if shift != 1:   # single channels a lane: sums in another order
                assert torch.equal(got[k], want[k]), (k, shift)
            edge = torch.cat([bufs[k][:64 + shift], bufs[k][64 + shift + 2 * L * D:]])
            assert (edge == 7).all(), (k, shift)


@pytest.mark.parametrize("sign", [1., -1.])
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("L", [13, 130, 1400])
def test_glr_a_nan_gate_reaches_the_rest_of_its_document(L, packed, sign):
    """Whatever the sign of the NaN, and with k = 1, where the input's term of the
    recurrence stays finite: forward every token behind it, backward every
    token before it, in its document and in no other."""
    D = 34
    io, s, grad = glr_inputs((2, L, D, "f32", False, True, 0, False, None), seed=8)
    s["normalize"] = False
    lo, hi = (L // 3, 2 * L // 3) if packed else (0, L)
    if packed:
        s["seq_idx"] = torch.zeros(2, L, dtype=torch.int32, device=DEV)
        s["seq_idx"][:, lo:hi] = 1
    at = (lo + hi) // 2
    s["g"] = s["g"].clone()
    s["g"][0, at] = math.copysign(math.nan, sign)
    y, f = ssd.ssd_glr_fwd(**s)
    nan = torch.zeros(2, L, dtype=torch.bool, device=DEV)
    nan[0, at:hi] = True
    assert torch.equal(torch.isnan(y), nan[..., None].expand_as(y))
    assert bool(torch.isnan(f[0]).all()) == (not packed) and torch.isfinite(f[1]).all()
    dx = ssd.ssd_glr_bwd(**s, **grad)["dx"]
    nan = torch.zeros(2, L, dtype=torch.bool, device=DEV)
    nan[0, lo:at] = True
    assert torch.equal(torch.isnan(dx), nan[..., None].expand_as(dx))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [130, 33])
def test_glr_steps_are_the_sequence(dtype, D):
    """Prefill, then token by token: the states and outputs of the whole row."""
    io, s, _ = glr_inputs((3, 12, D, dtype, True, True, 0, True, None), seed=4)
    r = glr_reference(s)
    ry, rf = r.outputs()
    cut = lambda t, lo, hi: None if t is None else t[:, lo:hi]
    part = dict(s, x=s["x"][:, :5], g=s["g"][:, :5], z=s["z"][:, :5])
    part = {k: (v.contiguous() if torch.is_tensor(v) and v.dim() == 3 else v) for k, v in part.items()}
    y, state = ssd.ssd_glr_fwd(**part)
    ys = [y]
    for t in range(5, 12):
        # a token of a longer buffer: rows 12 tokens apart
        ys.append(ssd.ssd_glr_step(s["x"][:, t], s["g"][:, t], s["A"], state, bias=s["bias"], z=s["z"][:, t])[:, None])
    within("y", torch.cat(ys, 1), ry, io)
    within("state", state, rf, torch.float32)


def test_glr_splits_at_every_length():
    """Rows around the lengths where the planner adds a split."""
    for L in (255, 256, 257, 511, 512, 513, 767, 1025):
        io, s, _ = glr_inputs((1, L, 34, "f32", False, True, 60, True, None), seed=L)
        y, final = ssd.ssd_glr_fwd(**s)
        ry, rf = glr_reference(s).outputs()
        within(f"y at {L}", y, ry, io)
        within(f"final at {L}", final, rf, io)


@pytest.mark.parametrize("D", [34, 33])
@pytest.mark.parametrize("L", [15, 16, 17, 31, 63, 64, 65])
def test_glr_around_the_tiles(L, D):
    """Rows of just under, exactly and just over a tile's tokens."""
    io, s, grad = glr_inputs((3, L, D, "f32", True, True, 9, True, None), seed=L)
    y, final = ssd.ssd_glr_fwd(**s)
    r = glr_reference(s)
    within("y", y, r.outputs()[0], io)
    within("final", final, r.outputs()[1], io)
    got = ssd.ssd_glr_bwd(**s, **grad)
    want = r.backward(cpu(grad["dy"]), cpu(grad["dfinal"]))
    for k in want:
        within(k, got[k], want[k], io)
    # and without the states at either end
    s["init_states"] = None
    got = ssd.ssd_glr_bwd(**s, dy=grad["dy"])
    want = glr_reference(s).backward(cpu(grad["dy"]), None)
    assert got["dinit"] is None
    for k in ("dx", "dg", "dz", "dA", "dbias"):
        within(k, got[k], want[k], io)


def directional(J, grads, inputs, gen):
    """<grad, d> against a central difference of J along d, in fp32 outputs
    summed in fp64."""
    for name, grad in grads.items():
        d = torch.randn(inputs[name].shape, generator=gen).to(DEV)
        step = 2.0 ** -7
        lo = J({**inputs, name: inputs[name] - step * d})
        hi = J({**inputs, name: inputs[name] + step * d})
        want = float((hi - lo) / (2 * step))
        got = float((grad.double() * d.double()).sum())
        # truncation: step^2 / 6 times the third derivative along d; the
        # maps here have third derivatives of the order of the sum of the
        # gradient's magnitudes
        size = float((grad.double().abs() * d.double().abs()).sum())
        assert abs(got - want) <= step * size, (name, got, want, size)


def test_glr_gradients_against_differences():
    io, s, grad = glr_inputs((2, 150, 36, "f32", True, True, 40, True, None), seed=6)
    inputs = {k: s[k] for k in ("x", "g", "z", "A", "bias", "init_states")}

    def J(q):
        y, f = ssd.ssd_glr_fwd(**{**s, **q})
        return (y.double() * grad["dy"].double()).sum() + (f.double() * grad["dfinal"].double()).sum()

    g = ssd.ssd_glr_bwd(**s, **grad)
    directional(J, {"x": g["dx"], "g": g["dg"], "z": g["dz"], "A": g["dA"], "bias": g["dbias"],
                    "init_states": g["dinit"]}, inputs, torch.Generator().manual_seed(7))


# ------------------------------------------------------------- convolution

CONV_CASES = [
    # b, L, D, W, dtype, silu, mean document, init, pad, bias
    (1, 1, 1, 2, "f32", True, 0, False, None, True),
    (2, 1, 8, 4, "bf16", True, 0, True, None, True),
    (3, 2, 16, 4, "bf16", True, 1, True, None, False),
    (2, 3, 9, 4, "f32", False, 2, True, None, True),
    (2, 15, 24, 3, "bf16", True, 4, True, 8, True),
    (1, 16, 260, 4, "f32", True, 0, False, None, True),
    (2, 17, 264, 4, "bf16", True, 3, True, None, True),
    (2, 64, 33, 2, "bf16", False, 10, False, 1, False),
    (1, 65, 520, 4, "bf16", True, 2, True, 4, True),
    (3, 257, 136, 4, "f32", True, 20, True, None, True),
    (1, 1030, 72, 3, "f32", True, 100, True, 5, True),
    (4, 2000, 512, 4, "bf16", True, 50, True, None, True),
    (9, 2049, 640, 4, "bf16", True, 300, False, None, True),    # runs of 256 tokens
]


def conv_inputs(case, seed=0):
    b, L, D, W, dtype, silu, mean, init, pad, bias = case
    gen = torch.Generator().manual_seed(seed)
    io = TYPES[dtype]
    x = sliced(gen, 1, (b, L), D, io, pad)[0] if pad is not None else rand(gen, b, L, D, dtype=io)
    s = dict(x=x, weight=rand(gen, D, W, scale=W ** -0.5), bias=rand(gen, D, scale=0.2) if bias else None,
             seq_idx=documents(gen, b, L, mean) if mean else None,
             init_states=rand(gen, b, W - 1, D, dtype=io) if init else None, silu=silu)
    grad = dict(dy=rand(gen, b, L, D, dtype=io), dfinal=rand(gen, b, W - 1, D) if init else None)
    return io, s, grad


def conv_reference(s, dy=None, dfinal=None):
    seq = None if s["seq_idx"] is None else s["seq_idx"].cpu()
    return ref.conv(cpu(s["x"]), cpu(s["weight"]), cpu(s["bias"]), seq, cpu(s["init_states"]), s["silu"], cpu(dy),
                    cpu(dfinal))


@pytest.mark.parametrize("case", CONV_CASES, ids=str)
def test_conv_fwd(case):
    io, s, _ = conv_inputs(case)
    y, final = ssd.ssd_conv_fwd(**s)
    ry, rf = conv_reference(s)
    within("y", y, ry, io)
    assert torch.equal(final.double().cpu(), rf)


@pytest.mark.parametrize("case", CONV_CASES, ids=str)
def test_conv_bwd(case):
    io, s, grad = conv_inputs(case, seed=1)
    got = ssd.ssd_conv_bwd(**s, **grad)
    want = conv_reference(s, **grad)
    within("dx", got["dx"], want["dx"], io)
    within("dweight", got["dweight"], want["dweight"], torch.float32)
    if s["bias"] is None:
        assert got["dbias"] is None
    else:
        within("dbias", got["dbias"], want["dbias"], torch.float32)
    if s["init_states"] is None:
        assert got["dinit"] is None
    else:
        within("dinit", got["dinit"], want["dinit"], torch.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,W", [(40, 4), (33, 3), (64, 2)])
def test_conv_steps_are_the_sequence(dtype, D, W):
    io, s, _ = conv_inputs((3, 12, D, W, dtype, True, 0, True, None, True), seed=4)
    ry, rf = conv_reference(s)
    y, state = ssd.ssd_conv_fwd(**dict(s, x=s["x"][:, :2].contiguous()))
    ys = [y]
    for t in range(2, 12):
        ys.append(ssd.ssd_conv_step(s["x"][:, t], s["weight"], state, bias=s["bias"])[:, None])
    within("y", torch.cat(ys, 1), ry, io)
    assert torch.equal(state.double().cpu(), rf)


@pytest.mark.parametrize("L", [9, 70])
def test_conv_nonfinite_values_stay_in_their_document(L):
    io, s, grad = conv_inputs((1, L, 16, 4, "f32", True, 0, True, None, True), seed=3)
    seq = torch.zeros(1, L, dtype=torch.int32, device=DEV)
    a, b = L // 3, 2 * L // 3
    seq[:, a:b] = 1
    s["seq_idx"] = seq
    bad = torch.zeros(1, L, 16, dtype=torch.bool, device=DEV)
    bad[:, a:b] = True
    ok = ~bad
    dirty = dict(s, x=torch.where(bad, torch.full_like(s["x"], math.nan), s["x"]))
    dy = torch.where(bad, torch.full_like(grad["dy"], math.inf), grad["dy"])
    y, f = ssd.ssd_conv_fwd(**s)
    yd, fd = ssd.ssd_conv_fwd(**dirty)
    assert torch.equal(yd[ok], y[ok]) and torch.equal(fd, f)
    g, gd = ssd.ssd_conv_bwd(**s, **grad), ssd.ssd_conv_bwd(**dirty, dy=dy, dfinal=grad["dfinal"])
    assert torch.equal(gd["dx"][ok], g["dx"][ok]) and torch.equal(gd["dinit"], g["dinit"])


def test_conv_gradients_against_differences():
    io, s, grad = conv_inputs((2, 70, 36, 4, "f32", True, 15, True, None, True), seed=6)
    inputs = {k: s[k] for k in ("x", "weight", "bias", "init_states")}

    def J(q):
        y, f = ssd.ssd_conv_fwd(**{**s, **q})
        return (y.double() * grad["dy"].double()).sum() + (f.double() * grad["dfinal"].double()).sum()

    g = ssd.ssd_conv_bwd(**s, **grad)
    directional(J, {"x": g["dx"], "weight": g["dweight"], "bias": g["dbias"], "init_states": g["dinit"]}, inputs,
                torch.Generator().manual_seed(7))


# -------------------------------------------------------------------- norm

NORM_CASES = [
    # rows, columns, ngroups, dtype, kind, pad, weight
    (1, 1, 1, "f32", "plain", None, True),
    (1, 8, 1, "bf16", "residual", None, True),
    (3, 40, 1, "bf16", "gate", None, True),
    (5, 129, 1, "f32", "residual", None, True),
    (7, 257, 1, "bf16", "gate", 1, True),
    (4, 512, 4, "bf16", "plain", 8, False),
    (9, 1477, 7, "f32", "plain", None, True),
    (17, 2560, 1, "bf16", "residual", None, True),
    (6, 2568, 1, "f32", "gate", 4, True),
    (2100, 200, 1, "bf16", "residual", None, True),     # a wave per row
    (2049, 1032, 1, "bf16", "gate", None, True),
    (600, 1536, 2, "f32", "plain", None, True),
    (3, 4104, 1, "bf16", "gate", None, True),
    (2, 8195, 1, "f32", "residual", None, True),        # over 8192 single elements
    (2, 8195, 1, "bf16", "gate", None, True),
    (2, 16384, 1, "bf16", "gate", None, True),
    (2, 16384, 1, "f32", "residual", None, True),
    (2, 32768, 2, "f32", "plain", None, True),
]


def norm_inputs(case, seed=0):
    rows, columns, ngroups, dtype, kind, pad, weight = case
    gen = torch.Generator().manual_seed(seed)
    io = TYPES[dtype]
    other = kind != "plain"
    cols = sliced(gen, 1 + other, (rows,), columns, io, pad) if pad is not None else \
        [rand(gen, rows, columns, dtype=io) for _ in range(1 + other)]
    s = dict(x=cols[0], weight=1 + rand(gen, columns, scale=0.2) if weight else None, eps=1e-5, ngroups=ngroups,
             residual=cols[1] if kind == "residual" else None, z=cols[1] if kind == "gate" else None)
    return io, s, gen


def norm_reference(s, io):
    v, ev = ref.norm_input(cpu(s["x"]), cpu(s["residual"]), cpu(s["z"]), io)
    y, ey, *_ = ref.norm(v, ev, cpu(s["weight"]), s["eps"], s["ngroups"])
    return (y, ey), v


@pytest.mark.parametrize("case", NORM_CASES, ids=str)
def test_norm_fwd(case):
    io, s, _ = norm_inputs(case)
    y, stream = ssd.ssd_norm_fwd(**s)
    ry, v = norm_reference(s, io)
    within("y", y, ry, io)
    if s["residual"] is None:
        assert stream is None
    else:
        assert torch.equal(stream.double().cpu(), v)


def e4m3_bound(t):
    """Half a step of e4m3 at t: 2^-4 relative, and 2^-10 below 2^-6."""
    return torch.maximum(t.abs() * 2.0 ** -4, torch.full_like(t, 2.0 ** -10))


@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("case", NORM_CASES, ids=str)
def test_norm_quant_fwd(case, block):
    io, s, _ = norm_inputs(case, seed=1)
    q, scales, stream = ssd.ssd_norm_quant_fwd(**s, block=block)
    (y, ey), v = norm_reference(s, io)
    rows, columns = y.shape
    per = columns // s["ngroups"]
    width = block or per
    y, ey = y.reshape(rows, s["ngroups"], per), ey.reshape(rows, s["ngroups"], per)
    sc = scales.double().cpu().reshape(rows, s["ngroups"], -(-per // width))
    got = q.float().double().cpu().reshape(y.shape)
    for i in range(sc.shape[-1]):
        part = slice(i * width, min(per, (i + 1) * width))
        m = y[..., part].abs().amax(-1).clamp(min=1e-12)
        assert (sc[..., i] - m / 448).abs().le((ey[..., part].amax(-1) + 2 * ref.U * m) / 448).all()
        t = y[..., part] / sc[..., i, None]
        # the value before its rounding: y's bound and three roundings
        fuzz = ey[..., part] / sc[..., i, None] + 4 * ref.U * t.abs()
        off = (got[..., part] - t).abs()
        assert off.le(e4m3_bound(t.abs() + fuzz) + fuzz).all(), float((off - e4m3_bound(t)).max())
    if stream is not None:
        assert torch.equal(stream.double().cpu(), v)


def test_norm_quant_zero_and_nonfinite_rows():
    x = torch.zeros(4, 256, device=DEV)
    x[1, 3] = 1e-30
    x[2, 200] = math.nan
    x[3, 5] = math.inf
    q, scales, _ = ssd.ssd_norm_quant_fwd(x, None)
    tiny = torch.tensor(1e-12) / 448
    assert torch.equal(scales[0].cpu(), tiny.expand(2)) and not q[0].float().any()
    assert torch.isfinite(scales[1]).all() and torch.isfinite(q[1].float()).all()
    # a NaN anywhere makes the row's statistic NaN
    assert torch.isnan(scales[2]).all() and torch.isnan(q[2].float()).all()
    # an infinity makes the statistic infinite: inf * 0 at its place, 0 elsewhere
    assert torch.isnan(scales[3, 0]) and torch.isnan(q[3, :128].float()).all()
    assert torch.equal(scales[3, 1:].cpu(), tiny.expand(1)) and not q[3, 128:].float().any()
    # a NaN weight only spoils its own block
    w = torch.ones(256, device=DEV)
    w[130] = math.nan
    q, scales, _ = ssd.ssd_norm_quant_fwd(torch.ones(1, 256, device=DEV), w)
    assert torch.isfinite(scales[0, 0]) and torch.isnan(scales[0, 1])
    assert torch.isfinite(q[0, :128].float()).all() and torch.isnan(q[0, 128:].float()).all()


@pytest.mark.parametrize("case", NORM_CASES, ids=str)
def test_norm_bwd(case):
    io, s, gen = norm_inputs(case, seed=2)
    kind = case[4]
    dy = rand(gen, *s["x"].shape, dtype=io)
    dres = rand(gen, *s["x"].shape, dtype=io) if kind == "residual" else None
    got = ssd.ssd_norm_bwd(s["x"], s["weight"], dy, z=s["z"], dresidual=dres, eps=s["eps"], ngroups=s["ngroups"])
    want = ref.norm_backward(cpu(s["x"]), cpu(s["z"]), cpu(s["weight"]), cpu(dy), cpu(dres), s["eps"], s["ngroups"])
    within("dx", got["dx"], want["dx"], io)
    if kind == "gate":
        within("dz", got["dz"], want["dz"], io)
    else:
        assert got["dz"] is None
    if s["weight"] is None:
        assert got["dweight"] is None
    else:
        within("dweight", got["dweight"], want["dweight"], torch.float32)


def test_norm_gradients_against_differences():
    io, s, gen = norm_inputs((6, 72, 3, "f32", "gate", None, True), seed=6)
    dy = rand(gen, 6, 72)
    inputs = {k: s[k] for k in ("x", "z", "weight")}
    g = ssd.ssd_norm_bwd(s["x"], s["weight"], dy, z=s["z"], eps=s["eps"], ngroups=3)
    directional(lambda q: (ssd.ssd_norm_fwd(**{**s, **q})[0].double() * dy.double()).sum(),
                {"x": g["dx"], "z": g["dz"], "weight": g["dweight"]}, inputs, gen)


def test_norm_residual_in_place_and_leading_dimensions():
    gen = torch.Generator().manual_seed(8)
    x, r = rand(gen, 2, 3, 136, dtype=torch.bfloat16), rand(gen, 2, 3, 136, dtype=torch.bfloat16)
    w = rand(gen, 136)
    y, stream = ssd.ssd_norm_fwd(x, w, residual=r)
    again = r.clone()
    y2, same = ssd.ssd_norm_fwd(x, w, residual=again, residual_out=again)
    assert same is again and torch.equal(again, stream) and torch.equal(y, y2) and y.shape == x.shape
    assert torch.equal(stream, (x.float() + r.float()).bfloat16())
    q, scales, s3 = ssd.ssd_norm_quant_fwd(x, w, residual=r)
    assert scales.shape == (2, 3, 2) and q.dtype is torch.float8_e4m3fn and torch.equal(s3, stream)
    one, _ = ssd.ssd_norm_fwd(x[0, 0], w)
    assert torch.equal(one, ssd.ssd_norm_fwd(x, w)[0][0, 0])


# ----------------------------------------------------- streams and buffers


def every_call(seed=0):
    """name -> a call that returns its output tensors, on fixed inputs."""
    _, g, gg = glr_inputs((2, 700, 66, "bf16", True, True, 90, True, None), seed)
    _, c, cg = conv_inputs((2, 200, 72, 4, "bf16", True, 30, True, None, True), seed)
    io, n, gen = norm_inputs((40, 264, 1, "bf16", "residual", None, True), seed)
    dy = rand(gen, 40, 264, dtype=io)
    flat = lambda d: [t for t in (d.values() if isinstance(d, dict) else d) if t is not None]
    return {
        "glr_fwd": lambda **k: flat(ssd.ssd_glr_fwd(**g, **k)),
        "glr_bwd": lambda **k: flat(ssd.ssd_glr_bwd(**g, **gg, **k)),
        "conv_fwd": lambda **k: flat(ssd.ssd_conv_fwd(**c, **k)),
        "conv_bwd": lambda **k: flat(ssd.ssd_conv_bwd(**c, **cg, **k)),
        "norm_fwd": lambda **k: flat(ssd.ssd_norm_fwd(**n, **k)),
        "norm_quant": lambda **k: flat(ssd.ssd_norm_quant_fwd(**n, **k)),
        "norm_bwd": lambda **k: flat(ssd.ssd_norm_bwd(n["x"], n["weight"], dy, dresidual=n["residual"], **k)),
    }


NAMES = ["glr_fwd", "glr_bwd", "conv_fwd", "conv_bwd", "norm_fwd", "norm_quant", "norm_bwd"]


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x.float(), y.float()) for x, y in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
def test_repeatable_on_another_stream(name):
    call = every_call()[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    handle = call(stream=side.cuda_stream)
    side.synchronize()
    assert same(handle, want)
    with torch.cuda.stream(side):
        under = call()
    side.synchronize()
    assert same(under, want)
    assert same(call(stream=0), want)


@pytest.mark.parametrize("name", NAMES)
def test_graph_replays(name):
    """Captured once, replayed between eager work, the inputs kept: the eager
    result each time."""
    call = every_call()[name]
    want = call()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = call()
    for k in range(4):
        for t in out:
            t.view(torch.uint8).fill_(0xFF)
        busy = torch.randn(1 << 20, device=DEV).sum()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want), k
        assert same(call(), want) and torch.isfinite(busy)


@pytest.mark.parametrize("name,bytes_of", [("glr_fwd", None), ("glr_bwd", None), ("conv_bwd", None), ("norm_bwd", None)])
def test_poisoned_workspace(name, bytes_of):
    call = every_call()[name]
    want = call()
    for fill in (0x00, 0xFF):
        ws = torch.full((64 << 20,), fill, dtype=torch.uint8, device=DEV)
        assert same(call(workspace=ws), want)


def test_rows_beside_the_outputs_are_untouched():
    """Outputs inside larger buffers: what lies in front and behind stays."""
    for D, dtype in ((66, torch.bfloat16), (33, torch.float32)):
        case = (2, 130, D, "bf16" if dtype is torch.bfloat16 else "f32", False, True, 0, False, None)
        _, s, grad = glr_inputs(case)
        n = 2 * 130 * D
        buf = torch.full((n + 2 * 256,), 7.0, dtype=dtype, device=DEV)
        y = buf[256:256 + n].view(2, 130, D)
        ssd.ssd_glr_fwd(**s, y=y)
        assert (buf[:256] == 7).all() and (buf[256 + n:] == 7).all() and torch.isfinite(y).all()
        w = torch.ones(D, 4, device=DEV)
        buf.fill_(7.0)
        ssd.ssd_conv_fwd(s["x"], w, y=y)
        assert (buf[:256] == 7).all() and (buf[256 + n:] == 7).all()
        buf.fill_(7.0)
        ssd.ssd_norm_fwd(s["x"], None, y=y)
        assert (buf[:256] == 7).all() and (buf[256 + n:] == 7).all()


def test_offsets_past_32_bits():
    """A token offset over 2^32 bytes: one long row of a wide projection."""
    L, W, D = 70000, 32768, 16        # 4.6 GB of bf16
    wide = torch.zeros(1, L, W, dtype=torch.bfloat16, device=DEV)
    gen = torch.Generator().manual_seed(9)
    x, g = rand(gen, 1, L, D, dtype=torch.bfloat16), rand(gen, 1, L, D, dtype=torch.bfloat16)
    wide[..., W - D:] = x
    wide[..., W - 2 * D:W - D] = g
    A, bias = torch.full((D,), -4.0, device=DEV), torch.full((D,), -3.0, device=DEV)
    xs, gs = wide[..., W - D:], wide[..., W - 2 * D:W - D]
    y, f = ssd.ssd_glr_fwd(xs, gs, A, bias=bias)
    y2, f2 = ssd.ssd_glr_fwd(x, g, A, bias=bias)
    assert torch.equal(y, y2) and torch.equal(f, f2)
    b1 = ssd.ssd_glr_bwd(xs, gs, A, bias, x)
    b2 = ssd.ssd_glr_bwd(x, g, A, bias, x)
    assert all(torch.equal(b1[k], b2[k]) for k in ("dx", "dg", "dA", "dbias"))
    w = rand(gen, D, 4)
    assert torch.equal(ssd.ssd_conv_fwd(xs, w)[0], ssd.ssd_conv_fwd(x, w)[0])
    c1, c2 = ssd.ssd_conv_bwd(xs, w, None, x), ssd.ssd_conv_bwd(x, w, None, x)
    assert torch.equal(c1["dx"], c2["dx"]) and torch.equal(c1["dweight"], c2["dweight"])
    assert torch.equal(ssd.ssd_norm_fwd(xs, None)[0], ssd.ssd_norm_fwd(x, None)[0])
    n1, n2 = ssd.ssd_norm_bwd(xs, None, gs), ssd.ssd_norm_bwd(x, None, g)
    assert torch.equal(n1["dx"], n2["dx"])


def test_single_tokens_far_apart():
    """One token of each row of a long, wide buffer."""
    gen = torch.Generator().manual_seed(10)
    b, L, W, D = 3, 2000, 6000, 64
    wide = torch.zeros(b, L, W, dtype=torch.bfloat16, device=DEV)
    x, g, z = (rand(gen, b, D, dtype=torch.bfloat16) for _ in range(3))
    for i, t in enumerate((x, g, z)):
        wide[:, 7, i * D:(i + 1) * D] = t
    xs, gs, zs = (wide[:, 7, i * D:(i + 1) * D] for i in range(3))
    A, bias = -1 - rand(gen, D).abs(), rand(gen, D) - 2
    s1, s2 = (torch.ones(b, D, device=DEV) for _ in range(2))
    assert torch.equal(ssd.ssd_glr_step(xs, gs, A, s1, bias=bias, z=zs), ssd.ssd_glr_step(x, g, A, s2, bias=bias, z=z))
    assert torch.equal(s1, s2)
    seq = lambda t: t[:, None]
    assert torch.equal(ssd.ssd_glr_fwd(seq(xs), seq(gs), A, bias=bias)[0], ssd.ssd_glr_fwd(seq(x), seq(g), A, bias=bias)[0])
    w = rand(gen, D, 4)
    c1, c2 = (torch.ones(b, 3, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    assert torch.equal(ssd.ssd_conv_step(xs, w, c1), ssd.ssd_conv_step(x, w, c2)) and torch.equal(c1, c2)
    assert torch.equal(ssd.ssd_conv_fwd(seq(xs), w)[0], ssd.ssd_conv_fwd(seq(x), w)[0])
    d1, d2 = ssd.ssd_conv_bwd(seq(xs), w, None, seq(gs)), ssd.ssd_conv_bwd(seq(x), w, None, seq(g))
    assert torch.equal(d1["dx"], d2["dx"]) and torch.equal(d1["dweight"], d2["dweight"])
    g1, g2 = ssd.ssd_glr_bwd(seq(xs), seq(gs), A, bias, seq(zs)), ssd.ssd_glr_bwd(seq(x), seq(g), A, bias, seq(z))
    assert all(torch.equal(g1[k], g2[k]) for k in ("dx", "dg", "dA", "dbias"))
    assert torch.equal(ssd.ssd_norm_fwd(xs, None, z=zs)[0], ssd.ssd_norm_fwd(x, None, z=z)[0])


# -------------------------------------------------------------- refusals


def test_refusals_of_tensors():
    x = torch.zeros(2, 8, 16, dtype=torch.bfloat16, device=DEV)
    A = torch.full((16,), -1.0, device=DEV)
    state = torch.zeros(2, 16, device=DEV)
    w = torch.zeros(16, 4, device=DEV)
    with pytest.raises(ValueError):
        ssd.ssd_glr_fwd(x.cpu(), x, A)
    with pytest.raises(TypeError):
        ssd.ssd_glr_fwd(x.half(), x.half(), A)
    with pytest.raises(TypeError):
        ssd.ssd_glr_fwd(x, x.float(), A)
    with pytest.raises(ValueError):
        ssd.ssd_glr_fwd(x, x[:, :7], A)
    with pytest.raises(ValueError):
        ssd.ssd_glr_fwd(x.transpose(1, 2), x.transpose(1, 2), A)            # channels not contiguous
    with pytest.raises(ValueError):
        ssd.ssd_glr_fwd(torch.zeros(2, 16, 16, dtype=x.dtype, device=DEV)[:, :8], x, A)   # rows not evenly spaced
    with pytest.raises(ValueError):
        ssd.ssd_glr_fwd(x[:, :1].expand(2, 8, 16), x, A)                    # overlapping tokens
    with pytest.raises(TypeError):
        ssd.ssd_glr_fwd(x, x, A.double())
    with pytest.raises(TypeError):
        ssd.ssd_glr_fwd(x, x, A, seq_idx=torch.zeros(2, 8, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        ssd.ssd_glr_fwd(x, x, A, workspace=torch.zeros(4, device=DEV))
    with pytest.raises(ValueError):
        ssd.ssd_glr_bwd(x, x, A, None, x, out={"dx": x.clone()})
    with pytest.raises(ValueError):
        ssd.ssd_glr_step(x, x, A, state)
    with pytest.raises(ssd.SsdError):
        ssd.ssd_glr_fwd(x[:, :0], x[:, :0], A)
    with pytest.raises(ssd.SsdError):
        ssd.ssd_conv_fwd(x, torch.zeros(16, 5, device=DEV))
    with pytest.raises(ValueError):
        ssd.ssd_conv_fwd(x, w.t())
    with pytest.raises(TypeError):
        ssd.ssd_conv_fwd(x, w, init_states=torch.zeros(2, 3, 16, device=DEV))
    with pytest.raises(ValueError):
        ssd.ssd_conv_step(x[:, 0], w, torch.zeros(2, 4, 16, dtype=x.dtype, device=DEV))
    with pytest.raises(ssd.SsdError):
        ssd.ssd_norm_fwd(x, None, residual=x, z=x)
    with pytest.raises(ssd.SsdError):
        ssd.ssd_norm_fwd(x, None, ngroups=3)
    with pytest.raises(ssd.SsdError):
        ssd.ssd_norm_fwd(x, None, ngroups=0)
    with pytest.raises(ssd.SsdError):
        ssd.ssd_norm_fwd(x, None, eps=0.0)
    with pytest.raises(ssd.SsdError):
        ssd.ssd_norm_quant_fwd(x, None, block=64)
    with pytest.raises(ssd.SsdError):
        ssd.ssd_norm_bwd(x, None, x, z=x, dresidual=x)
    with pytest.raises(ValueError):
        ssd.ssd_norm_fwd(x, None, residual_out=x.clone())
    with pytest.raises(ssd.SsdError):
        ssd.ssd_norm_fwd(torch.zeros(1, 16385, device=DEV), None)
