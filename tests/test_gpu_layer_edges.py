"""The layer operators where other values or another loop come in: non-finite
inputs beside a row's ragged end, many rows to a workgroup, long runs and long
rows, and gradients against differences along their own signs."""
import math

import pytest
import torch

import layer_reference as ref
import test_gpu_layer as base
from test_gpu_layer import DEV, cpu, rand, within

import ssd_chunked_scan_amd as ssd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("D", [34, 33])
@pytest.mark.parametrize("L", [1, 5, 16, 70, 128, 1500])
def test_glr_a_nonfinite_last_input_stays_out_of_the_parameters(L, D, gate, bad):
    """With k = 1 the last token's x enters its own h, y and dz and nothing else:
    every other gradient is the one for a finite x, whatever the row's length."""
    _, s, grad = base.glr_inputs((2, L, D, "f32", gate, False, 9, True, None), seed=11)
    dirty = dict(s, x=s["x"].clone())
    dirty["x"][:, -1] = bad
    want, got = ssd.ssd_glr_bwd(**s, **grad), ssd.ssd_glr_bwd(**dirty, **grad)
    exact = base.glr_reference(s).backward(cpu(grad["dy"]), cpu(grad["dfinal"]))
    for k in ("dA", "dbias", "dinit", "dx", "dg"):
        assert torch.equal(got[k], want[k]), k
        within(k, got[k], exact[k], torch.float32)
    if gate:
        assert torch.equal(got["dz"][:, :-1], want["dz"][:, :-1]) and not torch.isfinite(got["dz"][:, -1]).any()


# ---------------------------------------------------- many rows, long runs
# Shapes that take a kernel's inner loop more than once, with ragged ends, and a
# check that they do: compute units, threads of a workgroup and rows it takes at
# a time (4 where a wave holds a row's group) give the rows in flight.

NORM_ROWS = [
    # rows, columns, ngroups, dtype, kind, weight, threads, rows at a time
    (16387, 40, 1, "bf16", "residual", True, 256, 4),
    (16387, 37, 1, "f32", "gate", True, 256, 4),
    (3001, 320, 8, "f32", "residual", True, 256, 4),
    (3001, 2056, 8, "bf16", "gate", False, 256, 4),      # odd groups of 257
    (3500, 2560, 1, "bf16", "residual", True, 320, 1),
    (3500, 2560, 1, "bf16", "gate", True, 320, 1),
    (3301, 2064, 2, "f32", "plain", True, 192, 1),
    (5003, 1031, 1, "f32", "residual", True, 192, 1),
    (1100, 8195, 1, "bf16", "gate", True, 576, 1),       # 16 single columns a thread
    (700, 16384, 1, "bf16", "residual", True, 1024, 1),
]


def norm_rows(case, seed):
    rows, columns, ngroups, dtype, kind, weight, threads, at_a_time = case
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert rows > max(1, cus * (2048 // threads) // ngroups) * at_a_time, "each row in a workgroup of its own"
    return base.norm_inputs((rows, columns, ngroups, dtype, kind, None, weight), seed)


@pytest.mark.parametrize("case", NORM_ROWS, ids=str)
def test_norm_walks_the_rows(case):
    io, s, gen = norm_rows(case, seed=21)
    ry, v = base.norm_reference(s, io)
    y, stream = ssd.ssd_norm_fwd(**s)
    within("y", y, ry, io)
    if s["residual"] is not None:
        assert torch.equal(stream.double().cpu(), v)
        again = s["residual"].clone()
        y2, same = ssd.ssd_norm_fwd(**dict(s, residual=again), residual_out=again)
        assert same is again and torch.equal(again, stream) and torch.equal(y2, y)
    dy = rand(gen, *s["x"].shape, dtype=io)
    dres = rand(gen, *s["x"].shape, dtype=io) if case[4] == "residual" else None
    got = ssd.ssd_norm_bwd(s["x"], s["weight"], dy, z=s["z"], dresidual=dres, eps=s["eps"], ngroups=s["ngroups"])
    want = ref.norm_backward(cpu(s["x"]), cpu(s["z"]), cpu(s["weight"]), cpu(dy), cpu(dres), s["eps"], s["ngroups"])
    within("dx", got["dx"], want["dx"], io)
    if s["z"] is not None:
        within("dz", got["dz"], want["dz"], io)
    if s["weight"] is not None:
        within("dweight", got["dweight"], want["dweight"], torch.float32)


@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("case", NORM_ROWS, ids=str)
def test_norm_quant_walks_the_rows(case, block):
    """Bounds as for the few-row cases: the scale within y's bound and two
    roundings, the 8-bit value within half a step of e4m3 of the value before it."""
    io, s, _ = norm_rows(case, seed=22)
    q, scales, stream = ssd.ssd_norm_quant_fwd(**s, block=block)
    (y, ey), v = base.norm_reference(s, io)
    rows, per = y.shape[0], y.shape[1] // s["ngroups"]
    width = block or per
    y, ey = y.reshape(rows, s["ngroups"], per), ey.reshape(rows, s["ngroups"], per)
    sc = scales.double().cpu().reshape(rows, s["ngroups"], -(-per // width))
    got = q.float().double().cpu().reshape(y.shape)
    for i in range(sc.shape[-1]):
        part = slice(i * width, min(per, (i + 1) * width))
        m = y[..., part].abs().amax(-1).clamp(min=1e-12)
        assert (sc[..., i] - m / 448).abs().le((ey[..., part].amax(-1) + 2 * ref.U * m) / 448).all()
        t = y[..., part] / sc[..., i, None]
        fuzz = ey[..., part] / sc[..., i, None] + 4 * ref.U * t.abs()
        assert (got[..., part] - t).abs().le(base.e4m3_bound(t.abs() + fuzz) + fuzz).all(), i
    if stream is not None:
        assert torch.equal(stream.double().cpu(), v)


CONV_RUNS = [
    # b, L, D, W, dtype, silu, mean document, init, pad, bias, channels of a strip
    (86, 520, 130, 4, "bf16", True, 60, True, None, True, 128),    # a last run of 8 tokens, a last strip of 2 channels
    (86, 520, 130, 3, "f32", True, 0, True, None, True, 128),
    (60, 530, 129, 4, "bf16", True, 200, True, None, True, 64),    # single channels
    (60, 530, 129, 2, "f32", False, 40, True, None, False, 64),
    (13, 2049, 640, 4, "bf16", True, 300, True, None, True, 128),
]


@pytest.mark.parametrize("case", CONV_RUNS, ids=str)
def test_conv_bwd_runs_of_256_tokens(case):
    b, L, D, strip = *case[:3], case[-1]
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert b * -(-L // 256) * -(-D // strip) >= 2 * cus, "runs of 64 tokens"
    io, s, grad = base.conv_inputs(case[:-1], seed=23)
    got = ssd.ssd_conv_bwd(**s, **grad)
    want = base.conv_reference(s, **grad)
    within("dx", got["dx"], want["dx"], io)
    for k in ("dweight", "dbias", "dinit"):
        if want[k] is not None and got[k] is not None:
            within(k, got[k], want[k], torch.float32)
    assert (got["dbias"] is None) == (s["bias"] is None) and got["dinit"] is not None


@pytest.mark.parametrize("case", [(1, 9000, 34, "f32", True, True, 800, True, None), (1, 9000, 33, "bf16", True, False, 0, True, None),
                                  (1, 20011, 33, "f32", False, True, 3000, True, None), (2, 20011, 34, "f32", True, True, 0, True, None)],
                         ids=str)
def test_glr_long_rows(case):
    """Rows of 141 and 313 blocks: runs of blocks that are loaded eight at a time
    more than once, and forward many splits."""
    io, s, grad = base.glr_inputs(case, seed=24)
    r = base.glr_reference(s)
    y, final = ssd.ssd_glr_fwd(**s)
    within("y", y, r.outputs()[0], io)
    within("final", final, r.outputs()[1], torch.float32)
    got = ssd.ssd_glr_bwd(**s, **grad)
    want = r.backward(cpu(grad["dy"]), cpu(grad["dfinal"]))
    for k in want:
        if want[k] is not None:
            within(k, got[k], want[k], io if k in ("dx", "dg", "dz") else torch.float32)


# ------------------------------------------------ gradients and differences


def along_the_gradient(J, big, grads, inputs):
    """Each gradient against a central difference of J along d = sign(gradient)
    (times |A| for A), where the difference is sum |gradient d|: a gradient of
    independent signs along a random d would leave next to nothing to compare.

    J is a sum of terms, `big` the sum of their magnitudes.  With steps of 2^-7:
    the outputs' rounding, under 30 U of a term each side, 30 U / step = 2.3e-4;
    the inputs', U |input| / step, 128 U; and the truncation, step^2 / 6 times the
    third derivative: moving every element of an input by t changes a term by a
    factor of at most exp(4 t) (a decay product exp(s) by exp(s t), which is below
    exp(-3) where |s| > 3; silu's third derivative is below 1), so 64 step^2 / 6 =
    6.5e-4.  Together below 2^-10 of `big`."""
    step = 2.0 ** -7
    for name, grad in grads.items():
        d = torch.sign(grad.float()) * (inputs[name].abs() if name == "A" else 1.0)
        up, down = (J({**inputs, name: inputs[name] + s * d}) for s in (step, -step))
        want = float((up - down) / (2 * step))
        got = float((grad.double() * d.double()).sum())
        assert got > 2.0 ** -7 * big, (name, "too small to tell", got, big)
        assert abs(got - want) <= 2.0 ** -10 * big, (name, got, want, big)


def test_glr_gradients_along_their_signs():
    _, s, grad = base.glr_inputs((2, 150, 36, "f32", True, True, 40, True, None), seed=6)
    inputs = {k: s[k] for k in ("x", "g", "z", "A", "bias", "init_states")}

    def J(q, dy=grad["dy"], df=grad["dfinal"]):
        y, f = ssd.ssd_glr_fwd(**{**s, **q})
        return (y.double() * dy.double()).sum() + (f.double() * df.double()).sum()

    def magnitude():
        q = {**s, "x": s["x"].abs(), "init_states": s["init_states"].abs()}
        y, f = ssd.ssd_glr_fwd(**q)
        return float((y.double() * grad["dy"].double()).abs().sum() + (f.double() * grad["dfinal"].double()).abs().sum())

    g = ssd.ssd_glr_bwd(**s, **grad)
    along_the_gradient(J, magnitude(), {"x": g["dx"], "g": g["dg"], "z": g["dz"], "A": g["dA"], "bias": g["dbias"],
                                        "init_states": g["dinit"]}, inputs)


def test_conv_gradients_along_their_signs():
    _, s, grad = base.conv_inputs((2, 70, 36, 4, "f32", True, 15, True, None, True), seed=6)
    inputs = {k: s[k] for k in ("x", "weight", "bias", "init_states")}

    def J(q):
        y, f = ssd.ssd_conv_fwd(**{**s, **q})
        return (y.double() * grad["dy"].double()).sum() + (f.double() * grad["dfinal"].double()).sum()

    p, f = ssd.ssd_conv_fwd(s["x"].abs(), s["weight"].abs(), bias=s["bias"].abs(), seq_idx=s["seq_idx"],
                            init_states=s["init_states"].abs(), silu=False)
    big = float((p.double() * grad["dy"].double()).abs().sum() + (f.double() * grad["dfinal"].double()).abs().sum())
    g = ssd.ssd_conv_bwd(**s, **grad)
    along_the_gradient(J, big, {"x": g["dx"], "weight": g["dweight"], "bias": g["dbias"], "init_states": g["dinit"]}, inputs)


def test_norm_gradients_along_their_signs():
    _, s, gen = base.norm_inputs((60, 72, 3, "f32", "gate", None, True), seed=6)
    dy = rand(gen, 60, 72)
    inputs = {k: s[k] for k in ("x", "z", "weight")}
    g = ssd.ssd_norm_bwd(s["x"], s["weight"], dy, z=s["z"], eps=s["eps"], ngroups=3)
    J = lambda q: (ssd.ssd_norm_fwd(**{**s, **q})[0].double() * dy.double()).sum()
    big = float((ssd.ssd_norm_fwd(**s)[0].double() * dy.double()).abs().sum())
    along_the_gradient(J, big, {"x": g["dx"], "z": g["dz"], "weight": g["dweight"]}, inputs)


# ------------------------------------------------------- the documented limits


def test_the_longest_token_stride():
    """Tokens 2^22 fp32 elements apart: a round of 128 reaches 2^31 bytes."""
    L, W, D = 130, 1 << 22, 34
    gen = torch.Generator().manual_seed(31)
    wide = torch.zeros(1, L, W, device=DEV)
    x, g, w = rand(gen, 1, L, D), rand(gen, 1, L, D), rand(gen, D, 4)
    far = wide[..., W - D:]
    far.copy_(x)
    A = -1 - rand(gen, D).abs()
    for a, b in ((ssd.ssd_glr_fwd(far, g, A), ssd.ssd_glr_fwd(x, g, A)), (ssd.ssd_glr_fwd(g, far, A), ssd.ssd_glr_fwd(g, x, A)),
                 (ssd.ssd_conv_fwd(far, w), ssd.ssd_conv_fwd(x, w)), (ssd.ssd_norm_fwd(far)[:1], ssd.ssd_norm_fwd(x)[:1])):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    for a, b in ((ssd.ssd_glr_bwd(far, g, A, None, far), ssd.ssd_glr_bwd(x, g, A, None, x)),
                 (ssd.ssd_conv_bwd(far, w, None, far), ssd.ssd_conv_bwd(x, w, None, x)),
                 (ssd.ssd_norm_bwd(far, None, far), ssd.ssd_norm_bwd(x, None, x))):
        assert all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)


def test_the_most_channels():
    """2^20 channels: the last 66 as they are alone."""
    L, D, n = 70, 1 << 20, 66
    gen = torch.Generator(device=DEV).manual_seed(32)
    r = lambda *s: torch.randn(*s, generator=gen, device=DEV)
    x, g, dy, A, w = r(1, L, D), r(1, L, D), r(1, L, D), -1 - r(D).abs(), r(D, 4)
    last = lambda t: t[..., D - n:].contiguous()
    for a, b in zip(ssd.ssd_glr_fwd(x, g, A), ssd.ssd_glr_fwd(last(x), last(g), last(A))):
        assert torch.equal(last(a), b)
    a, b = ssd.ssd_glr_bwd(x, g, A, None, dy), ssd.ssd_glr_bwd(last(x), last(g), last(A), None, last(dy))
    assert all(torch.equal(last(a[k]), b[k]) for k in ("dx", "dg", "dA"))
    wl = w[D - n:].contiguous()
    assert torch.equal(last(ssd.ssd_conv_fwd(x, w)[0]), ssd.ssd_conv_fwd(last(x), wl)[0])
    a = ssd.ssd_conv_bwd(x, w, None, dy)
    assert torch.equal(last(a["dx"]), ssd.ssd_conv_bwd(last(x), wl, None, last(dy))["dx"])
    within("dweight", a["dweight"][D - n:], ref.conv(cpu(last(x)), cpu(wl), None, None, None, True, cpu(last(dy)))["dweight"],
           torch.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_most_norm_groups(dtype):
    """65535 groups of 2 columns: a launch dimension's limit."""
    io, s, gen = base.norm_inputs((9, 131070, 65535, dtype, "gate", None, True), seed=33)
    ry, _ = base.norm_reference(s, io)
    within("y", ssd.ssd_norm_fwd(**s)[0], ry, io)
    dy = rand(gen, 9, 131070, dtype=io)
    got = ssd.ssd_norm_bwd(s["x"], s["weight"], dy, z=s["z"], eps=s["eps"], ngroups=65535)
    want = ref.norm_backward(cpu(s["x"]), cpu(s["z"]), cpu(s["weight"]), cpu(dy), None, s["eps"], 65535)
    for k, t in (("dx", io), ("dz", io), ("dweight", torch.float32)):
        within(k, got[k], want[k], t)
    q, scales, _ = ssd.ssd_norm_quant_fwd(**s, block=0)
    assert scales.shape == (9, 65535) and float(q.float().abs().max()) == 448.0


def test_two_threads_at_once():
    """Each on a stream of its own: results and errors are the thread's."""
    import threading
    calls = base.every_call()
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    failed = []

    def work(shift):
        stream = torch.cuda.Stream()
        names = base.NAMES[shift:] + base.NAMES[:shift]
        with torch.cuda.stream(stream):
            for _ in range(10):
                for name in names:
                    got = calls[name]()
                    stream.synchronize()
                    if not base.same(got, want[name]):
                        failed.append(name)
                try:
                    ssd.ssd_norm_fwd(torch.zeros(1, 8, device=DEV), ngroups=3 + shift)
                except ssd.SsdError as e:
                    if f"ngroups ({3 + shift})" not in str(e):
                        failed.append(str(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
