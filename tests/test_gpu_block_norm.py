"""The block norm on the GPU against its fp64 definition, forward, backward and
from 8-bit checkpoints: every element within a bound that counts the roundings
of the evaluation."""
import math

import pytest
import torch

import block_reference as ref
from layer_reference import HALF, U, rounded

import ssd_chunked_scan_amd as ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def within(name, got, pair, io=None):
    want, err = pair if io is None else rounded(pair, io)
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= err)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / err).max()):.2f} times the "
                           f"bound, first at {torch.nonzero(bad)[0].tolist()}: {got[bad][0]} for {want[bad][0]}")


def cpu(t):
    return None if t is None else t.detach().double().cpu()


def sliced(t, pad):
    if pad is None:
        return t.to(DEV)
    wide = torch.full((t.shape[0], t.shape[1] + 2 * pad), math.nan, dtype=t.dtype, device=DEV)
    wide[:, pad:pad + t.shape[1]] = t.to(DEV)
    return wide[:, pad:pad + t.shape[1]]


def inputs(case):
    rows, columns, dtype, gate, weights, alpha, pad = case
    gen = torch.Generator().manual_seed(rows * 31 + columns)
    r = lambda *s: torch.randn(*s, generator=gen)
    io = TYPES[dtype]
    p = dict(x=3 * r(rows, columns), residual=4 * r(rows, columns), z=2 * r(rows, columns) if gate else None,
             dy=r(rows, columns), dstream=r(rows, columns))
    p = {k: None if v is None else sliced(v.to(io), pad) for k, v in p.items()}
    has = lambda i: weights >> i & 1
    p["post"] = (1 + 0.3 * r(columns)).to(DEV) if has(0) else None
    p["pre"] = (1 + 0.3 * r(columns)).to(DEV) if has(1) else None
    p["scale"] = (0.3 * r(columns)).to(DEV) if has(2) else None
    return p, io


# rows, columns, dtype, gate, which of post | pre | scale, alpha, pad (None: dense)
CASES = [
    (1, 1, "f32", False, 7, 1.0, None), (1, 1, "bf16", True, 7, 0.5, None), (3, 2, "bf16", True, 0, 1.0, None),
    (5, 7, "f32", True, 3, 1.0, None), (2, 8, "bf16", False, 5, -1.5, None), (9, 31, "bf16", True, 7, 1.0, 1),
    (64, 64, "bf16", True, 7, 1.0, 8), (70, 128, "f32", False, 7, 0.8125, 4), (11, 129, "bf16", True, 6, 1.0, None),
    (33, 256, "f32", True, 7, 1.0, None), (33, 257, "f32", True, 7, 1.0, 3), (40, 512, "bf16", True, 7, 1.0, None),
    (40, 512, "f32", True, 4, 1.0, None), (6, 513, "bf16", True, 7, 1.0, None), (6, 520, "bf16", True, 7, 1.0, None),
    (6, 516, "f32", False, 1, 1.0, None), (21, 1000, "bf16", True, 7, 0.0, 8), (300, 1477, "f32", False, 3, 0.8125, None),
    (130, 2560, "bf16", True, 7, 1.0, None), (130, 2560, "bf16", False, 2, 1.0, 16), (50, 2560, "f32", True, 7, 1.0, None),
    (7, 4097, "f32", True, 7, 1.0, None), (7, 4100, "bf16", True, 7, 1.0, None), (3, 8192, "bf16", True, 7, 1.0, None),
    (3, 8200, "bf16", True, 7, 1.0, None), (3, 8195, "f32", True, 7, 1.0, None), (2, 16384, "bf16", True, 7, 1.0, None),
    (2, 16384, "f32", True, 7, 1.0, None), (2, 16383, "bf16", True, 7, 1.0, None), (2, 16381, "f32", False, 7, 1.0, 3),
    (9000, 96, "bf16", True, 7, 1.0, None), (2900, 640, "bf16", True, 7, 1.0, None), (2200, 1003, "f32", True, 7, 1.0, None),
    # rows of whole 4-byte words that are not whole 16-byte pieces
    (7, 2, "bf16", True, 7, 1.0, None), (40, 510, "bf16", True, 7, 1.0, 2), (33, 1002, "bf16", True, 7, 1.0, None),
    (9, 4098, "bf16", True, 7, 1.0, 2), (5, 6003, "f32", True, 7, 1.0, 3), (5, 12290, "bf16", True, 7, 1.0, None),
    (5, 12292, "bf16", False, 5, 0.5, 4), (5, 12289, "f32", True, 7, 1.0, 1), (900, 4101, "f32", True, 7, 1.0, None),
]


def forward(p, alpha, checkpoint, **kw):
    return ssd.ssd_block_norm_fwd(p["x"], p["residual"], p["post"], p["pre"], z=p["z"], scale=p["scale"], alpha=alpha, eps=EPS,
                                  checkpoint=checkpoint, **kw)


def check_gradients(got, want, io):
    for name, pair in want.items():
        if pair is None:
            assert got[name] is None, name
        else:
            within(name, got[name], pair, io if name in ("dx", "dresidual", "dz") else torch.float32)


def check_kept(kept, name, v):
    """Each value within half a step of e4m3 of the block's scale: 2^-4 relative or
    half the smallest subnormal, 2^-10 scale; five roundings of 2^-24 besides."""
    v = cpu(v)
    scales = ref.kept_scales(v)
    within(name + "_scales", kept[name + "_scales"], (scales, 2 * U * scales))
    q = kept[name + "_q"].float().double().cpu() * ref.per_column(cpu(kept[name + "_scales"]), v.shape[1])
    step = torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -10 * ref.per_column(scales, v.shape[1]))
    assert ((q - v).abs() <= step * (1 + 2.0 ** -20) + 8 * U * v.abs()).all(), name


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward(case):
    p, io = inputs(case)
    alpha = case[5]
    y, stream, kept = forward(p, alpha, False)
    assert kept is None
    c = {k: cpu(v) for k, v in p.items()}
    within("stream", stream, ref.block_stream(c["x"], c["residual"], c["z"], c["post"], c["scale"], alpha, EPS), io)
    within("y", y, ref.block_out(cpu(stream), c["pre"], EPS), io)
    g = ssd.ssd_block_norm_bwd(p["x"], stream, p["post"], p["pre"], p["dy"], z=p["z"], scale=p["scale"],
                               dresidual_out=p["dstream"], alpha=alpha, eps=EPS)
    check_gradients(g, ref.block_backward(c["x"], cpu(stream), c["z"], c["post"], c["pre"], c["scale"], c["dy"], c["dstream"],
                                          alpha, EPS), io)
    g = ssd.ssd_block_norm_bwd(p["x"], stream, p["post"], p["pre"], p["dy"], z=p["z"], scale=p["scale"], alpha=alpha, eps=EPS)
    check_gradients(g, ref.block_backward(c["x"], cpu(stream), c["z"], c["post"], c["pre"], c["scale"], c["dy"], None,
                                          alpha, EPS), io)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_checkpoints(case):
    """They change nothing forward, hold x, z and the stream to half a step, and
    the backward pass from them is that at the values they hold."""
    p, io = inputs(case)
    alpha = case[5]
    y, stream, kept = forward(p, alpha, True)
    y0, stream0, _ = forward(p, alpha, False)
    assert torch.equal(y, y0) and torch.equal(stream, stream0)
    names = ["x", "residual"] + (["z"] if p["z"] is not None else [])
    assert sorted(kept) == sorted(n + s for n in names for s in ("_q", "_scales"))
    for name in names:
        check_kept(kept, name, stream if name == "residual" else p[name])
    held = {n: cpu(kept[n + "_q"].float()) * ref.per_column(cpu(kept[n + "_scales"]), y.shape[1]) for n in names}
    g = ssd.ssd_block_norm_bwd(None, None, p["post"], p["pre"], p["dy"], scale=p["scale"], dresidual_out=p["dstream"],
                               alpha=alpha, eps=EPS, checkpoint=kept)
    c = {k: cpu(v) for k, v in p.items()}
    # the product of code and scale rounds once in fp32, which moves every
    # quantity that the bound counts by a few of its roundings; twice the bound
    want = ref.block_backward(held["x"], held["residual"], held.get("z"), c["post"], c["pre"], c["scale"], c["dy"],
                              c["dstream"], alpha, EPS)
    check_gradients(g, {k: None if v is None else (v[0], 2 * v[1]) for k, v in want.items()}, io)


def test_checkpoint_blocks_with_infinities_and_nan():
    """An infinity or a NaN turns its 128 columns of the checkpoint into NaN and
    leaves the others; zeros stay zeros."""
    x = torch.ones(3, 300)
    x[0, 5], x[1, 200], x[2] = math.inf, math.nan, 0
    for io in TYPES.values():
        t = x.to(io).to(DEV)
        _, _, kept = ssd.ssd_block_norm_fwd(t, torch.zeros_like(t), checkpoint=True)
        held = kept["x_q"].float().cpu() * ref.per_column(kept["x_scales"].cpu(), 300)
        nan = torch.zeros(3, 300, dtype=torch.bool)
        nan[0, :128], nan[1, 128:256] = True, True
        assert torch.equal(held.isnan(), nan)
        assert (held[2] == 0).all() and ((held[:2] - 1).abs() <= 2.0 ** -4)[~nan[:2]].all()


def test_nonfinite_rows_leave_the_others():
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(*s, generator=gen).to(DEV)
    for columns in (100, 640):
        x, res, z, dy = (r(6, columns) for _ in range(4))
        y, s, _ = ssd.ssd_block_norm_fwd(x, res, z=z)
        g = ssd.ssd_block_norm_bwd(x, s, None, None, dy, z=z)
        x2 = x.clone()
        x2[2, 7] = math.nan
        y2, s2, _ = ssd.ssd_block_norm_fwd(x2, res, z=z)
        g2 = ssd.ssd_block_norm_bwd(x2, s2, None, None, dy, z=z)
        rest = [0, 1, 3, 4, 5]
        assert y2[2].isnan().all() and torch.equal(y[rest], y2[rest]) and torch.equal(s[rest], s2[rest])
        assert all(torch.equal(g[k][rest], g2[k][rest]) for k in ("dx", "dz", "dresidual"))


def test_gradients_along_their_signs():
    """A step along each gradient's signs changes the fp64 definition's value by
    the sum of its sizes."""
    case = (6, 96, "f32", True, 7, 0.75, None)
    p, _ = inputs(case)
    _, stream, _ = forward(p, 0.75, False)
    g = ssd.ssd_block_norm_bwd(p["x"], stream, p["post"], p["pre"], p["dy"], z=p["z"], scale=p["scale"],
                               dresidual_out=p["dstream"], alpha=0.75, eps=EPS)
    c = {k: cpu(v) for k, v in p.items()}

    def J(**moved):
        q = dict(c, **moved)
        s, _ = ref.block_stream(q["x"], q["residual"], q["z"], q["post"], q["scale"], 0.75, EPS)
        return float((ref.block_out(s, q["pre"], EPS)[0] * c["dy"]).sum() + (s * c["dstream"]).sum())

    for name, grad in (("x", "dx"), ("residual", "dresidual"), ("z", "dz"), ("post", "dpost_weight"), ("pre", "dpre_weight"),
                       ("scale", "dscale")):
        d = cpu(g[grad])
        h = 1e-6
        diff = (J(**{name: c[name] + h * d.sign()}) - J(**{name: c[name] - h * d.sign()})) / (2 * h)
        # fp32 gradients: 1e-5 of the sum covers the 400 roundings the bounds count
        assert abs(diff - float(d.abs().sum())) <= 1e-5 * float(d.abs().sum()), name


@pytest.mark.parametrize("columns,dtype", [(96, "bf16"), (2560, "bf16"), (333, "f32")])
def test_given_outputs_and_repeats(columns, dtype):
    """Outputs and workspace of the caller's, poisoned; the residual updated in
    place; the same bits on every call."""
    p, io = inputs((700, columns, dtype, True, 7, 1.0, None))
    y, stream, kept = forward(p, 1.0, True)
    args = (p["post"], p["pre"], p["dy"])
    kw = dict(scale=p["scale"], dresidual_out=p["dstream"], eps=EPS)
    g = ssd.ssd_block_norm_bwd(p["x"], stream, *args, z=p["z"], **kw)
    gk = ssd.ssd_block_norm_bwd(None, None, *args, checkpoint=kept, **kw)
    for fill in (0x00, 0xff):
        out = {k: torch.empty_like(v).view(torch.uint8).fill_(fill).view(v.dtype) for k, v in g.items()}
        ws = torch.full((1 << 26,), fill, dtype=torch.uint8, device=DEV)
        again = ssd.ssd_block_norm_bwd(p["x"], stream, *args, z=p["z"], workspace=ws, out=out, **kw)
        assert all(again[k] is not None and torch.equal(again[k], g[k]) for k in g)
        again = ssd.ssd_block_norm_bwd(None, None, *args, checkpoint=kept, workspace=ws, out=out, **kw)
        assert all(torch.equal(again[k], gk[k]) for k in gk)
        into = {k: v.clone().view(torch.uint8).fill_(fill).view(v.dtype) for k, v in kept.items()}
        res = p["residual"].clone()
        y2, s2, k2 = ssd.ssd_block_norm_fwd(p["x"], res, p["post"], p["pre"], z=p["z"], scale=p["scale"], eps=EPS,
                                            checkpoint=into, residual_out=res)
        assert s2 is res and torch.equal(s2, stream) and torch.equal(y2, y)
        assert all(torch.equal(k2[k].view(torch.uint8), kept[k].view(torch.uint8)) for k in kept)


def test_binding_refusals():
    x = torch.zeros(4, 200, device=DEV)
    w = torch.ones(200, device=DEV)
    _, s, kept = ssd.ssd_block_norm_fwd(x, x, checkpoint=True)
    small = {k: v[:3] for k, v in kept.items()}
    half = {k: v for k, v in kept.items() if k != "x_scales"}
    for f, what in ((lambda: ssd.ssd_block_norm_fwd(x, x[:3]), "residual"), (lambda: ssd.ssd_block_norm_fwd(x, x, w[:100]), "post_weight"),
                    (lambda: ssd.ssd_block_norm_fwd(x, x, z=x.t()), "z"), (lambda: ssd.ssd_block_norm_fwd(x, x, checkpoint=half), "x_scales"),
                    (lambda: ssd.ssd_block_norm_bwd(None, None, None, None, x, checkpoint=small), "x_q"),
                    (lambda: ssd.ssd_block_norm_bwd(x, None, None, None, x, checkpoint=kept), "stands for"),
                    (lambda: ssd.ssd_block_norm_bwd(x, None, None, None, x), "needed"),
                    (lambda: ssd.ssd_block_norm_bwd(x, s, w, None, x, out={}), "missing"),
                    (lambda: ssd.ssd_block_norm_bwd(x, s, w, None, x, workspace=torch.zeros(8, dtype=torch.uint8, device=DEV)), "workspace")):
        with pytest.raises(ValueError, match=what):
            f()
    for f in (lambda: ssd.ssd_block_norm_fwd(x.half(), x.half()), lambda: ssd.ssd_block_norm_fwd(x, x.bfloat16()),
              lambda: ssd.ssd_block_norm_fwd(x, x, w.bfloat16())):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: ssd.ssd_block_norm_fwd(x, x, eps=0.0), lambda: ssd.ssd_block_norm_fwd(x, x, alpha=math.inf),
              lambda: ssd.ssd_block_norm_fwd(x[:0], x[:0])):
        with pytest.raises(ssd.SsdError):
            f()
