"""Microscaled 4-bit values and products on the GPU: codes, scales and values
bit for bit, products within the roundings of their sums and exactly where
every partial sum is a number of fp32."""
import math

import pytest
import torch

import block_reference as ref
from layer_reference import rounded

import ssd_chunked_scan_amd as ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def within(name, got, pair, io):
    want, err = rounded(pair, io)
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= err)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / err).max()):.2f} times the "
                           f"bound, first at {torch.nonzero(bad)[0].tolist()}")


def spread(gen, rows, columns, dtype):
    """Blocks of very different sizes, a few zeros."""
    v = torch.randn(rows, columns, generator=gen) * torch.exp2(20 * torch.randn(rows, 1, generator=gen))
    v[torch.rand(rows, columns, generator=gen) < 0.05] = 0
    return v.to(dtype)


def sliced(t, pad):
    """t as a column slice of wider rows, NaN around it, on the GPU."""
    wide = torch.full((t.shape[0], t.shape[1] + 2 * pad), math.nan, dtype=t.dtype, device=DEV)
    wide[:, pad:pad + t.shape[1]] = t.to(DEV)
    return wide[:, pad:pad + t.shape[1]]


QUANT_CASES = [(1, 1), (1, 31), (3, 32), (2, 33), (17, 127), (16, 128), (5, 129), (33, 640), (7, 1477), (300, 2560), (2, 8192),
               (1000, 40), (1, 100001)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,columns", QUANT_CASES)
@pytest.mark.parametrize("pad", [None, 8, 3])
def test_quant_and_back(rows, columns, dtype, pad):
    gen = torch.Generator().manual_seed(rows * 7 + columns)
    x = spread(gen, rows, columns, TYPES[dtype])
    code, byte = ref.mx4(x.double())
    q, scales = ref.pack(code, byte)
    given = x.to(DEV) if pad is None else sliced(x, pad)
    got_q, got_s = ssd.ssd_mx4_quant(given)
    assert torch.equal(got_s.cpu(), scales)
    assert torch.equal(got_q.cpu(), q)
    want = ref.unpack(q, scales)[:, :columns]
    for io in TYPES.values():
        got = ssd.ssd_mx4_dequant(got_q, got_s, columns, dtype=io)
        assert torch.equal(got.double().cpu(), want)


def test_quant_at_the_edges_of_the_types():
    """Zeros of both signs, subnormals, ties, the largest numbers, and blocks with
    infinities and NaN, which stand for NaN and leave their neighbours alone."""
    big = torch.finfo(torch.float32).max
    rows = torch.zeros(12, 128)
    rows[0, :40] = -0.0
    rows[1, :4] = torch.tensor([2.0 ** -149, -2.0 ** -140, 2.0 ** -127, 2.0 ** -126])
    rows[2, :3] = torch.tensor([2.0 ** -127, 2.0 ** -129, 3 * 2.0 ** -130])
    rows[3, :3] = torch.tensor([big, -big, big / 16])
    rows[4, :8] = torch.tensor([4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -2.5]) * 2.0 ** -100
    rows[5, :4] = torch.tensor([7.999, 5.0, 5.0001, -6.5]) * 2.0 ** 90
    rows[6, 5] = math.inf
    rows[7, 33] = math.nan
    rows[8, 70] = -math.inf
    rows[9] = math.nan
    rows[10, :] = torch.linspace(-8, 8, 128)
    rows[11, 100:] = 2.0 ** -126
    rows[6:9, ::3] += 1
    for io in TYPES.values():
        x = rows.to(io)
        code, byte = ref.mx4(x.double())
        q, scales = ref.pack(code, byte)
        got_q, got_s = ssd.ssd_mx4_quant(x.to(DEV))
        assert torch.equal(got_s.cpu(), scales) and torch.equal(got_q.cpu(), q)
        for out in TYPES.values():
            got = ssd.ssd_mx4_dequant(got_q, got_s, 128, dtype=out).double().cpu()
            assert torch.equal(got.isnan(), ref.unpack(q, scales).isnan())
            assert torch.equal(got.nan_to_num(), ref.unpack(q, scales).nan_to_num())


def test_every_bf16_is_rounded_to_the_nearest():
    """All positive finite bf16 numbers, each in a block whose maximum is 4, 7.5
    or itself times something: the conversion's roundings and its scale."""
    bits = torch.arange(0, 0x7f80, dtype=torch.int32)
    v = (bits << 16).view(torch.float32)
    v = torch.cat([v, v.new_zeros(-v.numel() % 31)]).reshape(-1, 31)
    for factor in (1.0, 1.5, 4.0):
        x = torch.zeros(v.shape[0], 32)
        x[:, :31] = v
        x[:, 31] = (v.amax(1) * factor).clamp(max=3e38)
        x = x.to(torch.bfloat16)
        q, scales = ref.pack(*ref.mx4(x.double()))
        got_q, got_s = ssd.ssd_mx4_quant(x.to(DEV))
        assert torch.equal(got_s.cpu(), scales) and torch.equal(got_q.cpu(), q)


def operands(gen, m, n, k, exact):
    """Random codes; scales near one, or exactly 1/2, 1 or 2, where all partial
    sums are multiples of 1/16 below 2^19 for k < 3600."""
    def make(rows):
        kb = -(-k // 128)
        code = torch.randint(0, 16, (rows, kb * 128), generator=gen)
        code[:, k:] = 0
        byte = torch.randint(126, 129, (rows, 4 * kb), generator=gen) if exact else torch.randint(100, 140, (rows, 4 * kb), generator=gen)
        return ref.pack(code, byte)
    return make(m), make(n)


# m, n, k: the few-token kernels' and the tiles' sizes and borders
PRODUCTS = [(1, 1, 1), (1, 16, 128), (1, 17, 300), (2, 33, 129), (15, 100, 2560), (16, 130, 640), (17, 64, 256), (31, 47, 1000),
            (32, 64, 128), (33, 200, 500), (64, 129, 384), (65, 64, 128), (65, 1, 77), (100, 333, 1477), (128, 128, 1024),
            (129, 257, 200), (700, 1000, 256), (2000, 1030, 640), (1501, 1001, 1477), (2500, 2600, 300), (4100, 4200, 129),
            (1, 9000, 256), (20, 9001, 256), (5000, 20, 64), (4100, 4200, 700), (3333, 3001, 385), (3400, 2900, 1024),
            (200, 70, 2900), (66, 5000, 257), (1300, 2111, 900), (9000, 1000, 300), (770, 8500, 513)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_matmul_exact_sums(m, n, k):
    gen = torch.Generator().manual_seed(m + n + k)
    (q, s), (wq, ws) = operands(gen, m, n, k, True)
    got = ssd.ssd_mx4_matmul(*(t.to(DEV) for t in (q, s, wq, ws)), dtype=torch.float32)
    want = (ref.unpack(q, s).float().to(DEV) @ ref.unpack(wq, ws).float().to(DEV).t())
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("m,n,k", [c for c in PRODUCTS if c[0] * c[1] * c[2] < 3_000_000_000])
def test_matmul_and_linear(m, n, k, bias, dtype):
    gen = torch.Generator().manual_seed(m * 3 + n + k)
    io = TYPES[dtype]
    (q, s), (wq, ws) = operands(gen, m, n, k, False)
    b = torch.randn(n, generator=gen) * 100 if bias else None
    bd = None if b is None else b.to(DEV)
    wq, ws = wq.to(DEV), ws.to(DEV)
    want = ref.product(ref.unpack(q, s), ref.unpack(wq.cpu(), ws.cpu()), None if b is None else b.double())
    within("matmul", ssd.ssd_mx4_matmul(q.to(DEV), s.to(DEV), wq, ws, bias=bd, dtype=io), want, io)
    x = torch.randn(m, k, generator=gen).to(io)
    a = ref.unpack(*ref.pack(*ref.mx4(x.double())))
    want = ref.product(a, ref.unpack(wq.cpu(), ws.cpu()), None if b is None else b.double())
    within("linear", ssd.ssd_mx4_linear(x.to(DEV), wq, ws, bias=bd), want, io)
    within("linear of a slice", ssd.ssd_mx4_linear(sliced(x, 5), wq, ws, bias=bd), want, io)


@pytest.mark.parametrize("m", [1, 16, 17, 64, 65, 300, 3000])
def test_the_two_ways_to_a_product_agree(m):
    """Quantised on the way or before: the same operands, and up to 16 or over 64
    tokens the same kernels' sums."""
    gen = torch.Generator().manual_seed(m)
    x = torch.randn(m, 700, generator=gen).to(torch.bfloat16).to(DEV)
    w = ssd.ssd_mx4_quant(torch.randn(300, 700, generator=gen).to(DEV))
    assert torch.equal(ssd.ssd_mx4_linear(x, *w), ssd.ssd_mx4_matmul(*ssd.ssd_mx4_quant(x), *w))


@pytest.mark.parametrize("m", [1, 16, 40, 64, 100, 600])
def test_nan_blocks_reach_their_row_only(m):
    gen = torch.Generator().manual_seed(m)
    x = torch.randn(m, 300, generator=gen)
    w = torch.randn(50, 300, generator=gen)
    clean = ssd.ssd_mx4_linear(x.to(DEV), *ssd.ssd_mx4_quant(w.to(DEV)))
    x[m // 2, 299] = math.inf
    w[17, 5] = math.nan
    for got in (ssd.ssd_mx4_linear(x.to(DEV), *ssd.ssd_mx4_quant(w.to(DEV))),
                ssd.ssd_mx4_matmul(*ssd.ssd_mx4_quant(x.to(DEV)), *ssd.ssd_mx4_quant(w.to(DEV)), dtype=torch.float32)):
        nan = torch.zeros(m, 50, dtype=torch.bool, device=DEV)
        nan[m // 2] = True
        nan[:, 17] = True
        assert torch.equal(got.isnan(), nan)
        assert torch.equal(got[~nan], clean[~nan])


def test_shapes_and_given_outputs():
    """Leading dimensions, one-dimensional rows, outputs and workspaces of the
    caller's, filled with NaN before; what lies behind them stays."""
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(2, 30, 200, generator=gen).to(torch.bfloat16).to(DEV)
    w = torch.randn(70, 200, generator=gen).to(torch.bfloat16).to(DEV)
    wq, ws = ssd.ssd_mx4_quant(w)
    assert wq.shape == (70, 128) and ws.shape == (2, 70, 4)
    q, s = ssd.ssd_mx4_quant(x)
    assert q.shape == (2, 30, 128) and s.shape == (2, 60, 4)
    y = ssd.ssd_mx4_linear(x, wq, ws)
    assert y.shape == (2, 30, 70)
    assert torch.equal(y, ssd.ssd_mx4_matmul(q, s, wq, ws))
    one = ssd.ssd_mx4_linear(x[0, 0], wq, ws)
    assert one.shape == (70,)
    room = torch.full((61 * 70,), 5.0, dtype=torch.bfloat16, device=DEV)
    out = room[:60 * 70].view(2, 30, 70)
    out.fill_(math.nan)
    ws_room = torch.full((1 << 16,), 255, dtype=torch.uint8, device=DEV)
    assert ssd.ssd_mx4_linear(x, wq, ws, y=out, workspace=ws_room) is out
    assert torch.equal(out, y) and (room[60 * 70:] == 5).all()
    q2, s2 = torch.full_like(q, 255), torch.full_like(s, 255)
    ssd.ssd_mx4_quant(x, q=q2, scales=s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    # an output that is not 16-byte aligned, and rows that no vector divides
    flat = torch.full((60 * 70 + 8,), math.nan, dtype=torch.bfloat16, device=DEV)
    off = flat[1:1 + 60 * 70].view(2, 30, 70)
    ssd.ssd_mx4_matmul(q, s, wq, ws, y=off)
    assert torch.equal(off, y) and flat[0].isnan() and flat[1 + 60 * 70:].isnan().all()


def test_binding_refusals():
    x = torch.zeros(4, 200, device=DEV)
    q, s = ssd.ssd_mx4_quant(x)
    for f, what in ((lambda: ssd.ssd_mx4_linear(x[:, :100], q, s), "columns"), (lambda: ssd.ssd_mx4_matmul(q, s, q[:, :64], s), "contiguous|columns|scales"),
                    (lambda: ssd.ssd_mx4_matmul(q, s[:1], q, s), "scales"), (lambda: ssd.ssd_mx4_dequant(q, s, 128), "columns"),
                    (lambda: ssd.ssd_mx4_dequant(q, s, 257), "columns"), (lambda: ssd.ssd_mx4_matmul(q[:, :60], s, q, s), "multiple of 128"),
                    (lambda: ssd.ssd_mx4_linear(x, q, s, bias=torch.zeros(5, device=DEV)), "bias"),
                    (lambda: ssd.ssd_mx4_linear(x, q[None], s), "wq"), (lambda: ssd.ssd_mx4_linear(x, q, s, y=torch.zeros(4, 5, device=DEV)), "y"),
                    (lambda: ssd.ssd_mx4_linear(x.t(), q, s), "contiguous|columns"), (lambda: ssd.ssd_mx4_quant(x, q=q[:3]), "q")):
        with pytest.raises(ValueError, match=what):
            f()
    for f in (lambda: ssd.ssd_mx4_quant(x.half()), lambda: ssd.ssd_mx4_dequant(q, s, 200, dtype=torch.float16),
              lambda: ssd.ssd_mx4_matmul(q, s, q.float(), s)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(ssd.SsdError, match="SHAPE"):
        ssd.ssd_mx4_quant(x[:0])
