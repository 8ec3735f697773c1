"""Products of 4-bit operands by the kernels of the largest and of the smallest
problems: 256 x 256 tiles in each of their forms and the few-token kernel with
one, two and four tiles of outputs, with scales that differ from block to block
and row to row, compared on the whole result.

Exactly: scales 1/2, 1 or 2 make every product a multiple of 1/16 of at most
144, so that sums over up to 7000 columns stay below 2^24 sixteenths, and the
bias is a few sixteenths more: any order of fp32 sums is exact.  And within the
roundings of a sum, with scales from 2^-27 to 2^12."""
import math

import pytest
import torch

import block_reference as ref
from layer_reference import rounded
from test_gpu_mx4 import operands

import ssd_chunked_scan_amd as ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32

# m, n, k, dtype: at least 5/8 of 256 compute units have a tile of 256 x 256;
# odd and even numbers of 128-column blocks, one to three tiles a workgroup, rows
# of results that are whole 16-byte pieces and ones that are not
TILES = [
    (4100, 4200, 700, BF16), (4100, 4200, 600, BF16), (4100, 8304, 300, BF16), (4360, 5000, 500, BF16),
    (3400, 3333, 2200, BF16), (3400, 3333, 2100, BF16), (4700, 4111, 2200, BF16),
    (3400, 3328, 4300, F32), (3400, 3328, 4200, F32), (4700, 4112, 4200, F32),
    (3400, 3333, 4300, F32), (3400, 3333, 4200, F32), (4700, 4111, 4300, F32),
]
# from operands in 4 bits, one and two tiles of 16 tokens
FEW = [(m, n, k, dtype) for dtype in (BF16, F32) for m, n, k in (
    (1, 10576, 2560), (16, 10577, 2560), (5, 6000, 2560), (16, 2000, 1300), (20, 6000, 700), (32, 8191, 2560), (20, 2000, 1300))]
# quantised on the way
FEW_QUANTISED = [(m, n, k, dtype) for dtype in (BF16, F32) for m, n, k in (
    (1, 10576, 2560), (7, 10576, 2560), (16, 10577, 2560), (3, 6000, 2570), (8, 2560, 5120), (16, 300, 900))]


def data(m, n, k, exact):
    gen = torch.Generator().manual_seed(m + 3 * n + 5 * k)
    a, w = operands(gen, m, n, k, exact)
    bias = torch.randint(-1000, 1000, (n,), generator=gen) / 16 if exact else 100 * torch.randn(n, generator=gen)
    values = [ref.unpack(*t).to(DEV) for t in (a, w)]
    return [t.to(DEV) for t in a], [t.to(DEV) for t in w], bias.to(DEV), values


def check(got, a, w, bias, exact):
    """Every element, in fp64 on the GPU."""
    want, err = ref.product(a, w, None if bias is None else bias.double())
    if exact:
        assert torch.equal(got, want.to(got.dtype))
        return
    want, err = rounded((want, err), got.dtype)
    off = (got.double() - want).abs()
    assert (off <= err).all(), f"{int((~(off <= err)).sum())} off, worst {float((off / err).max()):.2f} times the bound"


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("m,n,k,dtype", TILES + FEW, ids=str)
def test_whole_results(m, n, k, dtype, exact, bias):
    q, wq, b, (a, w) = data(m, n, k, exact)
    b = b if bias else None
    check(ssd.ssd_mx4_matmul(*q, *wq, bias=b, dtype=dtype), a, w, b, exact)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("m,n,k,dtype", FEW_QUANTISED + TILES[:1] + TILES[4:5] + TILES[7:8], ids=str)
def test_whole_results_from_activations(m, n, k, dtype, bias):
    """Activations that 4 bits hold exactly (a block's largest value only decides
    which of the equal codes is taken), and ones that they do not."""
    _, wq, b, (a, w) = data(m, n, k, True)
    b = b if bias else None
    x = a[:, :k].to(dtype)
    check(ssd.ssd_mx4_linear(x, *wq, bias=b), a, w, b, True)
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(m)).to(dtype)
    a = ref.unpack(*ref.pack(*ref.mx4(x.double()))) if m <= 16 else ref.unpack(*(t.cpu() for t in ssd.ssd_mx4_quant(x.to(DEV))))
    check(ssd.ssd_mx4_linear(x.to(DEV), *wq, bias=b), a.to(DEV), w, b, False)


@pytest.mark.parametrize("m,n,k,dtype", [(3400, 3328, 2200, BF16), (3400, 3328, 4200, F32)], ids=str)
def test_results_at_any_address(m, n, k, dtype):
    """Whole 16-byte rows at an address that is not a multiple of 16, and what lies
    before and behind them."""
    q, wq, b, (a, w) = data(m, n, k, True)
    room = torch.full((m * n + 16,), math.nan, dtype=dtype, device=DEV)
    y = room[1:1 + m * n].view(m, n)
    ssd.ssd_mx4_matmul(*q, *wq, bias=b, dtype=dtype, y=y)
    check(y, a, w, b, True)
    assert room[0].isnan() and room[1 + m * n:].isnan().all()


@pytest.mark.parametrize("m,n,k,dtype", [TILES[0], TILES[5], TILES[8], TILES[11]], ids=str)
def test_nan_blocks_in_large_products(m, n, k, dtype):
    """A block of scale byte 255 turns its token's or its output's results into
    NaN and leaves the others as they are, in the last tile and in the first."""
    q, wq, _, (a, w) = data(m, n, k, True)
    clean = ssd.ssd_mx4_matmul(*q, *wq, dtype=dtype)
    tokens, outputs, last = (0, 300, m - 1), (5, n - 1), q[1].shape[0] - 1
    for block, t in zip((0, 1, last), tokens):
        q[1][block, t, block % 4] = 255
    for block, t in zip((last, 0), outputs):
        wq[1][block, t, 0] = 255
    nan = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    for t in tokens:
        nan[t] = True
    for t in outputs:
        nan[:, t] = True
    got = ssd.ssd_mx4_matmul(*q, *wq, dtype=dtype)
    assert torch.equal(got.isnan(), nan) and torch.equal(got[~nan], clean[~nan])
