"""4-bit operands with every scale byte, those that ssd_mx4_quant does not write
among them."""
import pytest
import torch

import block_reference as ref

import ssd_chunked_scan_amd as ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_code_of_every_scale(dtype):
    """Exact up to byte 252; past it what the type does not hold is an infinity."""
    code = torch.arange(128).remainder(16).repeat(256, 1)
    byte = torch.arange(256)[:, None].repeat(1, 4)
    q, scales = ref.pack(code, byte)
    want = ref.unpack(q, scales)
    got = ssd.ssd_mx4_dequant(q.to(DEV), scales.to(DEV), 128, dtype=dtype).cpu()
    assert got[255].isnan().all()
    assert torch.equal(got[:253].double(), want[:253])
    assert torch.equal(got[:255], want[:255].to(dtype)) and got[253:255].isinf().any()


@pytest.mark.parametrize("m,n,k", [(3, 300, 700), (20, 300, 700), (100, 130, 700), (2000, 1030, 640), (4100, 4200, 600)])
@pytest.mark.parametrize("byte", [0, 1, 60, 200, 252, 253, 254])
def test_products_of_small_and_large_scales(m, n, k, byte):
    """One operand's scales 2^(byte - 127), the other's such that their products are
    1/2, 1 or 2: sums of multiples of 1/8 below 2^24 of them, exact in fp32."""
    gen = torch.Generator().manual_seed(m + byte)
    kb = -(-k // 128)

    def make(rows, scale):
        code = torch.randint(0, 16, (rows, kb * 128), generator=gen)
        code[:, k:] = 0
        return ref.pack(code, scale(rows, 4 * kb))

    low, high = max(253 - byte, 0), min(255 - byte, 254)
    a = make(m, lambda *s: torch.full(s, byte))
    w = make(n, lambda *s: torch.randint(low, high + 1, s, generator=gen))
    got = ssd.ssd_mx4_matmul(*(t.to(DEV) for t in (*a, *w)), dtype=torch.float32)
    assert torch.equal(got.double(), ref.unpack(*a).to(DEV) @ ref.unpack(*w).to(DEV).t())
