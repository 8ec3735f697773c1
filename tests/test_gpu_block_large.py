"""The operators between the layers on tensors of more than 2^32 bytes: the last
rows as a call on them alone gives them, bit by bit."""
import pytest
import torch

import ssd_chunked_scan_amd as ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def test_block_norm_of_many_rows():
    rows, columns, last = 900_000, 2560, 37          # 4.6 GB a tensor
    gen = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s, d=BF16: torch.randn(*s, generator=gen, device=DEV, dtype=d)
    x, residual, z, dy = (r(rows, columns) for _ in range(4))
    post, pre = 1 + 0.1 * r(columns, d=torch.float32), 1 + 0.1 * r(columns, d=torch.float32)
    tail = lambda t: t[-last:]
    y, stream, kept = ssd.ssd_block_norm_fwd(x, residual, post, pre, z=z, checkpoint=True)
    y1, stream1, kept1 = ssd.ssd_block_norm_fwd(tail(x), tail(residual), post, pre, z=tail(z), checkpoint=True)
    assert torch.equal(tail(y), y1) and torch.equal(tail(stream), stream1)
    for name in kept:
        assert torch.equal(tail(kept[name]).view(torch.uint8), kept1[name].view(torch.uint8)), name
    del y, y1
    for whole, part in (((x, stream, post, pre, dy, z), (tail(x), stream1, post, pre, tail(dy), tail(z))),
                        ((None, None, post, pre, dy), (None, None, post, pre, tail(dy)))):
        got = ssd.ssd_block_norm_bwd(*whole, checkpoint=kept if whole[0] is None else None)
        want = ssd.ssd_block_norm_bwd(*part, checkpoint=kept1 if whole[0] is None else None)
        for name in ("dx", "dresidual", "dz"):
            assert torch.equal(tail(got[name]), want[name]), name
        del got


def test_block_norm_of_rows_far_apart():
    columns, stride = 520, 1 << 31                   # 4 GiB from row to row
    gen = torch.Generator(device=DEV).manual_seed(2)
    memory = torch.empty(2 * stride + 4 * 1024, dtype=BF16, device=DEV)
    x, residual, z, dy = (memory.as_strided((3, columns), (stride, 1), 1024 * i) for i in range(4))
    for t in (x, residual, z, dy):
        t.copy_(torch.randn(3, columns, generator=gen, device=DEV))
    dense = lambda t: t.contiguous()
    y, stream, _ = ssd.ssd_block_norm_fwd(x, residual, z=z)
    y1, stream1, _ = ssd.ssd_block_norm_fwd(dense(x), dense(residual), z=dense(z))
    assert torch.equal(y, y1) and torch.equal(stream, stream1)
    far = residual
    far.copy_(stream)
    got = ssd.ssd_block_norm_bwd(x, far, None, None, dy, z=z, dresidual_out=dy)
    want = ssd.ssd_block_norm_bwd(dense(x), stream1, None, None, dense(dy), z=dense(z), dresidual_out=dense(dy))
    for name in ("dx", "dresidual", "dz"):
        assert torch.equal(got[name], want[name]), name
    q, scales = ssd.ssd_mx4_quant(x)
    q1, scales1 = ssd.ssd_mx4_quant(dense(x))
    assert torch.equal(q, q1) and torch.equal(scales, scales1)
    w = ssd.ssd_mx4_quant(torch.randn(70, columns, generator=gen, device=DEV).to(BF16))
    assert torch.equal(ssd.ssd_mx4_linear(x, *w), ssd.ssd_mx4_linear(dense(x), *w))


def whole_numbers(gen, rows, columns):
    """-3 .. 3, which 4 bits hold: products of up to 2^20 columns are exact."""
    return torch.randint(-3, 4, (rows, columns), generator=gen, device=DEV, dtype=torch.int8).to(BF16)


def test_mx4_of_many_rows():
    rows, columns, last = 1 << 20, 8320, 70          # 4.4 GB of codes
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = whole_numbers(gen, rows, columns)
    q, scales = ssd.ssd_mx4_quant(x)
    q1, scales1 = ssd.ssd_mx4_quant(x[-last:])
    assert torch.equal(q[-last:], q1) and torch.equal(scales[:, -last:], scales1)
    assert torch.equal(ssd.ssd_mx4_dequant(q, scales, columns)[-last:], x[-last:])
    w = whole_numbers(gen, 40, columns)
    want = (x[-last:].double() @ w.double().t()).float()
    y = ssd.ssd_mx4_matmul(q, scales, *ssd.ssd_mx4_quant(w), dtype=torch.float32)
    assert torch.equal(y[-last:], want)
    for m in (5, 20, 40):                            # the same as weights
        y = ssd.ssd_mx4_matmul(*ssd.ssd_mx4_quant(w[:m]), q, scales, dtype=torch.float32)
        assert torch.equal(y[:, -last:], want[:, :m].t())


@pytest.mark.parametrize("m,n,k,dtype", [(70_001, 33_000, 200, BF16), (70_001, 33_000, 600, BF16),
                                         (33_001, 33_001, 600, torch.float32)])
def test_products_of_many_results(m, n, k, dtype):
    gen = torch.Generator(device=DEV).manual_seed(k)
    a, w = whole_numbers(gen, m, k), whole_numbers(gen, n, k)
    y = ssd.ssd_mx4_matmul(*ssd.ssd_mx4_quant(a), *ssd.ssd_mx4_quant(w), dtype=dtype)
    assert y.numel() * y.element_size() > 1 << 32
    for rows in (slice(0, 70), slice(m - 70, m)):
        assert torch.equal(y[rows], (a[rows].double() @ w.double().t()).to(dtype))
