"""fp64 definitions of the operators between the layers (block norm and its
8-bit checkpoints, microscaled 4-bit values and products), each with a bound on
the rounding error of an fp32 evaluation; U, HALF and the pairs (result, bound)
as in layer_reference.py."""
import torch

from layer_reference import TINY, U, dsilu, silu

VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


# -------------------------------------------------------------- block norm


def rms(v, eps):
    return (v.square().mean(-1, keepdim=True) + eps).sqrt()


def ones(w, like):
    return torch.ones(like.shape[-1], dtype=torch.float64) if w is None else w


def block_stream(x, residual, z, post, scale, alpha, eps):
    """alpha residual + b: b is a product of seven factors; rstd has 48 additions
    of positive terms behind it, which the root halves."""
    n1 = x / rms(x, eps)
    b = n1 * ones(post, x) * ones(scale, x)
    e = 40 * U * b.abs()
    if z is not None:
        g, eg = silu(z)
        b, e = b * g, e * g.abs() + b.abs() * eg
    s = alpha * residual + b
    return s, e + 2 * U * (alpha * residual).abs() + U * s.abs()


def block_out(stream, pre, eps):
    """The second norm, of what the stream holds."""
    y = stream / rms(stream, eps) * ones(pre, stream)
    return y, 40 * U * y.abs()


def block_backward(x, stream, z, post, pre, scale, dy, dstream, alpha, eps):
    post1, pre1, scale1 = ones(post, x), ones(pre, x), ones(scale, x)
    mean = lambda q: q.mean(-1, keepdim=True)
    r1, r2 = 1 / rms(x, eps), 1 / rms(stream, eps)
    n1, n2 = x * r1, stream * r2
    g = pre1 * dy
    ds = r2 * (g - n2 * mean(g * n2))
    # every term of the difference is off by under 60 roundings: sums of 48,
    # which the root halves, and the products
    eds = 60 * U * r2 * (g.abs() + n2.abs() * mean((g * n2).abs()))
    if dstream is not None:
        ds = ds + dstream
        eds = eds + U * (ds.abs() + dstream.abs())
    c = scale1 * post1
    if z is None:
        f, ef = torch.ones_like(x), torch.zeros_like(x)
        dz = None
    else:
        f, ef = silu(z)
        d, ed = dsilu(z)
        v = ds * c * n1
        dz = (v * d, (c * n1).abs() * (eds * d.abs() + ds.abs() * ed) + 40 * U * (v * d).abs() + 40 * U * v.abs() * ed)
    h = ds * c * f
    eh = c.abs() * (eds * f.abs() + ds.abs() * ef) + 4 * U * h.abs()
    dx = r1 * (h - n1 * mean(h * n1))
    edx = r1 * (eh + n1.abs() * mean(eh * n1.abs()) + 100 * U * (h.abs() + n1.abs() * mean((h * n1).abs())))
    t = ds * f * n1
    et = n1.abs() * (eds * f.abs() + ds.abs() * ef) + 40 * U * t.abs()
    p = dy * n2
    # rows in a chain per part, parts: under 192 additions for the sizes tested
    m, em = t.sum(0), (et + 192 * U * t.abs()).sum(0)
    return {"dx": (dx, edx), "dresidual": (alpha * ds, abs(alpha) * eds + U * (alpha * ds).abs()), "dz": dz,
            "dpost_weight": None if post is None else (scale1 * m, scale1.abs() * em + 2 * U * (scale1 * m).abs() + TINY),
            "dscale": None if scale is None else (post1 * m, post1.abs() * em + 2 * U * (post1 * m).abs() + TINY),
            "dpre_weight": None if pre is None else (p.sum(0), ((40 + 192) * U * p.abs()).sum(0) + TINY)}


def kept_scales(v):
    """max(max |v|, 1e-12) / 448 of each 128 columns."""
    c = v.shape[-1]
    return torch.stack([v[..., i:i + 128].abs().amax(-1) for i in range(0, c, 128)], -1).clamp(min=1e-12) / 448


def per_column(scales, columns):
    return scales.repeat_interleave(128, -1)[..., :columns]


# ------------------------------------------------------------ 4-bit values


def mx4(v):
    """Codes [r, kp] and scale bytes [r, kp / 32] of v [r, c], fp64, from the
    nearest of the eight sizes, a tie to the even one."""
    r, c = v.shape
    blocks = torch.zeros(r, -(-c // 128) * 128, dtype=torch.float64)
    blocks[:, :c] = v
    blocks = blocks.reshape(r, -1, 32)
    m = blocks.abs().amax(-1)
    fine = torch.isfinite(m)
    exponent = torch.frexp(torch.where(fine, m, torch.ones_like(m))).exponent - 1   # floor(log2 m)
    byte = torch.where(m == 0, torch.zeros_like(exponent), (exponent + 125).clamp(min=0))
    unit = torch.ldexp(torch.ones_like(m), byte - 127)
    t = torch.where(fine[..., None], blocks.abs() / unit[..., None], torch.zeros_like(blocks))
    off = (t[..., None] - VALUES).abs()
    nearest = off.amin(-1, keepdim=True)
    even = torch.arange(8) % 2 == 0
    tied = off == nearest
    pick = torch.where((tied & even).any(-1), (tied & even).int().argmax(-1), tied.int().argmax(-1))
    code = pick + 8 * torch.signbit(blocks)
    code = torch.where(fine[..., None], code, torch.zeros_like(code)).reshape(r, -1)
    return code, torch.where(fine, byte, torch.full_like(byte, 255))


def pack(code, byte):
    """The layout of ssd_mx4_quant."""
    q = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    return q, byte.to(torch.uint8).reshape(code.shape[0], -1, 4).transpose(0, 1).contiguous()


def unpack(q, scales):
    """fp64 values [r, kp] of packed codes; NaN where the byte is 255."""
    q = q.long()
    code = torch.stack([q % 16, q // 16], -1).reshape(q.shape[0], -1)
    byte = scales.transpose(0, 1).reshape(q.shape[0], -1).long().repeat_interleave(32, 1)
    v = torch.where(code >= 8, -1.0, 1.0) * VALUES[code % 8] * torch.ldexp(torch.ones(()).double(), byte - 127)
    return torch.where(byte == 255, torch.full_like(v, float("nan")), v)


def product(a, w, bias):
    """The sums are of exact products, in any order and with what the matrix
    instruction rounds within its 64 or 128: one rounding an addition at most."""
    y = a @ w.t()
    size = a.abs() @ w.abs().t()
    if bias is not None:
        y, size = y + bias, size + bias.abs()
    return y, (a.shape[1] + 16) * U * size
