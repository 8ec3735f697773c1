"""The operators between the layers, as measured cases.

Two families: the block norm (``block_fwd``, ``block_bwd``: the norm after a
block with its gate and residual scale, the residual's addition and the norm
before the next block, with 8-bit checkpoints for the backward pass) and
microscaled 4-bit floating point (``mx4_quant``: to 4 bits and back,
``mx4_linear``: activations times 4-bit weights, ``mx4_matmul``: both already
in 4 bits).  With ``own`` false, ``run`` computes the plain form in elementary
torch operations (fp32, rounded once at the end); with ``own`` true it makes
the calls a user of ssd_chunked_scan_amd makes.  ``exact`` is the definition
in fp64.
"""
import math

import torch

own = False

# Sizes: layer27b is 8 x 2048 tokens; its block has a 2560-wide residual
# stream, a projection into z | x | B | C | dt of 2 * 5120 + 2 * 128 + 80
# columns and one from 5120 columns back.


def listed():
    return [
        # the activations of a decode step of 8 sequences into 4 bits and back
        dict(name="mx4_quant_b8", op="mx4_quant", rows=8, columns=2560, dtype="bf16"),
        # the weights of the layer's first projection, once when they are loaded
        dict(name="mx4_quant_weight", op="mx4_quant", rows=10576, columns=2560, dtype="bf16"),
        # one token of one sequence through the first projection
        dict(name="mx4_linear_b1", op="mx4_linear", m=1, n=10576, k=2560, dtype="bf16", bias=False),
        # one token of 8 sequences through the second projection
        dict(name="mx4_linear_b8", op="mx4_linear", m=8, n=2560, k=5120, dtype="bf16", bias=False),
        # a prompt's tokens through the first projection
        dict(name="mx4_linear_in", op="mx4_linear", m=16384, n=10576, k=2560, dtype="bf16", bias=False),
        # and through the second
        dict(name="mx4_linear_out", op="mx4_linear", m=16384, n=2560, k=5120, dtype="bf16", bias=False),
        # odd sizes, fp32 result, activations that several products share
        dict(name="mx4_matmul_odd_f32", op="mx4_matmul", m=1501, n=1001, k=1477, dtype="f32", bias=True),
        # the seam of a decode step of 8 sequences
        dict(name="block_fwd_b8", op="block_fwd", rows=8, columns=2560, dtype="bf16", gate=True, scale=True, alpha=1.0,
             checkpoint=False),
        # the training forward pass, keeping 8-bit checkpoints
        dict(name="block_fwd_layer", op="block_fwd", rows=16384, columns=2560, dtype="bf16", gate=True, scale=True,
             alpha=1.0, checkpoint=True),
        # the training backward pass from what the forward pass saw
        dict(name="block_bwd_layer", op="block_bwd", rows=16384, columns=2560, dtype="bf16", gate=True, scale=True,
             alpha=1.0, checkpoint=False),
        # and from its checkpoints
        dict(name="block_bwd_ckpt", op="block_bwd", rows=16384, columns=2560, dtype="bf16", gate=True, scale=True,
             alpha=1.0, checkpoint=True),
        # odd width, fp32, no gate, the residual scaled
        dict(name="block_bwd_odd_f32", op="block_bwd", rows=1501, columns=1477, dtype="f32", gate=False, scale=False,
             alpha=0.8125, checkpoint=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mx4_quant", "mx4_linear", "mx4_linear", "mx4_matmul", "block_fwd", "block_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    yes = lambda: rng.random() < 0.5
    if op in ("mx4_linear", "mx4_matmul"):
        n, k = _log(rng, 64, 10576), _log(rng, 64, 8192)
        if yes():
            n, k = max(64, n // 16 * 16), max(64, k // 128 * 128)
        m = _log(rng, 1, max(1, min(16384, 40_000_000_000 // (n * k))))
        return dict(op=op, m=m, n=n, k=k, dtype=dtype, bias=yes())
    columns = _log(rng, 32, 8192)
    if yes():
        columns = max(32, columns // 8 * 8)
    rows = _log(rng, 1, max(1, min(32768, 27_000_000 // columns)))
    case = dict(op=op, rows=rows, columns=columns, dtype=dtype)
    if op != "mx4_quant":
        case.update(gate=yes(), scale=yes(), alpha=rng.choice([1.0, 1.0, 0.8125]), checkpoint=yes())
    return case


# ------------------------------------------------------------------ inputs


def _io(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    io = _io(case)
    f32 = torch.float32

    def normal(*shape, dtype=f32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=f32).to(dtype)

    def activations(rows, columns):
        # a few columns are much larger than the others, as in a residual stream
        size = torch.exp(0.5 * normal(columns)) * (1 + 15 * (torch.rand(columns, generator=gen, device="cuda") < 0.01))
        return (normal(rows, columns) * size).to(io)

    s = dict(case)
    op = case["op"]
    if op == "mx4_quant":
        s["x"] = activations(case["rows"], case["columns"])
        return s
    if op in ("mx4_linear", "mx4_matmul"):
        m, n, k = case["m"], case["n"], case["k"]
        s["wq"], s["wscales"] = _mx4_pack(*_mx4_round(normal(n, k) / math.sqrt(k)))
        s["x"] = activations(m, k)
        if op == "mx4_matmul":
            s["q"], s["scales"] = _mx4_pack(*_mx4_round(s.pop("x").float()))
        s["bias"] = 0.1 * normal(n) if case["bias"] else None
        return s
    r, c = case["rows"], case["columns"]
    x, z = activations(r, c), normal(r, c, dtype=io) if case["gate"] else None
    stream = normal(r, c, dtype=io) * 4
    s["post"], s["pre"] = 1.0 + 0.1 * normal(c), 1.0 + 0.1 * normal(c)
    s["scale"] = 0.1 + 0.02 * normal(c) if case["scale"] else None
    if op == "block_fwd":
        s.update(x=x, z=z, residual=stream)
        return s
    s["dy"], s["dstream"] = normal(r, c, dtype=io), normal(r, c, dtype=io)
    if case["checkpoint"]:
        s["kept"] = {}
        for name, t in (("x", x), ("z", z), ("residual", stream)):
            if t is not None:
                s["kept"][name + "_q"], s["kept"][name + "_scales"] = _e4m3_blocks(t.float())
    else:
        s.update(x=x, z=z, stream=stream)
    return s


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("mx4"):
        bits = lambda rows, columns: rows * -(-columns // 128) * 68   # codes and scales of padded rows
        if op == "mx4_quant":
            r, c = case["rows"], case["columns"]
            return dict(bytes=2 * r * c * e + 2 * bits(r, c), flops=r * c * 10)
        m, n, k = case["m"], case["n"], case["k"]
        a = bits(m, k) if op == "mx4_matmul" else m * k * e
        return dict(bytes=a + bits(n, k) + m * n * e + 4 * n * case["bias"], flops=2 * m * n * k)
    r, c = case["rows"], case["columns"]
    n, weights = r * c, 4 * c * (2 + case["scale"])
    kept = r * (c + 4 * -(-c // 128)) * (2 + case["gate"])   # the checkpoints
    if op == "block_fwd":
        return dict(bytes=n * e * (4 + case["gate"]) + weights + kept * case["checkpoint"], flops=n * 25)
    saved = kept if case["checkpoint"] else n * e * (2 + case["gate"])
    return dict(bytes=saved + n * e * (4 + case["gate"]) + 2 * weights, flops=n * 45)


# --------------------------------------------------------- the plain forms


def _e4m3_blocks(v):
    """[r, c] fp32 as e4m3 with a scale for each 128 columns."""
    r, c = v.shape
    blocks = torch.cat([v, v.new_zeros(r, -c % 128)], 1).reshape(r, -1, 128)
    m = blocks.abs().amax(-1, keepdim=True).clamp(min=1e-12)
    q = (blocks * (448.0 / m)).clamp(-448.0, 448.0).reshape(r, -1)[:, :c]
    return q.to(torch.float8_e4m3fn).contiguous(), (m / 448.0).reshape(r, -1)


def _e4m3_values(q, scales):
    return q.float() * scales.repeat_interleave(128, 1)[:, :q.shape[1]]


def _mx4_round(v):
    """[r, c] fp32 -> the 4-bit values [r, cp] in units of their block's scale,
    and the scales' exponents [r, cp / 32]; cp = c padded to a multiple of 128."""
    r, c = v.shape
    blocks = torch.cat([v, v.new_zeros(r, -c % 128)], 1).reshape(r, -1, 32)
    e = (torch.frexp(blocks.abs().amax(-1)).exponent - 3).clamp(min=-127)   # 0.5 <= mantissa < 1
    # 2^-e may not fit fp32 at either end: in two factors
    u = torch.ldexp(torch.ldexp(blocks, -(e // 2)[..., None]), -(e - e // 2)[..., None])
    e = torch.where((blocks == 0).all(-1), torch.full_like(e, -127), e)
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(u / step) * step).clamp(-6, 6).reshape(r, -1), e


_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _mx4_pack(u, e):
    """Codes, two to a byte with the earlier column low, and scale bytes
    [cp / 128, r, 4]."""
    table = torch.tensor(_VALUES, device=u.device)
    code = torch.bucketize(u.abs(), table).to(torch.uint8) | (torch.signbit(u).to(torch.uint8) << 3)
    q = code[:, 0::2] | (code[:, 1::2] << 4)
    return q.contiguous(), (e + 127).to(torch.uint8).reshape(u.shape[0], -1, 4).transpose(0, 1).contiguous()


def _mx4_values(q, scales):
    """[r, cp] fp32 values of packed codes and scales."""
    r = q.shape[0]
    table = torch.tensor(_VALUES + tuple(-v for v in _VALUES), device=q.device)
    u = torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], -1).reshape(r, -1, 32)
    e = scales.transpose(0, 1).reshape(r, -1, 1).int() - 127
    return torch.ldexp(torch.ldexp(u, e // 2), e - e // 2).reshape(r, -1)


def _plain_mx4_quant(s):
    x = s["x"]
    u, e = _mx4_round(x.float())
    e = e.repeat_interleave(32, 1)
    return dict(values=torch.ldexp(torch.ldexp(u, e // 2), e - e // 2)[:, :x.shape[1]].to(x.dtype))


def _plain_product(s, a):
    y = a @ _mx4_values(s["wq"], s["wscales"]).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return dict(y=y.to(_io(s)))


def _plain_mx4_linear(s):
    u, e = _mx4_round(s["x"].float())
    e = e.repeat_interleave(32, 1)
    return _plain_product(s, torch.ldexp(torch.ldexp(u, e // 2), e - e // 2))


def _plain_mx4_matmul(s):
    return _plain_product(s, _mx4_values(s["q"], s["scales"]))


EPS = 1e-5


def _rstd(v):
    return torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _plain_block_fwd(s):
    io = s["x"].dtype
    x = s["x"].float()
    b = x * _rstd(x) * s["post"]
    if s["z"] is not None:
        z = s["z"].float()
        b = b * (z * torch.sigmoid(z))
    if s["scale"] is not None:
        b = b * s["scale"]
    stream = (s["alpha"] * s["residual"].float() + b).to(io)
    v = stream.float()
    out = dict(y=(v * _rstd(v) * s["pre"]).to(io), residual=stream)
    if s["checkpoint"]:
        out["kept"] = {}
        for name, t in (("x", s["x"]), ("z", s["z"]), ("residual", stream)):
            if t is not None:
                out["kept"][name + "_q"], out["kept"][name + "_scales"] = _e4m3_blocks(t.float())
    return out


def _plain_block_bwd(s):
    io = s["dy"].dtype
    if s["checkpoint"]:
        kept = s["kept"]
        x, v = (_e4m3_values(kept[n + "_q"], kept[n + "_scales"]) for n in ("x", "residual"))
        z = _e4m3_values(kept["z_q"], kept["z_scales"]) if s["gate"] else None
    else:
        x, v = s["x"].float(), s["stream"].float()
        z = s["z"].float() if s["gate"] else None
    dy = s["dy"].float()
    r2 = _rstd(v)
    n2 = v * r2
    g = dy * s["pre"]
    ds = r2 * (g - n2 * (g * n2).mean(-1, keepdim=True)) + s["dstream"].float()
    r1 = _rstd(x)
    n1 = x * r1
    ones = torch.ones_like(s["post"])
    scale = ones if s["scale"] is None else s["scale"]
    gate, dz = 1.0, None
    if z is not None:
        sig = torch.sigmoid(z)
        gate = z * sig
        dz = (ds * scale * s["post"] * n1 * (sig * (1 + z * (1 - sig)))).to(io)
    h = ds * scale * gate * s["post"]
    m = (ds * gate * n1).sum(0)
    return dict(dx=(r1 * (h - n1 * (h * n1).mean(-1, keepdim=True))).to(io), dresidual=(s["alpha"] * ds).to(io), dz=dz,
                dpost_weight=m * scale, dpre_weight=(dy * n2).sum(0), dscale=None if s["scale"] is None else m * s["post"])


_PLAIN = dict(mx4_quant=_plain_mx4_quant, mx4_linear=_plain_mx4_linear, mx4_matmul=_plain_mx4_matmul,
              block_fwd=_plain_block_fwd, block_bwd=_plain_block_bwd)


def _own(s):
    import ssd_chunked_scan_amd as ssd
    op = s["op"]
    if op == "mx4_quant":
        q, scales = ssd.ssd_mx4_quant(s["x"])
        return dict(values=ssd.ssd_mx4_dequant(q, scales, s["columns"], dtype=s["x"].dtype))
    if op == "mx4_linear":
        return dict(y=ssd.ssd_mx4_linear(s["x"], s["wq"], s["wscales"], bias=s["bias"]))
    if op == "mx4_matmul":
        return dict(y=ssd.ssd_mx4_matmul(s["q"], s["scales"], s["wq"], s["wscales"], bias=s["bias"], dtype=_io(s)))
    if op == "block_fwd":
        y, stream, kept = ssd.ssd_block_norm_fwd(s["x"], s["residual"], s["post"], s["pre"], z=s["z"], scale=s["scale"],
                                                 alpha=s["alpha"], eps=EPS, checkpoint=s["checkpoint"])
        return dict(y=y, residual=stream, kept=kept) if s["checkpoint"] else dict(y=y, residual=stream)
    if s["checkpoint"]:
        return ssd.ssd_block_norm_bwd(None, None, s["post"], s["pre"], s["dy"], scale=s["scale"],
                                      dresidual_out=s["dstream"], alpha=s["alpha"], eps=EPS, checkpoint=s["kept"])
    return ssd.ssd_block_norm_bwd(s["x"], s["stream"], s["post"], s["pre"], s["dy"], z=s["z"], scale=s["scale"],
                                  dresidual_out=s["dstream"], alpha=s["alpha"], eps=EPS)


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------- exact


def _nearest64(v):
    """Each element of v [r, c] as the value of its 4-bit code, in fp64."""
    r, c = v.shape
    out = torch.zeros(r, -(-c // 32) * 32, dtype=torch.float64, device=v.device)
    out[:, :c] = v
    block = out.view(r, -1, 32)
    most = block.abs().max(-1, keepdim=True).values
    unit = torch.where(most > 0, 2.0 ** (most.clamp(min=2.0 ** -300).log2().floor() - 2), torch.ones_like(most))
    # log2 may be off by an ulp next to a power of two
    unit = torch.where(most >= 8 * unit, 2 * unit, torch.where((most < 4 * unit) & (most > 0), unit / 2, unit))
    unit = unit.clamp(min=2.0 ** -127)
    t = block.abs() / unit
    # the borders between neighbouring values; a tie goes to the even code
    near = torch.zeros_like(t)
    values = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
    for i in range(1, 8):
        border = (values[i - 1] + values[i]) / 2
        above = t >= border if i % 2 == 0 else t > border
        near = torch.where(above, torch.full_like(t, values[i]), near)
    return (near * unit * torch.sign(block)).view(r, -1)[:, :c]


def _expand64(q, scales):
    """[r, cp] fp64 of packed 4-bit codes."""
    code = torch.stack([q % 16, q // 16], -1).reshape(q.shape[0], -1).long()
    low, mid = code % 2, (code // 2) % 4
    # exponent field 0: 0 or 1/2; else (1 + low / 2) 2^(mid - 1)
    size = torch.where(mid == 0, 0.5 * low.double(), (1 + 0.5 * low.double()) * 2.0 ** (mid.double() - 1))
    value = torch.where(code >= 8, -size, size)
    power = scales.permute(1, 0, 2).reshape(q.shape[0], -1).double() - 127
    return value * (2.0 ** power).repeat_interleave(32, 1)


def _values8(q, scales):
    columns = torch.arange(q.shape[1], device=q.device) // 128
    return q.to(torch.float32).double() * scales.double()[:, columns]


def _rms64(v):
    return (v.square().sum(-1, keepdim=True) / v.shape[1] + EPS).sqrt()


def _units8(v):
    """v in units of its block's scale, before the rounding, and the scales."""
    r, c = v.shape
    most = torch.stack([v[:, i:i + 128].abs().amax(1) for i in range(0, c, 128)], 1).clamp(min=1e-12)
    scale = most / 448
    return v / scale.repeat_interleave(128, 1)[:, :c], scale


def _exact_block(s):
    post, pre = s["post"].double(), s["pre"].double()
    scale = torch.ones_like(post) if s["scale"] is None else s["scale"].double()
    if s["op"] == "block_fwd":
        x = s["x"].double()
        v = x / _rms64(x) * post * scale
        if s["gate"]:
            z = s["z"].double()
            v = v * z / (1 + torch.exp(-z))
        v = v + s["alpha"] * s["residual"].double()
        # what is normed, and kept, is the stream as its type holds it
        stream = v.to(s["x"].dtype).double()
        out = dict(y=stream / _rms64(stream) * pre, residual=v)
        if s["checkpoint"]:
            out["kept"] = {}
            for name, t in (("x", x), ("z", z if s["gate"] else None), ("residual", stream)):
                if t is not None:
                    out["kept"][name + "_q"], out["kept"][name + "_scales"] = _units8(t)
        return out
    if s["checkpoint"]:
        x, v, z = (_values8(s["kept"][n + "_q"], s["kept"][n + "_scales"]) if n + "_q" in s["kept"] else None
                   for n in ("x", "residual", "z"))
    else:
        x, v, z = (None if t is None else t.double() for t in (s["x"], s["stream"], s["z"]))
    c = x.shape[1]
    dy = s["dy"].double()
    rms2 = _rms64(v)
    n2 = v / rms2
    w = pre * dy
    ds = (w - n2 * ((w * n2).sum(-1, keepdim=True) / c)) / rms2 + s["dstream"].double()
    rms1 = _rms64(x)
    n1 = x / rms1
    if z is None:
        silu, slope = torch.ones_like(x), None
    else:
        sig = 1 / (1 + torch.exp(-z))
        silu, slope = z * sig, sig + z * sig * (1 - sig)
    up = ds * silu * scale * post
    dx = (up - n1 * ((up * n1).sum(-1, keepdim=True) / c)) / rms1
    return dict(dx=dx, dresidual=s["alpha"] * ds, dz=None if z is None else ds * scale * post * n1 * slope,
                dpost_weight=(ds * scale * silu * n1).sum(0), dpre_weight=(dy * n2).sum(0),
                dscale=None if s["scale"] is None else (ds * post * silu * n1).sum(0))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("block"):
        return _exact_block(s)
    if case["op"] == "mx4_quant":
        return dict(values=_nearest64(s["x"].double()))
    k = case["k"]
    a = _nearest64(s["x"].double()) if case["op"] == "mx4_linear" else _expand64(s["q"], s["scales"])[:, :k]
    y = a @ _expand64(s["wq"], s["wscales"])[:, :k].t()
    return dict(y=y if s["bias"] is None else y + s["bias"].double())
