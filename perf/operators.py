"""The layer operators around the SSD scan, as measured cases.

Three families: the gated linear recurrence (``glr_*``), the short causal
depthwise convolution (``conv_*``) and the root-mean-square norm (``norm_*``).
With ``own`` false, ``run`` computes the plain form in elementary torch
operations (fp32, rounded once at the end); with ``own`` true it makes the
calls a user of ssd_chunked_scan_amd makes.  ``exact`` is the definition in
fp64, token by token where the operator is a recurrence.
"""
import math

import numpy as np
import torch

own = False

# Sizes: layer27b is 8 x 2048 tokens, 80 heads of 64 (5120 channels), one group
# of dstate 128; its block has a 2560-wide residual stream and a projection of
# z | x | B | C | dt, 2 * 5120 + 2 * 128 + 80 columns.  decay is 1 x 65536
# tokens of 1024 channels, packed 1 x 32768 tokens of 4096 channels (and
# 2 * 8 * 64 columns of B and C) in documents of 64 to 8192 tokens.


def listed():
    return [
        # one token for each of 8 sequences, at the 2.7B layer's width: what a
        # serving loop launches per layer and token
        dict(name="glr_step_b8", op="glr_step", batch=8, channels=5120, dtype="bf16", gate=True, normalize=True),
        # the training forward pass of a layer, gated output
        dict(name="glr_fwd_layer", op="glr_fwd", batch=8, seqlen=2048, channels=5120, dtype="bf16", gate=True,
             normalize=True, packed=False, init=False, sliced=True),
        # one long row and few channels: parallel over the sequence only
        dict(name="glr_fwd_long", op="glr_fwd", batch=1, seqlen=65536, channels=1024, dtype="bf16", gate=False,
             normalize=True, packed=False, init=True, sliced=False),
        # the training backward pass of a layer
        dict(name="glr_bwd_layer", op="glr_bwd", batch=8, seqlen=2048, channels=5120, dtype="bf16", gate=True,
             normalize=True, packed=False, init=False, sliced=True),
        # odd width and length, packed documents, fp32, unscaled input
        dict(name="glr_bwd_odd_f32", op="glr_bwd", batch=3, seqlen=1501, channels=1001, dtype="f32", gate=False,
             normalize=False, packed=True, init=True, sliced=False),
        # one token of 8 sequences through the window before the scan
        dict(name="conv_step_b8", op="conv_step", batch=8, channels=5376, width=4, dtype="bf16", silu=True),
        # the training forward pass: x | B | C read out of the projection's rows
        dict(name="conv_fwd_layer", op="conv_fwd", batch=8, seqlen=2048, channels=5376, width=4, dtype="bf16",
             silu=True, packed=False, init=False, row=10576),
        # the backward pass over packed documents
        dict(name="conv_bwd_packed", op="conv_bwd", batch=1, seqlen=32768, channels=5120, width=4, dtype="bf16",
             silu=True, packed=True, init=False, row=5120),
        # a decode step's entry norm with an 8-bit output for the projection
        dict(name="norm_quant_b8", op="norm_quant", rows=8, columns=2560, ngroups=1, dtype="bf16", residual=True,
             gate=False, block=128),
        # the training forward pass: the residual stream's addition and norm
        dict(name="norm_add_layer", op="norm_fwd", rows=16384, columns=2560, ngroups=1, dtype="bf16", residual=True,
             gate=False),
        # the gated norm after the scan, backward, at the layer's inner width
        dict(name="norm_gated_bwd_layer", op="norm_bwd", rows=16384, columns=5120, ngroups=1, dtype="bf16", gate=True,
             dresidual=False),
        # odd width in groups, fp32, with a gradient of the residual stream
        dict(name="norm_bwd_odd_f32", op="norm_bwd", rows=1501, columns=1477, ngroups=7, dtype="f32", gate=False,
             dresidual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["glr_step", "glr_fwd", "glr_bwd", "conv_step", "conv_fwd", "conv_bwd", "norm_quant", "norm_fwd",
                     "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    yes = lambda: rng.random() < 0.5
    if op in ("glr_step", "conv_step"):
        case = dict(op=op, batch=_log(rng, 1, 256), channels=_log(rng, 64, 8192), dtype=dtype)
        if op == "glr_step":
            case.update(gate=yes(), normalize=yes())
        else:
            case.update(width=rng.choice([2, 3, 4]), silu=yes())
        return case
    if op.startswith("norm"):
        ngroups = rng.choice([1, 1, 2, 8])
        per = _log(rng, 32, 8192 // ngroups)
        if yes():
            per = max(32, per // 8 * 8)
        columns = ngroups * per
        rows = _log(rng, 1, max(1, min(32768, 40_000_000 // columns)))
        case = dict(op=op, rows=rows, columns=columns, ngroups=ngroups, dtype=dtype, gate=False)
        kind = rng.choice(["none", "residual", "gate"])
        if op == "norm_bwd":
            case.update(gate=kind == "gate", dresidual=kind == "residual")
        else:
            case.update(gate=kind == "gate", residual=kind == "residual")
        if op == "norm_quant":
            case.update(block=rng.choice([0, 128]))
        return case
    channels = _log(rng, 64, 8192)
    if yes():
        channels = max(64, channels // 64 * 64)
    seqlen = _log(rng, 1, 65536)
    batch = _log(rng, 1, max(1, min(64, 40_000_000 // (seqlen * channels))))
    seqlen = max(1, min(seqlen, 40_000_000 // (batch * channels)))
    case = dict(op=op, batch=batch, seqlen=seqlen, channels=channels, dtype=dtype, packed=yes(), init=yes())
    if op.startswith("glr"):
        case.update(gate=yes(), normalize=yes(), sliced=yes())
    else:
        case.update(width=rng.choice([2, 3, 4]), silu=yes(), row=channels + rng.choice([0, 8, 137]))
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

    def uniform(n, lo, hi):
        return lo + (hi - lo) * torch.rand(n, generator=gen, device="cuda", dtype=f32)

    s = dict(case)
    op = case["op"]
    if op.startswith("norm"):
        r, c = case["rows"], case["columns"]
        s["x"] = normal(r, c, dtype=io)
        s["weight"] = 1.0 + 0.1 * normal(c)
        s["z"] = normal(r, c, dtype=io) if case["gate"] else None
        if op == "norm_bwd":
            s["dy"] = normal(r, c, dtype=io)
            s["dresidual"] = normal(r, c, dtype=io) if case["dresidual"] else None
        else:
            s["residual"] = normal(r, c, dtype=io) * 4 if case["residual"] else None
        return s
    b, d = case["batch"], case["channels"]
    step = op.endswith("step")
    lead = (b,) if step else (b, case["seqlen"])
    if op.startswith("glr"):
        # decays as in workloads.py: dt = softplus(bias) log-uniform in
        # [1e-3, 1e-1], A log-uniform in -[1, 16]
        dt = torch.exp(uniform(d, math.log(1e-3), math.log(1e-1)))
        s["bias"] = torch.log(torch.expm1(dt))
        s["A"] = -torch.exp(uniform(d, 0.0, math.log(16.0)))
        parts = 3 if case["gate"] else 2
        if case.get("sliced"):
            # the parts are column slices of one projection's rows
            cols = normal(*lead, parts * d, dtype=io).split(d, dim=-1)
        else:
            cols = [normal(*lead, d, dtype=io) for _ in range(parts)]
        s["x"], s["g"] = cols[0], cols[1]
        s["z"] = cols[2] if case["gate"] else None
        if step:
            s["state"] = normal(b, d)
            return s
        s["init"] = normal(b, d) if case["init"] else None
        if op == "glr_bwd":
            s["dy"] = normal(*lead, d, dtype=io)
            s["dfinal"] = normal(b, d) if case["init"] else None
    else:
        w = case["width"]
        s["weight"] = normal(d, w) / math.sqrt(w)
        s["bias"] = 0.1 * normal(d)
        if step:
            s["x"] = normal(b, d, dtype=io)
            s["state"] = normal(b, w - 1, d, dtype=io)
            return s
        s["x"] = normal(*lead, case["row"], dtype=io)[..., case["row"] - d:]
        s["init"] = normal(b, w - 1, d, dtype=io) if case["init"] else None
        if op == "conv_bwd":
            s["dy"] = normal(*lead, d, dtype=io)
            s["dfinal"] = normal(b, w - 1, d) if case["init"] else None
    s["seq_idx"] = None
    if case["packed"]:
        # documents of about 64 to 8192 tokens
        rng = np.random.default_rng(int(seed))
        length = np.exp(rng.uniform(math.log(64), math.log(8192)))
        starts = torch.from_numpy(rng.random(lead) < 1.0 / length)
        s["seq_idx"] = starts.cumsum(1).to(torch.int32).cuda()
    return s


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("norm"):
        n, c, r = case["rows"] * case["columns"], case["columns"], case["rows"]
        if op == "norm_bwd":
            tensors = 3 + 2 * case["gate"] + case["dresidual"]
            return dict(bytes=n * e * tensors + 8 * c, flops=n * (20 if case["gate"] else 10))
        read = 1 + case["gate"] + case["residual"]
        if op == "norm_fwd":
            return dict(bytes=n * e * (read + 1 + case["residual"]) + 4 * c, flops=n * (15 if case["gate"] else 6))
        per = c // case["ngroups"]
        scales = r * case["ngroups"] * (-(-per // case["block"]) if case["block"] else 1)
        return dict(bytes=n * (e * (read + case["residual"]) + 1) + 4 * c + 4 * scales, flops=n * 10)
    b, d = case["batch"], case["channels"]
    if op == "glr_step":
        return dict(bytes=b * d * (8 + e * (3 + case["gate"])) + 8 * d, flops=b * d * 40)
    if op == "conv_step":
        w = case["width"]
        return dict(bytes=b * d * e * (2 + 2 * (w - 1)) + 4 * d * (w + 1), flops=b * d * (2 * w + 10))
    n = b * case["seqlen"] * d
    seq = 4 * b * case["seqlen"] * case["packed"]
    if op.startswith("glr"):
        if op == "glr_fwd":
            return dict(bytes=n * e * (3 + case["gate"]) + 4 * b * d * (1 + case["init"]) + 8 * d + seq, flops=n * 40)
        return dict(bytes=n * e * (5 + 2 * case["gate"]) + 12 * b * d * case["init"] + 16 * d + seq, flops=n * 90)
    w = case["width"]
    win = b * d * (w - 1)
    if op == "conv_fwd":
        return dict(bytes=n * e * 2 + win * e * (1 + case["init"]) + 4 * d * (w + 1) + seq, flops=n * (2 * w + 10))
    return dict(bytes=n * e * 3 + win * (e + 8) * case["init"] + 8 * d * (w + 1) + seq, flops=n * (6 * w + 20))


# --------------------------------------------------------- the plain forms


def _starts(seq_idx):
    """True where a new document begins (never at a row's first token)."""
    s = torch.zeros_like(seq_idx, dtype=torch.bool)
    s[:, 1:] = seq_idx[:, 1:] != seq_idx[:, :-1]
    return s


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 1, by doubling: no elementary torch
    operation is such a scan, and log2(L) products of whole tensors are far
    quicker than L steps."""
    step = 1
    while step < a.shape[1]:
        u = torch.cat([u[:, :step], u[:, step:] + a[:, step:] * u[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return u


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _decay(s, x, g):
    """softplus, the log decay, the decay and the input's factor."""
    sp = _softplus(g + s["bias"])
    la = s["A"] * sp
    a = torch.exp(la)
    k = torch.sqrt(-torch.expm1(2 * la)) if s["normalize"] else torch.ones_like(a)
    return sp, la, a, k


def _glr_states(s, x, a, k):
    r = a
    if s["seq_idx"] is not None:
        r = torch.where(_starts(s["seq_idx"])[..., None], torch.zeros_like(a), a)
    u = k * x
    if s["init"] is not None:
        u = torch.cat([u[:, :1] + r[:, :1] * s["init"][:, None], u[:, 1:]], 1)
    return r, _scan(r, u)


def _plain_glr_fwd(s):
    io = s["x"].dtype
    x, g = s["x"].float(), s["g"].float()
    _, _, a, k = _decay(s, x, g)
    _, h = _glr_states(s, x, a, k)
    y = h
    if s["z"] is not None:
        z = s["z"].float()
        y = h * (z * torch.sigmoid(z))
    return dict(y=y.to(io), final=h[:, -1].clone())


def _plain_glr_bwd(s):
    io = s["x"].dtype
    x, g, dy = s["x"].float(), s["g"].float(), s["dy"].float()
    sp, la, a, k = _decay(s, x, g)
    r, h = _glr_states(s, x, a, k)
    e, dz = dy, None
    if s["z"] is not None:
        z = s["z"].float()
        sig = torch.sigmoid(z)
        e = dy * (z * sig)
        dz = (dy * h * (sig * (1 + z * (1 - sig)))).to(io)
    if s["dfinal"] is not None:
        e = torch.cat([e[:, :-1], e[:, -1:] + s["dfinal"][:, None]], 1)
    later = torch.cat([r[:, 1:], torch.zeros_like(r[:, :1])], 1)
    G = _scan(later.flip(1), e.flip(1)).flip(1)
    first = torch.zeros_like(h[:, :1]) if s["init"] is None else s["init"][:, None]
    dla = G * r * torch.cat([first, h[:, :-1]], 1)
    if s["normalize"]:
        dla = dla + torch.where(k > 0, -G * x * a * a / k, torch.zeros_like(k))
    dg = dla * s["A"] * torch.sigmoid(g + s["bias"])
    return dict(dx=(k * G).to(io), dg=dg.to(io), dz=dz, dA=(sp * dla).sum((0, 1)), dbias=dg.sum((0, 1)),
                dinit=None if s["init"] is None else r[:, 0] * G[:, 0])


def _plain_glr_step(s):
    x, g = s["x"].float(), s["g"].float()
    _, _, a, k = _decay(s, x, g)
    h = a * s["state"] + k * x
    y = h
    if s["z"] is not None:
        z = s["z"].float()
        y = h * (z * torch.sigmoid(z))
    s["state"].copy_(h)
    return dict(y=y.to(s["x"].dtype), state=s["state"])


def _windows(s):
    """[b, L, d, W]: the inputs each output sees, oldest first, with 0 for
    those before the start of its document; and which of them it sees."""
    x = s["x"].float()
    b, L, d = x.shape
    w = s["width"]
    before = torch.zeros(b, w - 1, d, device=x.device) if s["init"] is None else s["init"].float()
    win = torch.cat([before, x], 1).unfold(1, w, 1)
    if s["seq_idx"] is None:
        return win, None
    doc = torch.cat([torch.zeros(b, w - 1, dtype=torch.int64, device=x.device),
                     _starts(s["seq_idx"]).to(torch.int64).cumsum(1)], 1)
    same = (doc.unfold(1, w, 1) == doc[:, w - 1:, None])[:, :, None]
    return win * same, same


def _final_window(s):
    x = s["x"]
    b, L, d = x.shape
    w = s["width"]
    before = torch.zeros(b, w - 1, d, device=x.device, dtype=x.dtype) if s["init"] is None else s["init"]
    last = torch.cat([before, x], 1)[:, L:]
    if s["seq_idx"] is None:
        return last.clone()
    doc = torch.cat([torch.zeros(b, w - 1, dtype=torch.int64, device=x.device),
                     _starts(s["seq_idx"]).to(torch.int64).cumsum(1)], 1)
    return torch.where((doc[:, L:] == doc[:, -1:])[..., None], last, torch.zeros_like(last))


def _plain_conv_fwd(s):
    win, _ = _windows(s)
    p = (win * s["weight"]).sum(-1) + s["bias"]
    y = p * torch.sigmoid(p) if s["silu"] else p
    return dict(y=y.to(s["x"].dtype), final=_final_window(s))


def _plain_conv_bwd(s):
    win, same = _windows(s)
    b, L, d = s["x"].shape
    w = s["width"]
    ds = s["dy"].float()
    if s["silu"]:
        p = (win * s["weight"]).sum(-1) + s["bias"]
        sig = torch.sigmoid(p)
        ds = ds * (sig * (1 + p * (1 - sig)))
    taps = ds[..., None] * s["weight"]
    if same is not None:
        taps = taps * same
    # input at position q = t + i of [window | x] gets tap i of output t
    pad = torch.nn.functional.pad
    dcat = sum(pad(taps[..., i], (0, 0, i, w - 1 - i)) for i in range(w))
    if s["dfinal"] is not None:
        df = s["dfinal"]
        if s["seq_idx"] is not None:
            doc = torch.cat([torch.zeros(b, w - 1, dtype=torch.int64, device=ds.device),
                             _starts(s["seq_idx"]).to(torch.int64).cumsum(1)], 1)
            df = df * (doc[:, L:] == doc[:, -1:])[..., None]
        dcat[:, L:] += df
    return dict(dx=dcat[:, w - 1:].to(s["x"].dtype), dweight=(ds[..., None] * win).sum((0, 1)), dbias=ds.sum((0, 1)),
                dinit=None if s["init"] is None else dcat[:, :w - 1].clone())


def _plain_conv_step(s):
    win = torch.cat([s["state"], s["x"][:, None]], 1)
    p = (win.float() * s["weight"].t()).sum(1) + s["bias"]
    y = p * torch.sigmoid(p) if s["silu"] else p
    s["state"].copy_(win[:, 1:])
    return dict(y=y.to(s["x"].dtype), state=s["state"])


EPS = 1e-5


def _norm_input(s):
    """What is normalised, fp32, and the residual stream it leaves."""
    x = s["x"].float()
    if s.get("residual") is not None:
        stream = (x + s["residual"].float()).to(s["x"].dtype)
        return stream.float(), stream
    if s["z"] is not None:
        z = s["z"].float()
        return x * (z * torch.sigmoid(z)), None
    return x, None


def _normed(s, v):
    g = v.reshape(v.shape[0], s["ngroups"], -1)
    rstd = torch.rsqrt((g * g).mean(-1, keepdim=True) + EPS)
    return (g * rstd).reshape(v.shape), rstd


def _plain_norm_fwd(s):
    v, stream = _norm_input(s)
    n, _ = _normed(s, v)
    return dict(y=(n * s["weight"]).to(s["x"].dtype), residual=stream)


def _plain_norm_quant(s):
    v, stream = _norm_input(s)
    n, _ = _normed(s, v)
    y = (n * s["weight"]).reshape(v.shape[0], s["ngroups"], -1)
    per = y.shape[-1]
    block = s["block"] or per
    pad = -per % block
    blocks = torch.cat([y, y.new_zeros(*y.shape[:2], pad)], -1).reshape(*y.shape[:2], -1, block)
    m = blocks.abs().amax(-1, keepdim=True).clamp(min=1e-12)
    q = (blocks * (448.0 / m)).clamp(-448.0, 448.0)
    q = q.reshape(*y.shape[:2], -1)[..., :per].reshape(v.shape).to(torch.float8_e4m3fn)
    return dict(q=q, scales=(m / 448.0).reshape(v.shape[0], -1), residual=stream)


def _plain_norm_bwd(s):
    io = s["x"].dtype
    v, _ = _norm_input(s)
    n, rstd = _normed(s, v)
    dy = s["dy"].float()
    shape = (v.shape[0], s["ngroups"], -1)
    wdy = (dy * s["weight"]).reshape(shape)
    ng = n.reshape(shape)
    dv = (rstd * (wdy - ng * (wdy * ng).mean(-1, keepdim=True))).reshape(v.shape)
    if s["dresidual"] is not None:
        dv = dv + s["dresidual"].float()
    dx, dz = dv, None
    if s["z"] is not None:
        x, z = s["x"].float(), s["z"].float()
        sig = torch.sigmoid(z)
        dx = dv * (z * sig)
        dz = (dv * x * (sig * (1 + z * (1 - sig)))).to(io)
    return dict(dx=dx.to(io), dz=dz, dweight=(dy * n).sum(0))


_PLAIN = dict(glr_fwd=_plain_glr_fwd, glr_bwd=_plain_glr_bwd, glr_step=_plain_glr_step, conv_fwd=_plain_conv_fwd,
              conv_bwd=_plain_conv_bwd, conv_step=_plain_conv_step, norm_fwd=_plain_norm_fwd,
              norm_quant=_plain_norm_quant, norm_bwd=_plain_norm_bwd)


def _own(s):
    import ssd_chunked_scan_amd as ssd
    op = s["op"]
    if op == "glr_fwd":
        y, final = ssd.ssd_glr_fwd(s["x"], s["g"], s["A"], bias=s["bias"], z=s["z"], seq_idx=s["seq_idx"],
                                   init_states=s["init"], normalize=s["normalize"])
        return dict(y=y, final=final)
    if op == "glr_bwd":
        return ssd.ssd_glr_bwd(s["x"], s["g"], s["A"], s["bias"], s["dy"], z=s["z"], seq_idx=s["seq_idx"],
                               init_states=s["init"], dfinal=s["dfinal"], normalize=s["normalize"])
    if op == "glr_step":
        y = ssd.ssd_glr_step(s["x"], s["g"], s["A"], s["state"], bias=s["bias"], z=s["z"], normalize=s["normalize"])
        return dict(y=y, state=s["state"])
    if op == "conv_fwd":
        y, final = ssd.ssd_conv_fwd(s["x"], s["weight"], bias=s["bias"], seq_idx=s["seq_idx"], init_states=s["init"],
                                    silu=s["silu"])
        return dict(y=y, final=final)
    if op == "conv_bwd":
        return ssd.ssd_conv_bwd(s["x"], s["weight"], s["bias"], s["dy"], seq_idx=s["seq_idx"], init_states=s["init"],
                                dfinal=s["dfinal"], silu=s["silu"])
    if op == "conv_step":
        y = ssd.ssd_conv_step(s["x"], s["weight"], s["state"], bias=s["bias"], silu=s["silu"])
        return dict(y=y, state=s["state"])
    if op == "norm_fwd":
        y, stream = ssd.ssd_norm_fwd(s["x"], s["weight"], residual=s["residual"], z=s["z"], eps=EPS,
                                     ngroups=s["ngroups"])
        return dict(y=y, residual=stream)
    if op == "norm_quant":
        q, scales, stream = ssd.ssd_norm_quant_fwd(s["x"], s["weight"], residual=s["residual"], z=s["z"], eps=EPS,
                                                   ngroups=s["ngroups"], block=s["block"])
        return dict(q=q, scales=scales, residual=stream)
    return ssd.ssd_norm_bwd(s["x"], s["weight"], s["dy"], z=s["z"], dresidual=s["dresidual"], eps=EPS,
                            ngroups=s["ngroups"])


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------- exact


def _silu64(z):
    return z / (1 + torch.exp(-z))


def _dsilu64(z):
    sig = 1 / (1 + torch.exp(-z))
    return sig + z * sig * (1 - sig)


def _exact_glr(s):
    x, g = s["x"].double(), s["g"].double()
    A, bias = s["A"].double(), s["bias"].double()
    step = s["op"] == "glr_step"
    if step:
        x, g = x[:, None], g[:, None]
    L = x.shape[1]
    z = None if s["z"] is None else s["z"].double().reshape(x.shape)
    v = g + bias
    sp = torch.logaddexp(v, torch.zeros_like(v))
    la = A * sp
    a = la.exp()
    k = (-torch.special.expm1(2 * la)).sqrt() if s["normalize"] else torch.ones_like(a)
    keep = a
    if s.get("seq_idx") is not None:
        idx = s["seq_idx"]
        new = torch.cat([torch.zeros_like(idx[:, :1], dtype=torch.bool), idx[:, 1:] != idx[:, :-1]], 1)
        keep = a.masked_fill(new[..., None], 0.0)
    h0 = s["state"] if step else s["init"]
    h0 = x.new_zeros(x.shape[0], x.shape[2]) if h0 is None else h0.double()
    u = k * x
    h = torch.empty_like(u)
    last = h0
    for t in range(L):
        last = torch.addcmul(u[:, t], keep[:, t], last)
        h[:, t] = last
    if s["op"] != "glr_bwd":
        y = h if z is None else h * _silu64(z)
        return dict(y=y[:, 0], state=last) if step else dict(y=y, final=last)
    del u
    dy = s["dy"].double()
    G = dy if z is None else dy * _silu64(z)
    G = G.clone()
    if s["dfinal"] is not None:
        G[:, -1] += s["dfinal"].double()
    for t in range(L - 2, -1, -1):
        G[:, t] += keep[:, t + 1] * G[:, t + 1]
    dla = torch.empty_like(G)
    dla[:, 0] = G[:, 0] * keep[:, 0] * h0
    dla[:, 1:] = G[:, 1:] * keep[:, 1:] * h[:, :-1]
    if s["normalize"]:
        dla -= G * x * a.square() / k
    dg = dla * A / (1 + torch.exp(-v))
    return dict(dx=k * G, dg=dg, dz=None if z is None else dy * h * _dsilu64(z), dA=(dla * sp).sum((0, 1)),
                dbias=dg.sum((0, 1)), dinit=None if s["init"] is None else keep[:, 0] * G[:, 0])


def _exact_conv(s):
    w, wt, bias = s["width"], s["weight"].double(), s["bias"].double()
    x = s["x"].double()
    step = s["op"] == "conv_step"
    if step:
        x = x[:, None]
    b, L, d = x.shape
    before = s["state"] if step else s["init"]
    before = x.new_zeros(b, w - 1, d) if before is None else before.double()
    full = torch.cat([before, x], 1)
    begin = torch.zeros(b, L, dtype=torch.int64, device=x.device)   # first position of the token's document, in full
    if s.get("seq_idx") is not None:
        idx = s["seq_idx"]
        pos = torch.arange(L, device=x.device) + w - 1
        new = torch.cat([torch.zeros_like(idx[:, :1], dtype=torch.bool), idx[:, 1:] != idx[:, :-1]], 1)
        begin = torch.where(new, pos, torch.zeros_like(pos)).cummax(1).values
    q = torch.arange(L, device=x.device)
    p = bias.expand(b, L, d).clone()
    seen = []
    for i in range(w):   # tap i of output t reads full[t + i]
        seen.append(((q + i) >= begin)[..., None].double())
        p += wt[:, i] * full[:, i:i + L] * seen[i]
    last = full[:, L:] * (torch.arange(L, L + w - 1, device=x.device) >= begin[:, -1:])[..., None]
    if s["op"] != "conv_bwd":
        y = _silu64(p) if s["silu"] else p
        return dict(y=y[:, 0], state=last) if step else dict(y=y, final=last)
    ds = s["dy"].double()
    if s["silu"]:
        ds = ds * _dsilu64(p)
    dfull = torch.zeros_like(full)
    dw = torch.empty_like(wt)
    for i in range(w):
        t = ds * seen[i]
        dfull[:, i:i + L] += wt[:, i] * t
        dw[:, i] = (t * full[:, i:i + L]).sum((0, 1))
    if s["dfinal"] is not None:
        dfull[:, L:] += s["dfinal"].double() * (torch.arange(L, L + w - 1, device=x.device) >= begin[:, -1:])[..., None]
    return dict(dx=dfull[:, w - 1:], dweight=dw, dbias=ds.sum((0, 1)),
                dinit=None if s["init"] is None else dfull[:, :w - 1])


def _exact_norm(s):
    x, w = s["x"].double(), s["weight"].double()
    r, c = x.shape
    z = None if s["z"] is None else s["z"].double()
    stream = None
    v = x if z is None else x * _silu64(z)
    if s.get("residual") is not None:
        # the stream is rounded to the io type, and what is normalised is
        # what the stream holds; the sum of two io values is exact in fp64
        stream = (x + s["residual"].double()).to(s["x"].dtype)
        v = stream.double()
    ng = s["ngroups"]
    group = lambda t: t.reshape(r, ng, c // ng)
    rms = (group(v).square().sum(-1, keepdim=True) / (c // ng) + EPS).sqrt()
    n = (group(v) / rms).reshape(r, c)
    if s["op"] == "norm_fwd":
        return dict(y=n * w, residual=None if stream is None else stream.double())
    if s["op"] == "norm_quant":
        y = group(n * w)
        block = s["block"] or c // ng
        whole = -(-(c // ng) // block)
        m = torch.stack([y[..., i * block:(i + 1) * block].abs().amax(-1) for i in range(whole)], -1).clamp(min=1e-12)
        # the value each 8-bit number stands for, in units of its scale, before
        # its rounding
        q = (y / (m / 448.0).repeat_interleave(block, -1)[..., :c // ng]).reshape(r, c)
        return dict(q=q, scales=(m / 448.0).reshape(r, -1), residual=None if stream is None else stream.double())
    dy = s["dy"].double()
    wdy = group(w * dy)
    dot = (wdy * group(n)).sum(-1, keepdim=True) / (c // ng)
    dv = ((wdy - group(n) * dot) / rms).reshape(r, c)
    if s["dresidual"] is not None:
        dv = dv + s["dresidual"].double()
    return dict(dx=dv if z is None else dv * _silu64(z), dz=None if z is None else dv * x * _dsilu64(z),
                dweight=(dy * n).sum(0))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("glr"):
        return _exact_glr(s)
    return _exact_conv(s) if case["op"].startswith("conv") else _exact_norm(s)
