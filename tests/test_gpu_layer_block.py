"""The layer operators together, as a layer uses them: norm with the residual,
convolution, scan (gated recurrence or SSD), gated norm; forward, backward and
token by token, in fp32 against fp64 definitions of the whole chain.

Tolerances, relative to the largest value of the tensor: an operator's output
is off by a few tens of roundings of 2^-24 of its largest terms
(layer_reference.py counts them: under 60 for values of order one), and a
chain of four passes those on with factors of order one, each operator adding
its own; 64 roundings for each of the operators passed through, 4 x 64 x
2^-24 = 1.6e-5 forward and 8 x 64 x 2^-24 = 3.1e-5 forward and back.  The SSD
scan in fp32 is held to its own bound, 1e-4."""
import math

import pytest
import torch

import layer_reference as ref

import ssd_chunked_scan_amd as ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FWD, BWD = 4 * 64 * ref.U, 8 * 64 * ref.U


def near(name, got, want, tol):
    off = float((got.detach().double().cpu() - want.detach()).abs().max() / want.detach().abs().max())
    assert off <= tol, (name, off, tol)


def layer_inputs(b, L, D, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    dt = torch.exp(torch.rand(D, generator=gen) * math.log(100.0) + math.log(1e-3))
    return dict(proj=r(b, L, 3 * D), residual=r(b, L, D), w=0.5 * r(D, 4), cb=0.1 * r(D), bias=torch.log(torch.expm1(dt)),
                A=-torch.exp(torch.rand(D, generator=gen) * math.log(16.0)), nw=1 + 0.2 * r(D)), r


def run_layer(p, seq, conv_state=None, state=None):
    """conv -> gated recurrence -> residual addition and norm; the projection's
    columns are x | g | z."""
    D = p["A"].numel()
    x, g, z = p["proj"].split(D, dim=-1)
    xc, conv_state = ssd.ssd_conv_fwd(x, p["w"], bias=p["cb"], seq_idx=seq, init_states=conv_state)
    y, state = ssd.ssd_glr_fwd(xc, g, p["A"], bias=p["bias"], z=z, seq_idx=seq, init_states=state)
    out, stream = ssd.ssd_norm_fwd(y, p["nw"], residual=p["residual"])
    return dict(xc=xc, y=y, out=out, stream=stream, conv_state=conv_state, state=state)


def reference_layer(p, seq):
    D = p["A"].numel()
    x, g, z = p["proj"].split(D, dim=-1)
    (xc, _), conv_state = ref.conv(x, p["w"], p["cb"], seq, None, True)
    (y, _), (state, _) = ref.Glr(xc, g, p["A"], p["bias"], z, seq, None, True).outputs()
    stream = y + p["residual"]
    out = ref.norm(stream.reshape(-1, D), 0.0, p["nw"], 1e-5, 1)[0].reshape(stream.shape)
    return out, stream, conv_state, state


@pytest.mark.parametrize("b,L,D,packed", [(2, 150, 48, True), (1, 700, 33, False), (3, 1, 64, False)])
def test_layer_forward_and_backward(b, L, D, packed):
    p, r = layer_inputs(b, L, D, seed=L)
    seq = ((torch.rand(b, L) < 0.03).cumsum(1)).int() if packed else None
    dout, dstream = r(b, L, D), r(b, L, D)
    q = {k: v.to(DEV) for k, v in p.items()}
    sq = None if seq is None else seq.to(DEV)
    f = run_layer(q, sq)
    gn = ssd.ssd_norm_bwd(f["stream"], q["nw"], dout.to(DEV), dresidual=dstream.to(DEV))
    x, g, z = q["proj"].split(D, dim=-1)
    gg = ssd.ssd_glr_bwd(f["xc"], g, q["A"], q["bias"], gn["dx"], z=z, seq_idx=sq)
    gc = ssd.ssd_conv_bwd(x, q["w"], q["cb"], gg["dx"], seq_idx=sq)

    t = {k: v.double().requires_grad_() for k, v in p.items()}
    out, stream, conv_state, state = reference_layer(t, seq)
    ((out * dout.double()).sum() + (stream * dstream.double()).sum()).backward()
    near("out", f["out"], out, FWD)
    near("stream", f["stream"], stream, FWD)
    near("state", f["state"], state, FWD)
    near("dproj", torch.cat([gc["dx"], gg["dg"], gg["dz"]], -1), t["proj"].grad, BWD)
    near("dresidual", gn["dx"], t["residual"].grad, BWD)
    for name, got in (("w", gc["dweight"]), ("cb", gc["dbias"]), ("A", gg["dA"]), ("bias", gg["dbias"]),
                      ("nw", gn["dweight"])):
        near("d" + name, got, t[name].grad, BWD)


def test_layer_served_token_by_token():
    """A prompt in two pieces, then single tokens from the same states."""
    p, _ = layer_inputs(2, 40, 66, seed=5)
    q = {k: v.to(DEV) for k, v in p.items()}
    D = 66
    piece = lambda lo, hi: dict(q, proj=q["proj"][:, lo:hi].contiguous(), residual=q["residual"][:, lo:hi].contiguous())
    a = run_layer(piece(0, 17), None)
    c = run_layer(piece(17, 30), None, a["conv_state"], a["state"])
    conv_state, state, outs = c["conv_state"], c["state"], [a["out"], c["out"]]
    for t in range(30, 40):
        x, g, z = q["proj"][:, t].split(D, dim=-1)
        xc = ssd.ssd_conv_step(x, q["w"], conv_state, bias=q["cb"])
        y = ssd.ssd_glr_step(xc, g, q["A"], state, bias=q["bias"], z=z)
        outs.append(ssd.ssd_norm_fwd(y, q["nw"], residual=q["residual"][:, t])[0][:, None])
    out, _, want_conv, want_state = reference_layer({k: v.double() for k, v in p.items()}, None)
    near("out", torch.cat(outs, 1), out, FWD)
    near("state", state, want_state, FWD)
    assert torch.equal(conv_state.double().cpu(), want_conv)


def test_two_layers_in_one_graph_share_nothing():
    """Two captured graphs of the layer, replayed in turn: each call's workspace
    is its own."""
    qs, want = [], []
    for seed in (1, 2):
        p, _ = layer_inputs(1, 3000, 64, seed=seed)
        qs.append({k: v.to(DEV) for k, v in p.items()})
        want.append(run_layer(qs[-1], None))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run_layer(q, None))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(o[k], w[k]) for k in w)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_ssd_layer_sequence_and_steps_agree(io):
    """Convolution of x, B and C out of the projection's rows, the SSD scan, the
    gated norm: the sequence at once and token by token give the same, to the
    rounding of the activations between the operators (bf16: three roundings of
    2^-8 and the scan's 1e-2 bound)."""
    gen = torch.Generator().manual_seed(3)
    b, L, H, P, N, G, W = 2, 70, 4, 32, 16, 2, 4
    D, row = H * P, 2 * H * P + 2 * G * N
    r = lambda *s: torch.randn(*s, generator=gen).to(DEV)
    proj = r(b, L, row).to(io)
    dt = 0.05 + 0.05 * torch.rand(b, L, H, generator=gen).to(DEV)
    A, skip, nw = -1 - r(H).abs(), r(H), 1 + 0.2 * r(D)
    w, cb = 0.5 * r(D + 2 * G * N, W), 0.1 * r(D + 2 * G * N)
    cut = [0, D, D + G * N, D + 2 * G * N]

    def columns(t):
        z, xbc = t[..., :D], t[..., D:]
        return z, [xbc[..., lo:hi] for lo, hi in zip(cut, cut[1:])]

    z, parts = columns(proj)
    conv = [ssd.ssd_conv_fwd(t, w[lo:hi].contiguous(), bias=cb[lo:hi].contiguous())
            for t, lo, hi in zip(parts, cut, cut[1:])]
    x, B, C = (c[0] for c in conv)
    y, state = ssd.ssd_fwd(x.view(b, L, H, P), dt, A, B.view(b, L, G, N), C.view(b, L, G, N), skip, chunk_size=64)
    out, _ = ssd.ssd_norm_fwd(y.view(b, L, D), nw, z=z, ngroups=G)

    windows = [torch.zeros(b, W - 1, hi - lo, dtype=io, device=DEV) for lo, hi in zip(cut, cut[1:])]
    carried = torch.zeros(b, H, P, N, device=DEV)
    outs = []
    for t in range(L):
        zt, pt = columns(proj[:, t])
        xt, Bt, Ct = (ssd.ssd_conv_step(q, w[lo:hi].contiguous(), s, bias=cb[lo:hi].contiguous())
                      for q, s, lo, hi in zip(pt, windows, cut, cut[1:]))
        yt = ssd.ssd_decode_step(xt.view(b, H, P), dt[:, t].contiguous(), A, Bt.view(b, G, N), Ct.view(b, G, N), skip, carried)
        outs.append(ssd.ssd_norm_fwd(yt.view(b, D), nw, z=zt, ngroups=G)[0][:, None])
    tol = 1e-4 if io is torch.float32 else 1e-2 + 3 * 2.0 ** -8
    near("out", torch.cat(outs, 1), out.double().cpu(), tol)
    near("state", carried, state.double().cpu(), tol)
    for (_, f), s in zip(conv, windows):
        assert torch.equal(f, s)
