"""The operators between the layers run together, as a model uses them: 4-bit
projections around the convolution, the scan and the gated norm, block norms
between the layers; a prompt at once and token by token, training with
checkpoints, captured graphs, other streams and threads.

Tolerances: an fp32 chain of operators, relative to the largest value of the
tensor, 64 roundings of 2^-24 for each (each operator's own bound counts under 60
for values of order one) and 1e-4 for the SSD scan in fp32, its own bound."""
import threading

import pytest
import torch

import block_reference as ref
import layer_reference as lref
from layer_reference import U

import ssd_chunked_scan_amd as ssd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def near(name, got, want, tol):
    off = float((got.detach().double().cpu() - want.detach()).abs().max() / want.detach().abs().max())
    assert off <= tol, (name, off, tol)


class Model:
    """`layers` layers of width D: 4-bit projection into z | x | g, convolution,
    gated recurrence, 4-bit projection back, block norm."""

    def __init__(self, layers, D, inner, seed, io=torch.float32):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen)
        self.D, self.inner, self.io = D, inner, io
        self.layers = []
        for _ in range(layers):
            p = dict(w_in=r(3 * inner, D) / D ** 0.5, w_out=r(D, inner) / inner ** 0.5, conv=0.5 * r(inner, 4),
                     A=-1 - r(inner).abs(), post=1 + 0.1 * r(D), pre=1 + 0.1 * r(D), scale=0.5 + 0.1 * r(D))
            p = {k: v.to(DEV) for k, v in p.items()}
            p["w_in"], p["w_out"] = ssd.ssd_mx4_quant(p["w_in"]), ssd.ssd_mx4_quant(p["w_out"])
            self.layers.append(p)

    def states(self, b):
        return [dict(window=torch.zeros(b, 3, self.inner, dtype=self.io, device=DEV), state=torch.zeros(b, self.inner, device=DEV))
                for _ in self.layers]

    def prompt(self, h, stream, states):
        for p, s in zip(self.layers, states):
            z, x, g = ssd.ssd_mx4_linear(h, *p["w_in"]).split(self.inner, dim=-1)
            xc, s["window"] = ssd.ssd_conv_fwd(x, p["conv"], init_states=s["window"])
            y, s["state"] = ssd.ssd_glr_fwd(xc, g, p["A"], z=z, init_states=s["state"])
            o = ssd.ssd_mx4_linear(y, *p["w_out"])
            h, stream, _ = ssd.ssd_block_norm_fwd(o, stream, p["post"], p["pre"], scale=p["scale"])
        return h, stream

    def step(self, h, stream, states):
        for p, s in zip(self.layers, states):
            z, x, g = ssd.ssd_mx4_linear(h, *p["w_in"]).split(self.inner, dim=-1)
            xc = ssd.ssd_conv_step(x, p["conv"], s["window"])
            y = ssd.ssd_glr_step(xc, g, p["A"], s["state"], z=z)
            o = ssd.ssd_mx4_linear(y, *p["w_out"])
            h, stream, _ = ssd.ssd_block_norm_fwd(o, stream, p["post"], p["pre"], scale=p["scale"])
        return h, stream


def test_a_layer_against_its_definition():
    """One layer of the chain, operator by operator, in fp64 from the operator's
    own inputs: what is quantised between is quantised from the same bits."""
    m = Model(1, 200, 96, seed=1)
    p = m.layers[0]
    gen = torch.Generator().manual_seed(2)
    h, stream = (torch.randn(2, 90, 200, generator=gen).to(DEV) for _ in range(2))
    wide = ssd.ssd_mx4_linear(h, *p["w_in"])
    weights = lambda w, k: ref.unpack(w[0].cpu(), w[1].cpu())[:, :k]
    quantised = lambda t: ref.unpack(*ref.pack(*ref.mx4(t.double().cpu().reshape(-1, t.shape[-1]))))[:, :t.shape[-1]]
    near("projection", wide.reshape(-1, 288), quantised(h) @ weights(p["w_in"], 200).t(), 64 * U)
    z, x, g = wide.split(96, dim=-1)
    xc, _ = ssd.ssd_conv_fwd(x, p["conv"])
    y, _ = ssd.ssd_glr_fwd(xc, g, p["A"], z=z)
    c = lambda t: t.double().cpu()
    (conv, _), _ = lref.conv(c(x), c(p["conv"]), None, None, None, True)
    near("convolution", xc, conv, 64 * U)
    (want, _), _ = lref.Glr(c(xc), c(g), c(p["A"]), None, c(z), None, None, True).outputs()
    near("recurrence", y, want, 64 * U)
    o = ssd.ssd_mx4_linear(y, *p["w_out"])
    near("projection back", o.reshape(-1, 200), quantised(y) @ weights(p["w_out"], 96).t(), 64 * U)
    out, s, _ = ssd.ssd_block_norm_fwd(o, stream, p["post"], p["pre"], scale=p["scale"])
    want, _ = ref.block_stream(c(o), c(stream), None, c(p["post"]), c(p["scale"]), 1.0, 1e-5)
    near("stream", s, want, 64 * U)
    near("out", out, ref.block_out(c(s), c(p["pre"]), 1e-5)[0], 64 * U)


@pytest.mark.parametrize("b", [1, 5, 20])
def test_served_token_by_token(b):
    """A prompt, then tokens one by one, each step against the same layer's
    whole-sequence form of one token: the same operands reach the same kernels,
    or sums of the same products in another order."""
    m = Model(1, 160, 128, seed=3)
    gen = torch.Generator().manual_seed(4)
    h, stream = (torch.randn(b, 24, 160, generator=gen).to(DEV) for _ in range(2))
    steps, whole = m.states(b), m.states(b)
    m.prompt(h[:, :17].contiguous(), stream[:, :17].contiguous(), steps)
    m.prompt(h[:, :17].contiguous(), stream[:, :17].contiguous(), whole)
    for t in range(17, 24):
        out, s = m.step(h[:, t].contiguous(), stream[:, t].contiguous(), steps)
        out2, s2 = m.prompt(h[:, t:t + 1].contiguous(), stream[:, t:t + 1].contiguous(), whole)
        near("state", steps[0]["state"], whole[0]["state"].double().cpu(), 64 * U)
        assert torch.equal(steps[0]["window"], whole[0]["window"])
        # y is quantised from values that may differ in their last bits: a code
        # next to a border may fall on either side.  One code in the 128 of a
        # token is off by at most a step, 2 of 6: under 1/30 of the largest output.
        near("stream", s, s2[:, 0].double().cpu(), 1 / 30)
        near("out", out, out2[:, 0].double().cpu(), 1 / 30)


def test_training_seam_with_checkpoints():
    """Two seams in a row, forward keeping only checkpoints and backward from them:
    the gradient of the second is the first one's input, and both are those at
    the values that the checkpoints hold."""
    gen = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen).to(DEV)
    D = 384
    x1, x2, z1, z2, res = (r(3, 50, D) for _ in range(5))
    post, pre, scale = 1 + 0.1 * r(D), 1 + 0.1 * r(D), 0.5 + 0.1 * r(D)
    h1, s1, k1 = ssd.ssd_block_norm_fwd(x1, res, post, pre, z=z1, scale=scale, checkpoint=True)
    h2, s2, k2 = ssd.ssd_block_norm_fwd(x2 + h1, s1, post, pre, z=z2, scale=scale, checkpoint=True)
    dh2, ds2 = r(3, 50, D), r(3, 50, D)
    g2 = ssd.ssd_block_norm_bwd(None, None, post, pre, dh2, scale=scale, dresidual_out=ds2, checkpoint=k2)
    g1 = ssd.ssd_block_norm_bwd(None, None, post, pre, g2["dx"], scale=scale, dresidual_out=g2["dresidual"], checkpoint=k1)
    c = lambda t: t.double().cpu().reshape(-1, D)
    held = lambda k, n: c(k[n + "_q"].float()) * ref.per_column(k[n + "_scales"].double().cpu().reshape(-1, 3), D)
    w = [c(t)[0] for t in (post, pre, scale)]
    a2 = ref.block_backward(held(k2, "x"), held(k2, "residual"), held(k2, "z"), w[0], w[1], w[2], c(dh2), c(ds2), 1.0, 1e-5)
    a1 = ref.block_backward(held(k1, "x"), held(k1, "residual"), held(k1, "z"), w[0], w[1], w[2], a2["dx"][0],
                            a2["dresidual"][0], 1.0, 1e-5)
    for name in a1:
        want = a1[name][0]
        near(name, g1[name].reshape(want.shape), want, 2 * 64 * U)
    # and against the gradient without checkpoints: 8-bit numbers are off by
    # 2^-5 on average of 2^-4 at most, and a gradient is linear in them to first
    # order: its largest error stays under 1/4 of its largest value
    f2 = ssd.ssd_block_norm_bwd(x2 + h1, s2, post, pre, dh2, z=z2, scale=scale, dresidual_out=ds2)
    for name in ("dx", "dresidual", "dz", "dpost_weight", "dpre_weight", "dscale"):
        near(name, g2[name], f2[name].double().cpu(), 0.25)


def run_all(seed):
    """Every operator once, the ones with workspaces among them."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).to(DEV)
    x, res, z, w, xl = r(70, 640), r(70, 640), r(70, 640), r(300, 640), r(9, 640)
    post = torch.randn(640, generator=gen).to(DEV)
    wq, ws = ssd.ssd_mx4_quant(w)
    q, s = ssd.ssd_mx4_quant(x)

    def go():
        y, stream, kept = ssd.ssd_block_norm_fwd(x, res, post, post, z=z, scale=post, checkpoint=True)
        g = ssd.ssd_block_norm_bwd(x, stream, post, post, y, z=z, scale=post, dresidual_out=res)
        gk = ssd.ssd_block_norm_bwd(None, None, post, post, y, scale=post, checkpoint=kept)
        return [y, stream, *(k.view(torch.uint8) for k in kept.values()), *g.values(), *gk.values(), ssd.ssd_mx4_linear(y, wq, ws),
                ssd.ssd_mx4_linear(xl, wq, ws), ssd.ssd_mx4_matmul(q, s, wq, ws), ssd.ssd_mx4_dequant(*ssd.ssd_mx4_quant(y), 640)]

    return go


def test_two_graphs_in_turn_share_nothing():
    runs = [run_all(1), run_all(2)]
    want = [[t.clone() for t in f()] for f in runs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for f in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for _ in range(3):
        for g in (*graphs, graphs[0]):
            g.replay()
        runs[0]()          # eager work between the replays
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_streams_and_threads():
    """On a stream of the caller's, by torch's current stream and by its handle,
    and from two threads at once."""
    f = run_all(3)
    want = [t.clone() for t in f()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = f()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = torch.randn(100, 300, device=DEV)
    a, s, _ = ssd.ssd_block_norm_fwd(x, x)
    w = ssd.ssd_mx4_quant(x)
    y = ssd.ssd_mx4_linear(x, *w)
    torch.cuda.synchronize()
    b, *_ = ssd.ssd_block_norm_fwd(x, x, stream=side.cuda_stream)
    y2 = ssd.ssd_mx4_linear(x, *ssd.ssd_mx4_quant(x, stream=side.cuda_stream), stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(y, y2)
    results = [None, None]

    def work(i):
        torch.cuda.set_device(0)
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                results[i] = [t.clone() for t in f()]
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for r in results:
        assert all(torch.equal(a, b) for a, b in zip(r, want))


@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
def test_model_step_in_a_graph(io):
    """A decode step of two layers captured once and replayed for new tokens."""
    m = Model(2, 256, 192, seed=6, io=io)
    gen = torch.Generator().manual_seed(7)
    tokens = [torch.randn(4, 256, generator=gen).to(io).to(DEV) for _ in range(4)]
    eager = m.states(4)
    want = [[t.clone() for t in m.step(t, t, eager)] for t in tokens]
    states, h = m.states(4), torch.zeros(4, 256, dtype=io, device=DEV)
    m.step(h, h, m.states(4))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = m.step(h, h, states)
    for t, w in zip(tokens, want):
        h.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])
