"""fp64 definitions of the layer operators (gated linear recurrence, causal
depthwise convolution, root-mean-square norm), token by token, with a bound on
the rounding error of an fp32 evaluation beside every result.

A bound counts roundings: U = 2^-24 is half a step of fp32 relative to the
value, HALF[io] half a step of an output's type.  The device's exp2, log2, rcp
and sqrt are taken as 2 U, and exp2's argument carries its own rounding, so
exp(x) is (2 + 2 |x|) U.  A fused or an ordinary multiply-add is one U of its
result.  Every returned value is a pair (result, bound)."""
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
TINY = 1e-30        # results below fp32's range


def rounded(pair, io):
    """The bound of a result stored in the io type."""
    v, e = pair
    return v, e + HALF[io] * (v.abs() + e) + TINY


def sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def silu(z):
    """z / (1 + exp(-z)): exp (2 + 2 |z|) U, the sum, rcp and product 4 U."""
    v = z * sigmoid(z)
    return v, (6 + 2 * z.abs()) * U * v.abs()


def dsilu(z):
    """s (1 + z (1 - s)): s is (5 + 2 |z|) U; 1 - s is off by that times s plus
    one rounding, all against s (1 + |z|)."""
    s = sigmoid(z)
    return s * (1 + z * (1 - s)), (16 + 4 * z.abs()) * U * s * (1 + z.abs())


def starts(seq_idx, L, b):
    r = torch.zeros(b, L, dtype=torch.bool)
    if seq_idx is not None:
        r[:, 1:] = seq_idx[:, 1:] != seq_idx[:, :-1]
    return r


class Glr:
    """Forward quantities of h_t = r_t a_t h_{t-1} + k_t x_t, with bounds:

    s = softplus(v): relative (8 + 2 |v|) U (v's own rounding moves s by at
    most |v| U relative, exp the same, log and sums the rest).
    la = A s one more.  a = exp(la): |la| times that plus 3 U.
    1 - a^2: its relative sensitivity to la's relative error is at most 1; the
    series and the select point add 18 U at most; the root halves.
    """

    def __init__(self, x, g, A, bias, z, seq_idx, init, normalize):
        self.x, self.z, self.A = x, z, A
        b, L, D = x.shape
        v = g if bias is None else g + bias
        self.sig = sigmoid(v)
        self.s = torch.logaddexp(v, torch.zeros_like(v))
        es = (8 + 2 * v.abs()) * U                       # relative
        self.es = es
        la = A * self.s
        self.a = la.exp()
        self.ea = (la.abs() * (es + U) + 3 * U)          # relative
        if normalize:
            k2 = -torch.special.expm1(2 * la)
            self.k = k2.sqrt()
            self.ek = (es + U + 18 * U) / 2 + 2 * U      # relative
        else:
            self.k = torch.ones_like(self.a)
            self.ek = torch.zeros_like(self.a)
        self.normalize = normalize
        self.cut = starts(seq_idx, L, b)[..., None].expand(b, L, D)
        self.p = torch.where(self.cut, torch.zeros_like(self.a), self.a)
        u = self.k * x
        h = x.new_zeros(b, D) if init is None else init
        big, err = h.abs(), torch.zeros_like(h)
        self.h0 = h
        H, E = [], []
        for t in range(L):
            # the decay's error acts on what is carried; composing segments
            # rounds each product and each sum once more (3 U)
            c = self.cut[:, t]
            carried = torch.where(c, torch.zeros_like(h), self.p[:, t] * h)
            mag = torch.where(c, torch.zeros_like(h), self.p[:, t] * big)
            err = torch.where(c, torch.zeros_like(h), self.p[:, t] * err + (self.ea[:, t] + 3 * U) * mag)
            h = carried + u[:, t]
            big = mag + u[:, t].abs()
            err = err + (self.ek[:, t] + U) * u[:, t].abs() + 2 * U * big
            H.append(h)
            E.append(err)
        self.h, self.eh = torch.stack(H, 1), torch.stack(E, 1)

    def outputs(self):
        final = (self.h[:, -1], self.eh[:, -1] + TINY)
        if self.z is None:
            return (self.h, self.eh + TINY), final
        g, eg = silu(self.z)
        y = self.h * g
        return (y, self.eh * g.abs() + self.h.abs() * eg + U * y.abs() + TINY), final

    def backward(self, dy, dfinal):
        x, z, A, k, p = self.x, self.z, self.A, self.k, self.p
        b, L, D = x.shape
        if z is None:
            e, ee = dy, torch.zeros_like(dy)
        else:
            g, eg = silu(z)
            e, ee = dy * g, dy.abs() * (eg + 2 * U * g.abs())
        c = x.new_zeros(b, D) if dfinal is None else dfinal
        bigc, errc = c.abs(), torch.zeros_like(c)
        G, EG, C, EC, MC = [None] * L, [None] * L, [None] * L, [None] * L, [None] * L
        for t in range(L - 1, -1, -1):
            gt = e[:, t] + c
            big = e[:, t].abs() + bigc
            G[t], EG[t] = gt, ee[:, t] + errc + 2 * U * big
            cut = self.cut[:, t]
            zero = torch.zeros_like(gt)
            c = torch.where(cut, zero, p[:, t] * gt)
            bigc = torch.where(cut, zero, p[:, t] * big)
            errc = torch.where(cut, zero, p[:, t] * EG[t] + (self.ea[:, t] + 4 * U) * bigc)
            C[t], EC[t], MC[t] = c, errc, bigc
        G, EG, C, EC = (torch.stack(q, 1) for q in (G, EG, C, EC))
        hp = torch.cat([self.h0[:, None], self.h[:, :-1]], 1)
        ehp = torch.cat([torch.zeros_like(self.h0[:, None]), self.eh[:, :-1]], 1)
        hp = torch.where(self.cut, torch.zeros_like(hp), hp)
        dx = k * G
        edx = k * EG + (self.ek + U) * dx.abs()
        dla = C * hp
        edla = C.abs() * ehp + EC * hp.abs() + 2 * U * dla.abs()
        if self.normalize:
            dk = self.a.square() / k
            term = G * x * dk
            dla = dla - term
            # a^2 twice a's, 1/k and the products 8 U
            edla = edla + EG * (x * dk).abs() + (2 * self.ea + self.ek + 8 * U) * term.abs()
        dg = A * dla * self.sig
        v_err = 2 * self.es                               # of the sigmoid, relative
        edg = (A * self.sig).abs() * edla + (v_err + 3 * U) * dg.abs()
        dA = self.s * dla
        edA = self.s * edla + (self.es + U) * dA.abs()
        # sums over a segment, the segments, the parts: under 128 additions in
        # a chain for the lengths tested
        total = lambda q, eq: (q.sum((0, 1)), eq.sum((0, 1)) + 128 * U * q.abs().sum((0, 1)) + TINY)
        dz = None
        if z is not None:
            d, ed = dsilu(z)
            dz = dy * self.h * d
            dz = (dz, dy.abs() * (self.eh * d.abs() + self.h.abs() * ed) + 3 * U * dz.abs())
        return {"dx": (dx, edx), "dg": (dg, edg), "dz": dz, "dA": total(dA, edA), "dbias": total(dg, edg),
                "dinit": (C[:, 0], EC[:, 0] + TINY)}


def conv(x, weight, bias, seq_idx, init, silu_on, dy=None, dfinal=None):
    """(y, final) or, with dy, the gradients; each a (result, bound)."""
    b, L, D = x.shape
    W = weight.shape[1]
    before = x.new_zeros(b, W - 1, D) if init is None else init
    full = torch.cat([before, x], 1)
    cut = starts(seq_idx, L, b)
    begin = torch.zeros(b, L, dtype=torch.int64)      # first visible position of `full`
    for i in range(b):
        for t in range(1, L):
            begin[i, t] = t + W - 1 if cut[i, t] else begin[i, t - 1]
    p = x.new_zeros(b, L, D) if bias is None else bias.expand(b, L, D).clone()
    mag = p.abs()
    live = []
    for i in range(W):
        ok = (torch.arange(L) + i >= begin)[..., None]
        live.append(ok)
        term = torch.where(ok, weight[:, i] * full[:, i:i + L], torch.zeros(()).double())
        p = p + term
        mag = mag + term.abs()
    ep = (W + 1) * U * mag
    keep = (torch.arange(L, L + W - 1) >= begin[:, -1:])[..., None]
    final = torch.where(keep, full[:, L:], torch.zeros(()).double())
    if dy is None:
        if not silu_on:
            return (p, ep + TINY), final
        y, ey = silu(p)
        return (y, 1.1 * ep + ey + TINY), final      # |silu'| <= 1.1
    ds, eds = dy, torch.zeros_like(dy)
    if silu_on:
        d, ed = dsilu(p)
        ds = dy * d
        eds = dy.abs() * (ed + 0.5 * ep + 2 * U * d.abs())   # |silu''| <= 0.5
    dfull, edfull = torch.zeros_like(full), torch.zeros_like(full)
    dw, edw = torch.empty_like(weight), torch.empty_like(weight)
    zero = torch.zeros(()).double()
    for i in range(W):
        t = torch.where(live[i], ds, zero)
        et = torch.where(live[i], eds, zero)
        dfull[:, i:i + L] += weight[:, i] * t
        edfull[:, i:i + L] += weight[:, i].abs() * (et + (W + 2) * U * t.abs())
        xi = torch.where(live[i], full[:, i:i + L], zero)
        dw[:, i] = (t * xi).sum((0, 1))
        # a run's 64 tokens, four waves, the parts: under 128 additions
        edw[:, i] = (et * xi.abs() + 128 * U * (t * xi).abs()).sum((0, 1))
    if dfinal is not None:
        df = torch.where(keep, dfinal, zero)
        dfull[:, L:] += df
        edfull[:, L:] += 2 * U * (df.abs() + dfull[:, L:].abs())
    return {"dx": (dfull[:, W - 1:], edfull[:, W - 1:]), "dweight": (dw, edw + TINY),
            "dbias": (ds.sum((0, 1)), (eds + 128 * U * ds.abs()).sum((0, 1)) + TINY),
            "dinit": (dfull[:, :W - 1], edfull[:, :W - 1] + TINY)}


def norm_input(x, residual, z, io):
    """v and its relative bound; with a residual the stream, exactly."""
    if residual is not None:
        # in fp32 as the kernel adds (one rounding of the exact sum), then the
        # io type: for bf16 the fp32 sum decides the rounding
        return (x.float() + residual.float()).to(io).double(), 0.0
    if z is not None:
        g, eg = silu(z)
        return x * g, (7 + 2 * z.abs()) * U
    return x, 0.0


def norm(v, ev, weight, eps, ngroups):
    """y = v rstd w: the sum of squares 2 ev + 48 additions of positive terms,
    the root halves it, and six more roundings."""
    r, c = v.shape
    g = v.reshape(r, ngroups, -1)
    rms = (g.square().mean(-1, keepdim=True) + eps).sqrt()
    n = (g / rms).reshape(r, c)
    worst = ev if isinstance(ev, float) else ev.reshape(r, ngroups, -1).amax(-1, keepdim=True).expand_as(g).reshape(r, c)
    y = n if weight is None else n * weight
    return y, (ev + worst + 30 * U) * y.abs() + TINY, n, rms.expand_as(g).reshape(r, c), worst


def norm_backward(x, z, weight, dy, dresidual, eps, ngroups):
    v, ev = norm_input(x, None, z, None)
    r, c = x.shape
    _, _, n, rms, worst = norm(v, ev, weight, eps, ngroups)
    wdy = dy if weight is None else dy * weight
    group = lambda q: q.reshape(r, ngroups, -1)
    mean = lambda q: group(q).mean(-1, keepdim=True).expand(r, ngroups, c // ngroups).reshape(r, c)
    dot, dotmag = mean(wdy * n), mean((wdy * n).abs())
    dv = (wdy - n * dot) / rms
    # every product under 60 roundings, v's error twice in each
    edv = (60 * U + 3 * worst + 2 * ev) * (wdy.abs() + n.abs() * dotmag) / rms
    if dresidual is not None:
        dv = dv + dresidual
        edv = edv + U * dv.abs()
    out = {"dz": None, "dx": (dv, edv)}
    if z is not None:
        g, eg = silu(z)
        d, ed = dsilu(z)
        out["dx"] = (dv * g, edv * g.abs() + dv.abs() * eg + U * (dv * g).abs())
        out["dz"] = (dv * x * d, x.abs() * (edv * d.abs() + dv.abs() * ed) + 3 * U * (dv * x * d).abs())
    # rows in a chain per part, parts: under 192 additions for the sizes tested
    t = dy * n
    out["dweight"] = (t.sum(0), ((ev + worst + 30 * U + 192 * U) * t.abs()).sum(0) + TINY)
    return out
