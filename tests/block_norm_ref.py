"""The block norm from its formulas in 64 bits, with error bounds of a 32-bit evaluation.

Every bound is ``K * 2^-24`` times a magnitude that is the formula evaluated on absolute
values (what cancellation can blow up a 32-bit rounding to), plus half a step of the output's
type. K counts the roundings on the way to a value: a tree sum of up to 16384 terms (14), the
reciprocal square root and its argument (8), the products and sums of the formula (at most 16
for each of two norms), so 64 covers a forward value and 128 a gradient, in which the
statistics enter twice. A sum over N rows adds at most N roundings of its terms."""
import torch

U = 2.0 ** -24


def act_of(name, g):
    if name == "sigmoid":
        a = torch.sigmoid(g)
        return a, a * (1 - a)
    if name == "tanh":
        a = torch.tanh(g)
        return a, 1 - a * a
    return g, torch.ones_like(g)


def stats_of(v, norm, eps):
    mean = v.mean(1, keepdim=True) if norm == "layer" else torch.zeros_like(v[:, :1])
    return mean, 1.0 / torch.sqrt(((v - mean) ** 2).mean(1, keepdim=True) + eps)


def expand_gate(gate, N):
    return gate.reshape(-1, gate.shape[-1]).double().repeat_interleave(N // (gate.numel() // gate.shape[-1]), 0)


def half_step(t, ref):
    """Half a step of type t at ref (and the smallest subnormal's half below its normal range)."""
    f = torch.finfo(t)
    return ref.abs() * (f.eps / 2) + f.tiny * f.eps


def forward(x, residual, gate, post_weight, post_bias, weight, bias, norm, eps, scale, act, off):
    """{name: (value, bound of the 32-bit error)} and what the backward pass needs."""
    N, D = x.shape
    d = lambda t: None if t is None else t.double()  # noqa: E731
    x, w1, b1, w2, b2 = d(x), d(post_weight), d(post_bias), d(weight), d(bias)
    s = {}
    u, mu = x, x.abs()
    if w1 is not None:
        m, r = stats_of(x, norm, eps)
        n, w = (x - m) * r, w1 + off
        u = n * w + (b1 if b1 is not None else 0)
        mu = ((x.abs() + x.abs().mean(1, keepdim=True)) * r + n.abs()) * w.abs() + (b1.abs() if b1 is not None else 0)
        s.update(m1=m, r1=r, n1=n)
    a = torch.ones_like(x)
    da = torch.zeros_like(x)
    if gate is not None:
        a, da = act_of(act, expand_gate(gate, N))
    res = d(residual) if residual is not None else torch.zeros_like(x)
    h = res + scale * a * u
    mh = res.abs() + abs(scale) * a.abs() * mu
    out = {"h": (h, 64 * U * mh)}
    if w2 is not None:
        m, r = stats_of(h, norm, eps)
        n, w = (h - m) * r, w2 + off
        y = n * w + (b2 if b2 is not None else 0)
        # an error in h reaches y directly, through the mean and through the deviation
        my = ((mh + mh.mean(1, keepdim=True)) * r + n.abs() * (1 + (n.abs() * mh * r).mean(1, keepdim=True))) * w.abs()
        out["y"] = (y, 64 * U * (my + (b2.abs() if b2 is not None else 0)))
        s.update(m2=m, r2=r, n2=n)
    s.update(a=a, da=da, u=u)
    return out, s


def backward(x, h, gate, post_weight, post_bias, weight, bias, stats, dh, dy, norm, scale, act, off):
    """Gradients from the kernel's own h and statistics: {name: (value, bound)}."""
    N, D = x.shape
    d = lambda t: None if t is None else t.double()  # noqa: E731
    x, h, w1, b1, w2, st = d(x), d(h), d(post_weight), d(post_bias), d(weight), d(stats).T
    zero = torch.zeros_like(x)
    g = zero if dh is None else d(dh)
    mg = g.abs()
    layer = norm == "layer"
    out = {}

    def back(t, mt, n, mn, r):
        dot, mdot = (t * n).mean(1, keepdim=True), (mt * mn).mean(1, keepdim=True)
        v = t - n * dot - (t.mean(1, keepdim=True) if layer else 0)
        return r * v, r * (mt + mn * mdot + (mt.mean(1, keepdim=True) if layer else 0))

    if w2 is not None:
        t = zero if dy is None else d(dy)
        m2, r2 = st[2][:, None], st[3][:, None]
        n, mn = (h - m2) * r2, (h.abs() + m2.abs()) * r2
        out["dweight"] = ((t * n).sum(0), (N + 128) * U * (t.abs() * mn).sum(0))
        out["dbias"] = (t.sum(0), (N + 128) * U * t.abs().sum(0))
        w = w2 + off
        v, mv = back(t * w, (t * w).abs(), n, mn, r2)
        g, mg = g + v, mg + mv
    out["dresidual"] = (g, 128 * U * mg)
    if w1 is not None:
        m1, r1 = st[0][:, None], st[1][:, None]
        n1, mn1 = (x - m1) * r1, (x.abs() + m1.abs()) * r1
        w = w1 + off
        u = n1 * w + (b1 if b1 is not None else 0)
        mu = mn1 * w.abs() + (b1.abs() if b1 is not None else 0)
    else:
        u, mu = x, x.abs()
    a, da = torch.ones_like(x), zero
    if gate is not None:
        a, da = act_of(act, expand_gate(gate, N))
        rows = gate.numel() // D
        e, me = scale * g * u * da, abs(scale) * mg * mu * (da.abs() + 2 * (a.abs() if act != "none" else 0))
        out["dgate"] = (e.view(rows, -1, D).sum(1), (N // rows + 128) * U * me.view(rows, -1, D).sum(1))
    g, mg = scale * g * a, abs(scale) * mg * a.abs()
    if w1 is not None:
        out["dpost_weight"] = ((g * n1).sum(0), (N + 128) * U * (mg * mn1).sum(0))
        out["dpost_bias"] = (g.sum(0), (N + 128) * U * mg.sum(0))
        g, mg = back(g * w, mg * w.abs(), n1, mn1, r1)
    out["dx"] = (g, 128 * U * mg)
    return out


def close(got, ref, bound, name):
    allowed = bound + half_step(got.dtype, ref)
    off = (got.double() - ref).abs()
    bad = ~(off <= allowed)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} values off, worst {float((off / allowed).max()):.3g} "
                           f"times the bound")
