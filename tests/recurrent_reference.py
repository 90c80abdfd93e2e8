"""Plain 64-bit forms of the gated linear recurrence, with bounds on the rounding errors of 32-bit ones.

The recurrence runs step by step from its definition, each sequence by itself, and so do its gradients.
The bounds follow the arithmetic (u = 2^-24, half a step of fp32 relative to a value): a term b[s] reaches h[t]
through t - s decays, each off by at most 2 u (its own rounding and the polynomial's error, 1.4e-8 of
something no larger), and through at most t - s + 24 roundings of products and sums, whatever way they are
grouped (24: two for the weight's square root and product, the rest where a lane's, a tile's and a
group's parts are joined).  So |error| <= sum over s of 3 u (t - s + 24) |decays b[s]|, which the recurrences
M[t] = a M[t-1] + |b[t]| and K[t] = a (K[t-1] + M[t-1]) give as 3 u (K + 24 M).  Gradients are products of such
values.  A weight sqrt(1 - a^2), from 1 - a good to 2 u, is good to 4 u, a reciprocal of it to 6 u; what has more
roundings than that is counted with 24 u.  Outputs of 16 bits are rounded once more: half a spacing.
"""
import numpy as np
import torch

from layer_reference import DT, half_spacing  # noqa: F401

U = 2.0 ** -24


def spans_of(B, L, lengths):
    """(row, first step, end) of every sequence."""
    if lengths is None:
        return [(b, 0, L) for b in range(B)]
    out, at = [], 0
    for n in lengths:
        out.append((0, at, at + n))
        at += n
    return out


def walk(a, b):
    """h[t] = a[t] h[t-1] + b[t] from 0, with M and K of the module's text; first dimension: steps."""
    h = m = k = torch.zeros_like(b[0])
    hs, ms, ks = [], [], []
    for t in range(a.shape[0]):
        k = a[t] * (k + m)
        m = a[t] * m + b[t].abs()
        h = a[t] * h + b[t]
        hs.append(h)
        ms.append(m)
        ks.append(k)
    return torch.stack(hs), torch.stack(ms), torch.stack(ks)


def linrec(x, g, lengths=None, h0=None, normalize=False, dout=None, dht=None):
    """Results and bounds: {name: (value, bound)} of out, ht and, with dout, dx, dg, dh0."""
    B, L, C = x.shape
    x, g = x.double(), g.double()
    spans = spans_of(B, L, lengths)
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    shapes = {"out": (B, L, C), "ht": (len(spans), C)}
    if dout is not None:
        shapes.update({"dx": (B, L, C), "dg": (B, L, C), "dh0": (len(spans), C)})
    v, e = ({n: zero(*s) for n, s in shapes.items()} for _ in range(2))
    for s, (r, t0, t1) in enumerate(spans):
        start = zero(C) if h0 is None else h0[s].double()
        if t0 == t1:
            v["ht"][s] = start
            if dout is not None and dht is not None:
                v["dh0"][s] = dht[s].double()
            continue
        a, y = g[r, t0:t1].exp(), -torch.expm1(g[r, t0:t1])
        w = torch.sqrt((y * (2 - y)).clamp(min=0)) if normalize else torch.ones_like(a)
        xs = x[r, t0:t1]
        b = w * xs
        # the state before the first step as a step of its own, so that its bound is counted the same way
        h, m, k = walk(torch.cat([torch.ones_like(a[:1]), a]), torch.cat([start[None], b]))
        bound = 3 * U * (k + 24 * m)
        v["out"][r, t0:t1], e["out"][r, t0:t1] = h[1:], bound[1:]
        v["ht"][s], e["ht"][s] = h[-1], bound[-1]
        if dout is None:
            continue
        d = dout[r, t0:t1].double().clone()
        if dht is not None:
            d[-1] += dht[s].double()
        D, dm, dk = (q.flip(0) for q in walk(torch.cat([a[1:], torch.ones_like(a[:1])]).flip(0), d.flip(0)))
        db = 3 * U * (dk + 24 * dm)
        v["dx"][r, t0:t1], e["dx"][r, t0:t1] = w * D, w * (db + 24 * U * dm)
        hp, mp, bp = h[:-1], m[:-1], bound[:-1]
        v["dg"][r, t0:t1] = a * hp * D
        e["dg"][r, t0:t1] = a * (bp * dm + mp * db + bp * db + 24 * U * mp * dm)
        if normalize:
            q = torch.where(w > 0, a * a / torch.where(w > 0, w, 1.0), 0.0) * xs.abs()
            v["dg"][r, t0:t1] -= q * xs.sign() * D
            e["dg"][r, t0:t1] += q * (db + 24 * U * dm)
        v["dh0"][s], e["dh0"][s] = a[0] * D[0], a[0] * (db[0] + 24 * U * dm[0])
    return {n: (v[n], e[n]) for n in v}


def assert_within(name, got, want, what="", least=1e-37):
    """Every element of `got` within its bound of the 64-bit value, and within half a spacing of its type more;
    fp32 results below `least` may be flushed to zero."""
    value, bound = want
    x = got.detach().cpu().double()
    assert x.shape == value.shape, (what, name, x.shape, value.shape)
    over = (x - value).abs() - bound - half_spacing(got.dtype, value.abs() + bound) - least
    assert bool(torch.isfinite(x).all()), f"{what} {name}: not finite"
    if over.numel():
        i = int(over.argmax())
        assert float(over.max()) <= 0, (f"{what} {name}: element {i} of {tuple(x.shape)} is {float(x.flatten()[i]):.9g}, not "
                                        f"{float(value.flatten()[i]):.9g} (bound {float(bound.flatten()[i]):.3g})")


def inputs(B, L, C, dtype="f32", gate="f32", seed=0, seqs=None, states=True, slow=0.999, pad=0):
    """x as it leaves the conv, log decays between a slow channel's and -8 a step (CPU)."""
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = rand(B, L, C + pad).to(DT[dtype])[..., :C]
    base = torch.log10(torch.tensor(1 - slow))
    size = 10 ** (base + (0.9 - base) * torch.rand(C, generator=gen) ** 2)
    g = (-size * torch.rand(B, L, C, generator=gen)).to(DT[gate])
    n = B if seqs is None else seqs
    return x, g, rand(n, C) if states else None


# ---- group norm -----------------------------------------------------------------------------------
#
# The bounds follow the formulas a value at a time: a sum of n terms made by threads is off by at most k u of the sum of
# its terms' sizes, k the roundings of one thread's chain (at most 32 elements, or a 1024th of a wider group) and of the joins (at
# most 16); sigmoid and exponential are off by the argument's rounding, 1.5 u of its size, and a few units, and
# a sigmoid below fp32's smallest normal number, 2^-126, is 0: the value v sigmoid(v) is then off by 2^-126 |v|.

def act(v, silu):
    """act, act' and bounds on their rounding errors, for v exact."""
    if not silu:
        return v, torch.ones_like(v), 0 * v, 0 * v
    s = 1 / (1 + torch.exp(-v))
    eps = (1.5 * v.abs() + 10) * U
    none = 2.0 ** -126
    return v * s, s * (1 + v * (1 - s)), eps * (v * s).abs() + none * v.abs(), eps * (1 + v.abs()) + none * (1 + v.abs())


def group_norm(x, groups, w, b, z, silu, eps, dout=None):
    """{name: (value, bound)} of out, mean, rstd and, with dout, dx, dw, db, dz; x [rows, C]."""
    rows, C = x.shape
    x = x.double().unflatten(1, (groups, -1))
    per = lambda t, other: (torch.full((C,), other, dtype=torch.float64) if t is None else t.double()).view(1, groups, -1)  # noqa: E731
    w, b = per(w, 1.0), per(b, 0.0)
    avg = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    k = (48 + x.shape[-1] / 1024) * U
    mu, emu = avg(x), k * avg(x.abs())
    d = x - mu
    ed = emu + U * d.abs()
    var = avg(d * d)
    rs = (var + eps) ** -0.5
    rel = 0.5 * (avg(2 * d.abs() * ed + ed * ed) + k * var) / (var + eps) + 4 * U
    n = d * rs
    en = rs * ed + n.abs() * (rel + U)
    y = n * w + b
    ey = w.abs() * en + 3 * U * ((n * w).abs() + b.abs())
    if z is None:
        v, slope, ev, es = act(y, silu)
        out, eo = v, 1.1 * ey + ev
    else:
        z = z.double().unflatten(1, (groups, -1))
        v, slope, ev, es = act(z, silu)
        out, eo = y * v, v.abs() * ey + y.abs() * ev + ey * ev + U * (y * v).abs()
    flat = lambda t: t.flatten(1)  # noqa: E731
    ans = {"out": (flat(out), flat(eo)), "mean": (mu[..., 0], emu[..., 0]), "rstd": (rs[..., 0], (rs * rel)[..., 0])}
    if dout is None:
        return ans
    g = dout.double().unflatten(1, (groups, -1))
    if z is None:
        dy, edy = g * slope, g.abs() * ((0.5 if silu else 0) * ey + es + U * slope.abs())
    else:
        dy, edy = g * v, g.abs() * (ev + U * v.abs())
        ans["dz"] = (flat(g * y * slope), flat(g.abs() * (slope.abs() * ey + (y.abs() + ey) * es) + 3 * U * (g * y * slope).abs()))
    e = dy * w
    ee = w.abs() * edy + U * e.abs()
    m1, em1 = avg(e), avg(ee) + k * avg(e.abs())
    m2, em2 = avg(e * n), avg(ee * n.abs() + e.abs() * en + ee * en) + k * avg((e * n).abs())
    inner = e - m1 - n * m2
    einner = ee + em1 + n.abs() * em2 + en * (m2.abs() + em2) + 4 * U * (e.abs() + m1.abs() + (n * m2).abs())
    ans["dx"] = (flat(rs * inner), flat(rs * (einner + (rel + 2 * U) * inner.abs()) * (1 + rel)))
    chain = min(rows, 1200) * U
    ans["dw"] = ((dy * n).sum(0).flatten(), (edy * n.abs() + dy.abs() * en + edy * en + chain * (dy * n).abs()).sum(0).flatten())
    ans["db"] = (dy.sum(0).flatten(), (edy + chain * dy.abs()).sum(0).flatten())
    return ans


# ---- rotary positions -----------------------------------------------------------------------------
#
# The kernel's angle p f is rounded three times in 64 bits, 3 2^-53 |p f|, and its remainder and the two series a few
# times in 32: cosines and sines are off by at most 3 2^-53 |p f| + 3 u, times the scale, and a pair's products and
# their sum are rounded once each.  The angle itself is made in 80 bits here.

def rotary(x, positions, freq, interleaved=False, scale=1.0, inverse=False):
    """(value, bound) of x [B, L, H, D] turned."""
    angle = positions.numpy().astype(np.longdouble)[..., None] * freq.cpu().numpy().astype(np.longdouble)
    cos, sin = (torch.from_numpy(f(angle).astype(np.float64))[:, :, None] * scale for f in (np.cos, np.sin))
    sin = -sin if inverse else sin
    off = (torch.from_numpy(np.abs(angle).astype(np.float64))[:, :, None] * 3 * 2.0 ** -53 + 3 * U) * abs(scale) + 2 * U * abs(scale)
    half = freq.numel()
    x = x.double()
    y, bound = x.clone(), torch.zeros_like(x)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    u, v = x[..., a], x[..., b]
    y[..., a], y[..., b] = u * cos - v * sin, v * cos + u * sin
    bound[..., a] = bound[..., b] = (u.abs() + v.abs()) * off + 2 * U * abs(scale) * (u.abs() + v.abs())
    return y, bound
