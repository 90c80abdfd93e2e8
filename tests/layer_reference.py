"""Plain 64-bit forms of the layer's operators, and the tolerances their tests use.

The delta rule runs step by step from its definition, one sequence and head group at a time, with
torch's autograd for the gradients; layer norm from its formula; the tables by a loop.

Tolerances, from the arithmetic (u = 2^-24, the rounding of fp32):
  * an fp32 result of the delta rule is a chain of at most four matrix products over 64 to 128 terms
    of fp32 values held in bf16 planes.  A product drops plane products below 2^-22 of a term and
    adds up at most 128 rounded terms; rounding errors of random sign give about sqrt(128) u = 11 u
    a product, so the chain about 2^-19 of the result in the 2-norm (32 u), and twice that again for
    gradients, which pass through two chains.
  * a 16-bit result is computed from products that drop terms below 2^-16, 2^-15 more, and rounded
    once: within half a spacing of the type, 2^-8 of an element in bf16 and 2^-11 in fp16, there at
    least 2^-25.  What is held to the limit is the error beyond that half spacing.
  * element by element, the limit is relative to the largest result in the place of the element, times
    8 for the spread between the largest error and its mean square over a tensor.
"""
import numpy as np
import torch

import causal_depthwise_conv1d_amd as ccv  # noqa: F401  (tests import it from here too)

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_spacing(dtype, y):
    """Largest error of rounding the 64-bit values y to dtype."""
    if dtype == torch.float16:
        return (2.0 ** -11 * y.abs()).clamp(min=2.0 ** -25)
    return (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) * y.abs()



def silu(x):
    return x / (1 + torch.exp(-x))


def delta_inputs(B, L, Hk, Hv, Dk, Dv, dtype="f32", gdt="f32", bdt="f32", seed=0, seqs=None, states=True, decay=0.3):
    """Inputs as they leave the conv: unit queries and keys, log decays, write strengths (CPU)."""
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    unit = lambda x: x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    q, k = (unit(silu(rand(B, L, Hk, Dk))).to(DT[dtype]) for _ in range(2))
    v = silu(rand(B, L, Hv, Dv)).to(DT[dtype])
    gate = (-decay * torch.rand(B, L, Hv, generator=g)).to(DT[gdt])
    beta = torch.rand(B, L, Hv, generator=g).to(DT[bdt])
    n = B if seqs is None else seqs
    h0 = rand(n, Hv, Dk, Dv) * 0.2 if states else None
    return q, k, v, gate, beta, h0


def cu_of(lengths):
    return torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32)


def delta_one(q, k, v, g, beta, scale, S):
    """One sequence: q, k [L, Hk, Dk], v [L, Hv, Dv], gates [L, Hv], S [Hv, Dk, Dv], all 64-bit."""
    group = v.shape[1] // q.shape[1]
    out = []
    for t in range(q.shape[0]):
        qt, kt = (x[t].repeat_interleave(group, 0)[..., None] for x in (q, k))
        S = torch.exp(g[t])[:, None, None] * S
        u = beta[t][:, None] * (v[t] - (S * kt).sum(1))
        S = S + kt * u[:, None]
        out.append(scale * (S * qt).sum(1))
    return (torch.stack(out) if out else v), S


def delta_reference(q, k, v, g, beta, scale=None, lengths=None, h0=None):
    """(out, final states) in 64 bits; differentiable.  Steps past the lengths' sum give zeros."""
    q, k, v, g, beta = (x if x.dtype == torch.float64 else x.double() for x in (q, k, v, g, beta))
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    B, L, Hv = g.shape
    zero = torch.zeros(Hv, q.shape[-1], v.shape[-1], dtype=torch.float64)
    spans = [(b, 0, L) for b in range(B)] if lengths is None else [
        (0, int(e) - int(n), int(e)) for n, e in zip(lengths, np.cumsum(lengths))]
    outs, states = [], []
    for s, (b, t0, t1) in enumerate(spans):
        S = zero if h0 is None else h0[s].double()
        o, S = delta_one(q[b, t0:t1], k[b, t0:t1], v[b, t0:t1], g[b, t0:t1], beta[b, t0:t1], scale, S)
        outs.append(o)
        states.append(S)
    if lengths is None:
        out = torch.stack(outs) if outs else v
    else:
        rest = L - sum(lengths)
        out = torch.cat(outs + [torch.zeros(rest, *v.shape[2:], dtype=torch.float64)])[None]
    return out, (torch.stack(states) if states else torch.zeros(0, *zero.shape, dtype=torch.float64))


def delta_gradients(q, k, v, g, beta, dout, scale=None, lengths=None, h0=None, dht=None):
    """Reference outputs and gradients: dict of out, ht, dq, dk, dv, dg, dbeta, dh0."""
    leaves = [x.double().requires_grad_() for x in (q, k, v, g, beta)]
    h = None if h0 is None else h0.double().requires_grad_()
    out, ht = delta_reference(*leaves, scale, lengths, h)
    loss = (out * dout.double()).sum()
    if dht is not None:
        loss = loss + (ht * dht.double()).sum()
    wrt = leaves + ([h] if h is not None else [])
    grads = torch.autograd.grad(loss, wrt, allow_unused=True)
    names = ["dq", "dk", "dv", "dg", "dbeta", "dh0"]
    res = {"out": out.detach(), "ht": ht.detach()}
    for n, w, x in zip(names, wrt, grads):
        res[n] = torch.zeros_like(w) if x is None else x
    return res


def assert_near(name, got, ref, chains=1, what=""):
    """`got` (any device) within the tolerances above of the 64-bit `ref`; chains: 1 forward, 2 gradients."""
    x, y = got.detach().cpu().double(), ref.detach().double()
    assert x.shape == y.shape, (name, x.shape, y.shape)
    assert torch.equal(torch.isfinite(x), torch.isfinite(y)), (what, name, "finite in other places")
    ok = torch.isfinite(y)
    x, y = x[ok], y[ok]
    if not y.numel():
        return
    wide = got.dtype == torch.float32
    eps = chains * 2.0 ** -19 + (0.0 if wide else 2.0 ** -15)
    d = (x - y).abs() if wide else ((x - y).abs() - half_spacing(got.dtype, y)).clamp(min=0)
    norm, big, err, worst = float(y.norm()), float(y.abs().max()), float(d.norm()), float(d.max())
    assert err <= eps * norm, f"{what} {name}: 2-norm error {err:.3g} of {norm:.3g} ({err / max(norm, 1e-300):.3g}, allowed {eps:.3g})"
    assert worst <= 8 * eps * big, f"{what} {name}: an element is {worst:.3g} off (largest value {big:.3g})"


def norm_reference(x, weight, bias, eps):
    x = x.double()
    d = x - x.mean(-1, keepdim=True)
    n = d / torch.sqrt(d.square().mean(-1, keepdim=True) + eps)
    out = n if weight is None else n * weight.double()
    return out if bias is None else out + bias.double()


def tables_reference(lengths, total):
    cu, seq, pos = [0], np.full(total, -1, np.int32), np.zeros(total, np.int32)
    for s, n in enumerate(lengths):
        e = min(cu[-1] + max(int(n), 0), total)
        seq[cu[-1]:e] = s
        pos[cu[-1]:e] = np.arange(e - cu[-1])
        cu.append(e)
    return np.array(cu, np.int32), seq, pos
