"""The operators together, as the example layer with both recurrences uses them: a packed row's result and
gradients against the same layer run in 64 bits on the CPU, and decoding against prefill.

Tolerance: every intermediate is rounded to bf16 (2^-9 in mean square) in about thirteen places between x and the
result (norm, projection, conv, unit length, turn, recurrence, gate, group norm, output, sum and the
decays' and strengths' three), and once more on the way back: sqrt(26) 2^-9 = 1.0 % in the 2-norm for values,
taken twice for gradients, where the roundings pass through a second chain.  The gradients of the decays' rates
are sums over all steps of terms that cancel, which such a bound does not cover: they are checked in
fp32, where every tensor has to be within 1e-4, the delta rule's 2^-18 and the library products'
own rounding."""
import os
import sys

import pytest
import torch
import torch.nn.functional as F

import layer_reference as ref
import recurrent_reference as rec
from gpu_support import log

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def turn(x, positions, freq, scale):
    """The pairs (i, i + turned / 2) as complex numbers, for autograd in 64 bits."""
    n = freq.numel()
    pair = torch.complex(x[..., :n], x[..., n:2 * n]) * torch.polar(torch.full((), scale, dtype=torch.float64), positions[:, None, None] * freq)
    return torch.cat([pair.real, pair.imag, x[..., 2 * n:]], -1)


def linear(u, a, lengths):
    """The recurrence step by step, for autograd in 64 bits, and every sequence's last state."""
    out, ends = [], []
    w = torch.sqrt(-torch.expm1(2 * a))
    for r, t0, t1 in rec.spans_of(1, u.shape[1], lengths):
        h = torch.zeros_like(u[0, 0])
        for t in range(t0, t1):
            h = a[0, t].exp() * h + w[0, t] * u[0, t]
            out.append(h)
        ends.append(h)
    out += [torch.zeros_like(u[0, 0])] * (u.shape[1] - len(out))
    return torch.stack(out)[None], ends


def plain(layer, x, lengths):
    """The layer's formula in 64 bits on the CPU; parameters as leaves of the same names."""
    p = {n: t.detach().cpu().double().requires_grad_() for n, t in layer.named_parameters()}
    n = F.layer_norm(x, x.shape[-1:], p["norm_w"], p["norm_b"], 1e-5)
    g = -p["decay"] * F.softplus(F.linear(n, p["w_gate"]))
    a = -p["rate"] * F.softplus(F.linear(n, p["w_rate"]))
    beta = torch.sigmoid(F.linear(n, p["w_beta"]))
    c, z = F.linear(n, p["w_in"]), F.linear(n, p["w_z"])
    parts, at, positions = [], 0, torch.zeros(x.shape[1], dtype=torch.float64)
    for ln in lengths:
        if ln:
            t = F.pad(c[:, at:at + ln].transpose(1, 2), (layer.conv_w.shape[1] - 1, 0))
            parts.append(F.silu(F.conv1d(t, p["conv_w"][:, None], groups=c.shape[2])).transpose(1, 2))
            positions[at:at + ln] = torch.arange(ln)
        at += ln
    parts.append(torch.zeros(1, x.shape[1] - at, c.shape[2], dtype=torch.float64))
    q, k, v, u = torch.cat(parts, 1).split(layer.split, -1)
    q, k = (turn(F.normalize(t.unflatten(-1, (layer.hk, layer.d)), dim=-1), positions, layer.freq.cpu(), layer.scale) for t in (q, k))
    o, s = ref.delta_reference(q, k, v.unflatten(-1, (layer.hv, layer.d)), g, beta, None, lengths)
    h, ends = linear(u, a, lengths)
    y = torch.cat([o.flatten(-2), h], -1)
    y = F.group_norm(y[0], layer.groups, p["out_w"], p["out_b"], 1e-5)[None] * F.silu(z)
    return x + F.linear(y, p["w_out"]), s, ends, p


def rel(a, b):
    return float((a.detach().cpu().double() - b.detach()).norm() / b.detach().norm())


@pytest.mark.parametrize("lengths,rest", [([100], 0), ([70, 0, 1, 65], 5), ([3, 2, 64], 0), ([129, 0, 130], 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_packed_row(lengths, rest, dtype):
    from mixed_layer import MixedLayer
    torch.manual_seed(1)
    layer = MixedLayer(dtype=dtype)
    wide = dtype == torch.float32
    live = sum(lengths)
    T = live + rest
    x, dout = torch.randn(1, T, 256).to(dtype), torch.randn(1, T, 256).to(dtype)
    dout[:, live:] = 0                              # the steps that belong to no sequence train nothing
    xd = x.double().requires_grad_()
    want, _, _, p = plain(layer, xd, lengths)
    wg = torch.autograd.grad(want, [xd, *p.values()], dout.double())
    xg = x.cuda().requires_grad_()
    y = layer.train_row(xg, torch.tensor(lengths, dtype=torch.int32).cuda())
    gg = torch.autograd.grad(y, [xg, *layer.parameters()], dout.cuda())
    log(f"  layer {lengths} out {rel(y[:, :live], want[:, :live]):.2e}")
    assert rel(y[:, :live], want[:, :live]) < (1e-4 if wide else 1e-2)
    for name, a, b in zip(["x", *p], gg, wg):
        log(f"    d{name} {rel(a, b):.2e}")
        assert wide or name in ("decay", "rate") or rel(a, b) < 2e-2, name
        assert not wide or rel(a, b) < 1e-4, name


def test_decode_continues_prefill():
    from mixed_layer import MixedLayer
    torch.manual_seed(2)
    layer = MixedLayer(dtype=torch.float32)
    lengths, more = [65, 1, 0, 30], 5
    full = [n + more for n in lengths]
    rows = [torch.randn(n, 256) for n in full]
    want, s, ends_of, _ = plain(layer, torch.cat(rows)[None].double(), full)
    _, cache = layer.prefill(torch.cat([r[:n] for r, n in zip(rows, lengths)])[None].cuda(), torch.tensor(lengths, dtype=torch.int32).cuda())
    ends = [sum(full[:i + 1]) for i in range(4)]
    # the states move to other slots of larger caches
    slots = torch.tensor([4, 0, 8, 3], dtype=torch.int32).cuda()
    for n in ("state", "linear"):
        big = torch.zeros(9, *cache[n].shape[1:], device="cuda")
        big[slots.long()] = cache[n]
        cache[n] = big
    for i in range(more):
        y = layer.decode(torch.stack([r[n + i] for r, n in zip(rows, lengths)]).cuda(), cache, slots)
        for j in range(4):
            err = rel(y[j], want[0, ends[j] - more + i])
            log(f"  token {i} of {j}: {err:.1e}")
            assert err < 1e-4          # fp32 throughout, about 2^-19 a part, and the library products' own rounding
    for j in range(4):
        assert rel(cache["linear"][slots[j]], ends_of[j]) < 1e-4 and rel(cache["state"][slots[j]], s[j]) < 1e-4


def test_decoding_in_a_graph():
    """Tokens decoded by replays of one captured step against the same steps run eagerly, bit for bit."""
    from mixed_layer import MixedLayer
    torch.manual_seed(3)
    layer = MixedLayer()
    lengths = torch.tensor([9, 0, 40], dtype=torch.int32).cuda()
    _, cache = layer.prefill(torch.randn(1, 49, 256).bfloat16().cuda(), lengths)
    eager = {n: t.clone() for n, t in cache.items()}
    x = torch.randn(6, 3, 256).bfloat16().cuda()
    token = x[0].clone()
    warm = {n: t.clone() for n, t in cache.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.decode(token, warm)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.decode(token, cache)
    for t in x:
        token.copy_(t)
        graph.replay()
        want = layer.decode(t, eager)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        for n in cache:
            assert torch.equal(cache[n], eager[n]), n
