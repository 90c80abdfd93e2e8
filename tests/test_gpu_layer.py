"""The operators together, as the example layer uses them: a packed row's result and gradients
against the same layer run in 64 bits on the CPU, and decoding against prefill.

Tolerance: every intermediate is rounded to bf16 (2^-9 in mean square) in about ten places
between x and the result, and once more on the way back: sqrt(20) 2^-9 = 0.9 % in the 2-norm for
values, taken twice for gradients, where the roundings pass through a second chain.  The decay's
gradient is a sum over all steps of terms that cancel, which such a bound does not cover (bf16
rounding of the intermediates alone moves it by up to 4 %): it is checked in fp32, where every
tensor has to be within 1e-4, the delta rule's 2^-18 and the library products' own rounding."""
import os
import sys

import pytest
import torch
import torch.nn.functional as F

import layer_reference as ref
from gpu_support import log

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def plain(layer, x, lengths):
    """The layer's formula in 64 bits on the CPU; parameters as leaves of the same names."""
    p = {n: t.detach().cpu().double().requires_grad_() for n, t in layer.named_parameters()}
    norm = lambda t, w, b: F.layer_norm(t, t.shape[-1:], w, b, 1e-5)  # noqa: E731
    n = norm(x, p["norm_w"], p["norm_b"])
    g = -p["decay"] * F.softplus(F.linear(n, p["w_gate"]))
    beta = torch.sigmoid(F.linear(n, p["w_beta"]))
    c = F.linear(n, p["w_in"])
    parts, at = [], 0
    for ln in lengths:
        if ln:
            t = F.pad(c[:, at:at + ln].transpose(1, 2), (layer.conv_w.shape[1] - 1, 0))
            parts.append(F.silu(F.conv1d(t, p["conv_w"][:, None], groups=c.shape[2])).transpose(1, 2))
        at += ln
    parts.append(torch.zeros(1, x.shape[1] - at, c.shape[2], dtype=torch.float64))
    q, k, v = torch.cat(parts, 1).split(layer.split, -1)
    q, k = (F.normalize(t.unflatten(-1, (layer.hk, layer.dk)), dim=-1) for t in (q, k))
    o, s = ref.delta_reference(q, k, v.unflatten(-1, (layer.hv, layer.dv)), g, beta, None, lengths)
    return x + F.linear(norm(o, p["out_w"], p["out_b"]).flatten(-2), p["w_out"]), s, p


@pytest.mark.parametrize("lengths,rest", [([100], 0), ([70, 0, 1, 65], 5), ([3, 2, 64], 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_packed_row(lengths, rest, dtype):
    from delta_layer import DeltaLayer
    torch.manual_seed(1)
    layer = DeltaLayer(dtype=dtype)
    wide = dtype == torch.float32
    T = sum(lengths) + rest
    x = torch.randn(1, T, 256).to(dtype)
    live = sum(lengths)
    dout = torch.randn(1, T, 256).to(dtype)
    dout[:, live:] = 0                              # the steps that belong to no sequence train nothing
    xd = x.double().requires_grad_()
    want, _, p = plain(layer, xd, lengths)
    wg = torch.autograd.grad(want, [xd, *p.values()], dout.double())
    xg = x.cuda().requires_grad_()
    y = layer.train_row(xg, torch.tensor(lengths, dtype=torch.int32).cuda())
    gg = torch.autograd.grad(y, [xg, *layer.parameters()], dout.cuda())
    rel = lambda a, b: float((a.detach().cpu().double() - b.detach()).norm() / b.detach().norm())  # noqa: E731
    log(f"  layer {lengths} out {rel(y[:, :live], want[:, :live]):.2e}")
    assert rel(y[:, :live], want[:, :live]) < (1e-4 if wide else 9e-3)
    for name, a, b in zip(["x", *p], gg, wg):
        log(f"    d{name} {rel(a, b):.2e}")
        assert wide or name == "decay" or rel(a, b) < 1.8e-2, name
        assert not wide or rel(a, b) < 1e-4, name


def test_decode_continues_prefill():
    from delta_layer import DeltaLayer
    torch.manual_seed(2)
    layer = DeltaLayer(dtype=torch.float32)
    lengths, more = [65, 1, 0, 30], 5
    full = [n + more for n in lengths]
    rows = [torch.randn(n, 256) for n in full]
    want, _, _ = plain(layer, torch.cat(rows)[None].double(), full)
    y, cache = layer.prefill(torch.cat([r[:n] for r, n in zip(rows, lengths)])[None].cuda(),
                             torch.tensor(lengths, dtype=torch.int32).cuda())
    ends = [sum(full[:i + 1]) for i in range(4)]
    # the states move to other slots of a larger cache
    big = torch.zeros(9, *cache["state"].shape[1:], device="cuda")
    slots = torch.tensor([4, 0, 8, 3], dtype=torch.int32).cuda()
    big[slots.long()] = cache["state"]
    cache["state"] = big
    for i in range(more):
        y = layer.decode(torch.stack([r[n + i] for r, n in zip(rows, lengths)]).cuda(), cache, slots)
        for s in range(4):
            w = want[0, ends[s] - more + i]
            err = float((y[s].cpu().double() - w).norm() / w.norm())
            log(f"  token {i} of {s}: {err:.1e}")
            assert err < 1e-4          # fp32 throughout, about 2^-19 a part, and the library products' own rounding
