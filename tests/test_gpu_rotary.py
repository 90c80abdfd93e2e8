"""Rotary positions on the GPU against their 64-bit form, element by element within the bounds derived in
recurrent_reference."""
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
import recurrent_reference as ref
from gpu_support import log
from layer_reference import DT

pytestmark = pytest.mark.gpu


def inputs(B, L, H, D, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(B, L, H, D, generator=gen).to(DT[dtype])


def check(what, q, k, pos, freq, interleaved=False, scale=1.0, inverse=False, views=None, **kw):
    qg, kg, pg = views or (q.cuda(), None if k is None else k.cuda(), pos.cuda())
    got = ccv.rotary_fwd(qg, kg, pg, freq.cuda(), interleaved, scale, inverse, **kw)
    for name, x, y in (("q", q, got[0]), ("k", k, got[1])):
        if x is None:
            assert y is None
        else:
            ref.assert_within(name, y, ref.rotary(x, pos, freq, interleaved, scale, inverse), what)
    log(f"  {what}: within the bounds")
    return got


def positions(B, L, far=0):
    return (torch.arange(L, dtype=torch.int32) + far)[None] * torch.ones(B, 1, dtype=torch.int32)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,turned", [(2, 2), (3, 2), (6, 4), (8, 8), (9, 8), (16, 16), (16, 8), (22, 22), (24, 10), (64, 64), (64, 32), (70, 70),
                                      (96, 64), (100, 50), (128, 128), (128, 64), (128, 2), (200, 120), (256, 256), (256, 64), (576, 64),
                                      (2048, 2048), (1000, 998)])
def test_widths(D, turned, interleaved, dtype):
    q, k = inputs(2, 5, 3, D, dtype, D), inputs(2, 5, 2, D, dtype, turned)
    freq, _ = ccv.rotary_frequencies(turned, device="cpu")
    check(f"D {D} turned {turned} {dtype}", q, k, positions(2, 5, 100), freq, interleaved)


@pytest.mark.parametrize("B,L,Hq,Hk", [(1, 1, 1, 0), (1, 1, 1, 1), (3, 1, 32, 8), (2, 300, 5, 1), (1, 1000, 1, 1), (4, 7, 40, 40), (257, 1, 3, 2),
                                       (1, 3, 300, 1)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_shapes(B, L, Hq, Hk, interleaved):
    q, k = inputs(B, L, Hq, 64, "bf16", 1), inputs(B, L, Hk, 64, "bf16", 2) if Hk else None
    freq, _ = ccv.rotary_frequencies(48, device="cpu")
    check(f"{B} {L} {Hq} {Hk}", q, k, positions(B, L, 5), freq, interleaved, 1.3)


@pytest.mark.parametrize("far", [0, 1 << 20, (1 << 31) - 8, -(1 << 31), -5])
def test_far_positions(far):
    q = inputs(1, 7, 2, 128, "f32", 3)
    freq, _ = ccv.rotary_frequencies(128, device="cpu")
    check(f"from {far}", q, None, positions(1, 7, far), freq)


@pytest.mark.parametrize("scaling", [None, "linear", "base", "parts"])
def test_scalings(scaling):
    q, k = inputs(1, 50, 2, 128, "f32", 4), inputs(1, 50, 1, 128, "f32", 5)
    freq, scale = ccv.rotary_frequencies(128, 500000.0, scaling, 8.0, 8192, device="cpu")
    check(f"{scaling}", q, k, positions(1, 50, 100000), freq, False, scale)


@pytest.mark.parametrize("dtype,D,turned", [("bf16", 128, 64), ("f32", 20, 12), ("f16", 100, 50), ("f32", 64, 64), ("bf16", 7, 6)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_and_in_place(dtype, D, turned, interleaved):
    """Views of one buffer at an odd offset; then in place, with what lies between left as it was."""
    B, L, Hq, Hk = 2, 9, 4, 2
    q, k = inputs(B, L, Hq, D, dtype, 6), inputs(B, L, Hk, D, dtype, 7)
    freq, _ = ccv.rotary_frequencies(turned, device="cpu")
    pos = torch.randint(-50, 5000, (B, L), dtype=torch.int32)
    buf = torch.full((B, L, 11 + (Hq + Hk) * (D + 3)), 9.0, dtype=DT[dtype]).cuda()
    heads = buf[..., 11:].unflatten(-1, (Hq + Hk, D + 3))
    vq, vk = heads[..., :Hq, 1:D + 1], heads[..., Hq:, 1:D + 1]
    vq.copy_(q)
    vk.copy_(k)
    at = torch.zeros(B, 2 * L, dtype=torch.int32).cuda()
    at[:, ::2] = pos.cuda()
    views = vq, vk, at[:, ::2]
    want = check("views", q, k, pos, freq, interleaved, 0.9, views=views)
    got = ccv.rotary_fwd(*views, freq.cuda(), interleaved, 0.9, q_out=vq, k_out=vk)
    assert got[0] is vq and torch.equal(vq, want[0]) and torch.equal(vk, want[1])
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[..., 11:].unflatten(-1, (Hq + Hk, D + 3))[..., 1:D + 1] = False
    assert bool((buf[mask] == 9).all())
    # one of the two in place
    vq.copy_(q)
    vk.copy_(k)
    a, b = ccv.rotary_fwd(vq, vk, at[:, ::2], freq.cuda(), interleaved, 0.9, q_out=vq)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(vk.cpu(), k)


def test_one_step_and_shared_positions():
    q, k = inputs(5, 1, 4, 64, "f16", 8), inputs(5, 1, 2, 64, "f16", 9)
    freq, _ = ccv.rotary_frequencies(64, device="cpu")
    pos = torch.randint(0, 5000, (5, 1), dtype=torch.int32)
    want = check("steps", q, k, pos, freq)
    a, b = ccv.rotary_fwd(q[:, 0].cuda(), k[:, 0].cuda(), pos[:, 0].cuda(), freq.cuda())
    assert torch.equal(a, want[0][:, 0]) and torch.equal(b, want[1][:, 0])
    same = torch.randint(0, 99, (1, 1), dtype=torch.int32).expand(5, 1)
    check("one position", q, k, same, freq, views=(q.cuda(), k.cuda(), same[:1].cuda().expand(5, 1)))


def test_back_and_forth():
    """The inverse takes a turn back, within both's roundings."""
    q = inputs(1, 40, 3, 64, "f32", 10)
    freq, _ = ccv.rotary_frequencies(64, device="cpu")
    there = check("there", q, None, positions(1, 40), freq)[0]
    back = check("back", there.cpu(), None, positions(1, 40), freq, inverse=True)[0]
    assert float((back.cpu() - q).abs().max()) < 32 * ref.U * float(q.abs().max())


def test_nothing_turned_and_empty():
    q = inputs(2, 3, 2, 9, "f32", 11).cuda()
    none = torch.zeros(0, dtype=torch.float64).cuda()
    pos = positions(2, 3).cuda()
    assert torch.equal(ccv.rotary_fwd(q, None, pos, none)[0], q)
    p = q.clone()
    ccv.rotary_fwd(p, None, pos, none, q_out=p)
    assert torch.equal(p, q)
    for shape in ((0, 3, 2, 8), (2, 0, 2, 8), (2, 3, 0, 8)):
        e = torch.zeros(shape).cuda()
        f, _ = ccv.rotary_frequencies(8)
        assert ccv.rotary_fwd(e, e, torch.zeros(shape[:2], dtype=torch.int32).cuda(), f)[0].shape == shape


def test_gradients():
    """The formula's (the inverse turn), and differences of the reference."""
    q, k = inputs(2, 6, 3, 24, "f32", 12), inputs(2, 6, 1, 24, "f32", 13)
    freq, _ = ccv.rotary_frequencies(20)
    pos = positions(2, 6, 900)
    dq, dk = torch.randn(q.shape), torch.randn(k.shape)
    for interleaved in (False, True):
        leaves = [t.cuda().requires_grad_() for t in (q, k)]
        out = ccv.rotary_fn(*leaves, pos.cuda(), freq, interleaved, 1.5)
        grads = torch.autograd.grad(out, leaves, [dq.cuda(), dk.cuda()])
        for n, g, d in (("dq", grads[0], dq), ("dk", grads[1], dk)):
            ref.assert_within(n, g, ref.rotary(d, pos, freq, interleaved, 1.5, True))
        step = torch.randn(q.shape).double()
        h = 2.0 ** -10
        f = lambda t: float((ref.rotary(q.double() + t * step, pos, freq, interleaved, 1.5)[0] * dq.double()).sum())  # noqa: E731
        slope = (f(h) - f(-h)) / (2 * h)                   # the map is linear: exact but for 64-bit rounding
        mine = float((grads[0].double().cpu() * step).sum())
        assert abs(mine - slope) <= 64 * ref.U * float((dq.abs() * 3 * step.abs()).sum()) + 1e-9
    # one of the two alone
    leaf = k.cuda().requires_grad_()
    out = ccv.rotary_fn(q.cuda(), leaf, pos.cuda(), freq)
    ref.assert_within("dk", torch.autograd.grad(out[1], leaf, dk.cuda())[0], ref.rotary(dk, pos, freq, inverse=True))


def test_streams_and_graphs():
    q, k = inputs(2, 50, 4, 64, "bf16", 14).cuda(), inputs(2, 50, 2, 64, "bf16", 15).cuda()
    freq, _ = ccv.rotary_frequencies(64)
    pos = positions(2, 50).cuda()
    want = ccv.rotary_fwd(q, k, pos, freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ccv.rotary_fwd(q, k, pos, freq)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ccv.rotary_fwd(q, k, pos, freq)
    for i in range(3):
        pos += 17                                          # the next tokens: positions are read by the replay
        want = ccv.rotary_fwd(q, k, pos, freq)
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
