"""The recurrence, group norm and rotary positions on arrays whose elements lie more than 2^32 bytes apart:
a step, row or state stride this large keeps the arrays' own sizes small."""
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
import recurrent_reference as ref

pytestmark = pytest.mark.gpu


def spread(t, stride, dim):
    """A copy of t whose dimension `dim` has this stride in elements; the dimensions behind it are contiguous."""
    inner = 1
    strides = [0] * t.dim()
    for d in range(t.dim() - 1, -1, -1):
        strides[d] = stride if d == dim else inner
        inner = strides[d] * t.shape[d] if d == dim else inner * t.shape[d]
    room = torch.empty(1 + sum((n - 1) * s for n, s in zip(t.shape, strides)), dtype=t.dtype, device="cuda")
    v = room.as_strided(t.shape, strides)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_recurrence_steps_far_apart(dtype):
    """Steps at the largest distance there is, 32 MB, over more than one tile: 4.5 GB an array."""
    x, g, h0 = ref.inputs(1, 135, 66, dtype, dtype)
    gen = torch.Generator().manual_seed(1)
    dout = torch.randn(x.shape, generator=gen).to(x.dtype)
    want = ref.linrec(x, g, None, h0, True, dout)
    step = (32 << 20) // x.element_size()
    far = [spread(t, step, 1) for t in (x, g)]
    out = spread(torch.zeros_like(x), step, 1)
    got, ht = ccv.gated_linear_recurrence_fwd(*far, initial_state=h0.cuda(), return_final_state=True, normalize=True, out=out)
    assert got is out
    ref.assert_within("out", out, want["out"])
    ref.assert_within("ht", ht, want["ht"])
    dx, dg, dh = ccv.gated_linear_recurrence_bwd(*far, spread(dout, step, 1), initial_state=h0.cuda(), normalize=True, return_dinitial_state=True)
    for n, t in (("dx", dx), ("dg", dg), ("dh0", dh)):
        ref.assert_within(n, t, want[n])


def test_recurrence_rows_and_states_far_apart():
    x, g, h0 = ref.inputs(3, 20, 70, "bf16")
    rows = (5 << 30) // 2
    far = [spread(t, rows, 0) for t in (x, g.bfloat16())]
    want = ref.linrec(x, g.bfloat16(), None, h0)
    state = spread(h0, rows // 2, 0)
    out, ht = ccv.gated_linear_recurrence_fwd(*far, initial_state=state, return_final_state=True, final_state_out=state)
    ref.assert_within("out", out, want["out"])
    ref.assert_within("ht", state, want["ht"])
    # and the steps behind them, in a cache of such states
    more = ref.linrec(x, g.bfloat16(), None, state.cpu())
    slots = torch.tensor([2, 0, 1], dtype=torch.int32)
    state.copy_(state[torch.tensor([1, 2, 0])].clone())
    out = ccv.gated_linear_recurrence_update(*far, state, slots.cuda())
    ref.assert_within("update", out, more["out"])
    ref.assert_within("state", state[slots.long().cuda()], more["ht"])


@pytest.mark.parametrize("width", [24, 1500])
def test_group_norm_rows_far_apart(width):
    gen = torch.Generator().manual_seed(2)
    x, z, dout = (torch.randn(4, 2 * width, generator=gen).bfloat16() for _ in range(3))
    w, b = torch.rand(2 * width, generator=gen), torch.rand(2 * width, generator=gen)
    want = ref.group_norm(x, 2, w, b, z, True, 1e-5, dout)
    far = lambda t: spread(t, (3 << 30) // 2, 0)  # noqa: E731
    xf, zf = far(x), far(z)
    out, mean, rstd = ccv.group_norm_fwd(xf, 2, w.cuda(), b.cuda(), zf, "silu", return_stats=True)
    dx, dw, db, dz = ccv.group_norm_bwd(xf, 2, w.cuda(), b.cuda(), far(dout), mean, rstd, zf, "silu")
    for n, t in (("out", out), ("mean", mean), ("rstd", rstd), ("dx", dx), ("dw", dw), ("db", db), ("dz", dz)):
        ref.assert_within(n, t, want[n])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_far_apart(interleaved):
    gen = torch.Generator().manual_seed(3)
    q, k = torch.randn(2, 3, 3, 40, generator=gen).bfloat16(), torch.randn(2, 3, 1, 40, generator=gen).bfloat16()
    pos = torch.randint(0, 1 << 20, (2, 3), generator=gen, dtype=torch.int32)
    freq, _ = ccv.rotary_frequencies(32)
    wq, wk = (ref.rotary(t, pos, freq, interleaved) for t in (q, k))
    qf, kf, pf = spread(q, (3 << 30) // 2, 2), spread(k, (5 << 30) // 2, 0), spread(pos, (5 << 30) // 4, 0)
    a, b = ccv.rotary_fwd(qf, kf, pf, freq, interleaved)
    ref.assert_within("q", a, wq)
    ref.assert_within("k", b, wk)
    ccv.rotary_fwd(qf, kf, pf, freq, interleaved, q_out=qf, k_out=kf)
    ref.assert_within("q in place", qf, wq)
    ref.assert_within("k in place", kf, wk)


@pytest.mark.parametrize("normalize", [False, True])
def test_rows_of_a_large_call_are_those_of_smaller_ones(normalize):
    """Calls of many tiles run in other numbers of workgroups a compute unit: the same bits, and the 64-bit results."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x, g, dout, h0, dht = rand(100, 300, 2688), -rand(100, 300, 2688).abs(), rand(100, 300, 2688), rand(100, 2688), rand(100, 2688)

    def results(rows, channels=slice(None)):
        a, b, d, h, e = (t[rows][..., channels] for t in (x, g, dout, h0, dht))
        out, ht, ca = ccv.gated_linear_recurrence_fwd(a, b, initial_state=h, return_final_state=True, normalize=normalize, return_carries=True)
        dx, dg, dh = ccv.gated_linear_recurrence_bwd(a, b, d, initial_state=h, dfinal_state=e, normalize=normalize, carries=ca, return_dinitial_state=True)
        return {"out": out, "ht": ht, "dx": dx, "dg": dg, "dh0": dh}

    large, few = results(slice(None)), slice(40, 44)
    for n, t in results(few).items():
        assert torch.equal(t, large[n][few]), n
    want = ref.linrec(*(t[few][..., :96].cpu() for t in (x, g)), None, h0[few][..., :96].cpu(), normalize, dout[few][..., :96].cpu(), dht[few][..., :96].cpu())
    for n, t in large.items():
        ref.assert_within(n, t[few][..., :96], want[n])
