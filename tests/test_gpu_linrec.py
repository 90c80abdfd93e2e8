"""The gated linear recurrence on the GPU against its 64-bit form, element by element within the bounds
derived in recurrent_reference."""
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
import recurrent_reference as ref
from gpu_support import log
from layer_reference import cu_of

pytestmark = pytest.mark.gpu


def cuda(t):
    return None if t is None else t.cuda()


def check(what, x, g, lengths=None, h0=None, normalize=False, grads=True, carries=True, seed=9, **kw):
    """Forward (and backward) through the entry points against the reference; returns the GPU's results."""
    B, L, C = x.shape
    gen = torch.Generator().manual_seed(seed)
    n = len(lengths) if lengths is not None else B
    dout = torch.randn(B, L, C, generator=gen).to(x.dtype) if grads else None
    dht = torch.randn(n, C, generator=gen) if grads and h0 is not None else None
    want = ref.linrec(x, g, lengths, h0, normalize, dout, dht)
    cu = None if lengths is None else cu_of(lengths).cuda()
    xs, gs = kw.pop("views", (x.cuda(), g.cuda()))
    o, ht, ca = ccv.gated_linear_recurrence_fwd(xs, gs, cu, cuda(h0), True, normalize, return_carries=True, **kw)
    got = {"out": o, "ht": ht}
    if grads:
        dx, dg, dh = ccv.gated_linear_recurrence_bwd(xs, gs, dout.cuda(), cu, cuda(h0), cuda(dht), normalize,
                                                     ca if carries else None, h0 is not None)
        got.update(dx=dx, dg=dg)
        if h0 is not None:
            got["dh0"] = dh
    for name, t in got.items():
        ref.assert_within(name, t, want[name], what)
    log(f"  {what}: within the bounds")
    return got


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 15, 16, 17, 127, 128, 129, 255, 256, 300])
def test_lengths(L, normalize):
    x, g, h0 = ref.inputs(2, L, 70, seed=L)
    check(f"L {L}", x, g, None, h0, normalize)


@pytest.mark.parametrize("C", [1, 2, 3, 63, 64, 65, 66, 127, 129, 200])
@pytest.mark.parametrize("dtype,gate", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
def test_widths(C, dtype, gate):
    x, g, h0 = ref.inputs(2, 150, C, dtype, gate, seed=C)
    check(f"C {C} {dtype}", x, g, None, h0, C % 2 == 1)


@pytest.mark.parametrize("gate", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("normalize", [False, True])
def test_types(dtype, gate, normalize):
    x, g, h0 = ref.inputs(2, 270, 66, dtype, gate, seed=5, slow=0.99)
    check(f"{dtype} {gate}", x, g, None, h0 if normalize else None, normalize)


@pytest.mark.parametrize("carries", [True, False])
@pytest.mark.parametrize("L", [4096, 4097, 9000])
def test_groups_of_tiles(L, carries):
    x, g, h0 = ref.inputs(2, L, 67, seed=L, slow=0.9999)
    check(f"L {L}", x, g, None, h0, True, carries=carries)


def test_many_groups():
    x, g, h0 = ref.inputs(1, 70001, 3, "bf16", "f32", seed=1, slow=0.9999)
    check("L 70001", x, g, None, h0, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("lengths,rest", [([300], 0), ([300], 1), ([0, 5, 0, 0, 120, 1, 1, 1, 128, 128, 7, 0], 9), ([1] * 40, 300),
                                          ([64, 64, 128, 4096, 0, 200], 0), ([0, 0], 5), ([128, 128, 128], 128)])
def test_packed(lengths, rest, normalize, dtype):
    L = sum(lengths) + rest
    x, g, h0 = ref.inputs(1, L, 66, dtype, "f32", seed=L, seqs=len(lengths))
    x[:, L - rest:] = float("nan")                  # behind the last sequence: not looked at
    g[:, L - rest:] = float("inf")
    clean, cg = x.clone(), g.clone()
    clean[:, L - rest:] = 0
    cg[:, L - rest:] = 0
    for states in (h0, None):
        got = check(f"packed {len(lengths)}", clean, cg, lengths, states, normalize, views=(x.cuda(), g.cuda()))
        for n in ("out", "dx", "dg"):
            assert not bool(got[n][:, L - rest:].any())


def test_many_sequences():
    """More than a piece of the table's kernel holds, most of them empty."""
    gen = torch.Generator().manual_seed(3)
    lengths = (torch.randint(0, 4, (9001,), generator=gen) * (torch.rand(9001, generator=gen) < 0.4)).tolist()
    x, g, h0 = ref.inputs(1, sum(lengths) + 3, 5, seed=4, seqs=len(lengths))
    check("9001 sequences", x, g, lengths, h0, False)


def test_offsets_out_of_order():
    """They count as their running maximum, clamped, and the first as 0."""
    x, g, h0 = ref.inputs(1, 500, 40, seed=2, seqs=6)
    cu = torch.tensor([7, 100, 60, 300, -5, 900, 450], dtype=torch.int32)
    lengths = [100, 0, 200, 0, 200, 0]
    want = ref.linrec(x, g, lengths, h0)
    o, ht = ccv.gated_linear_recurrence_fwd(x.cuda(), g.cuda(), cu.cuda(), h0.cuda(), True)
    ref.assert_within("out", o, want["out"])
    ref.assert_within("ht", ht, want["ht"])


def test_strides():
    """Views with padding, a broadcast row and a broadcast step; odd element offsets."""
    x, g, h0 = ref.inputs(2, 200, 65, "bf16", "bf16", seed=8)
    wide = torch.zeros(2, 200, 140, dtype=torch.bfloat16).cuda()
    wide[..., 3:68] = x.cuda()
    wide[..., 70:135] = g.cuda()
    check("slices", x, g, None, h0, True, views=(wide[..., 3:68], wide[..., 70:135]))
    one = x[:1].expand(2, -1, -1)
    check("broadcast row", one, g, None, h0, False, views=(x[:1].cuda().expand(2, -1, -1), g.cuda()))
    step = g[:, :1].expand(-1, 200, -1)
    check("broadcast step", x, step, None, h0, False, views=(x.cuda(), g[:, :1].cuda().expand(-1, 200, -1)))
    # neither: copied, and said so
    info = {}
    xt = x.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    narrow = g[..., :1].cuda().expand(-1, -1, 65)
    a = ccv.gated_linear_recurrence_fwd(xt, narrow, info=info)
    assert info["copied"] == ["x", "g"]
    assert torch.equal(a, ccv.gated_linear_recurrence_fwd(x.cuda(), narrow.contiguous()))


def test_outputs_given():
    x, g, h0 = (t.cuda() for t in ref.inputs(3, 300, 70, seed=11))
    want, ht = ccv.gated_linear_recurrence_fwd(x, g, initial_state=h0, return_final_state=True)
    buf = torch.full((3, 300, 100), 7.0).cuda()
    state = torch.full((3, 90), 7.0).cuda()
    state[:, 5:75] = h0
    o, s = ccv.gated_linear_recurrence_fwd(x, g, initial_state=state[:, 5:75], return_final_state=True, final_state_out=state[:, 5:75],
                                           out=buf[..., 11:81])
    assert torch.equal(o, want) and torch.equal(s, ht)
    assert bool((buf[..., :11] == 7).all()) and bool((buf[..., 81:] == 7).all())
    assert bool((state[:, :5] == 7).all()) and bool((state[:, 75:] == 7).all())


@pytest.mark.parametrize("lengths", [[100, 0, 5000, 3, 700], [130, 130]])
def test_states_in_place(lengths):
    """final_state over initial_state, in a long chain."""
    L = sum(lengths) + 5
    x, g, h0 = (t.cuda() for t in ref.inputs(1, L, 130, seed=12, seqs=len(lengths)))
    cu = cu_of(lengths).cuda()
    o, ht = ccv.gated_linear_recurrence_fwd(x, g, cu, h0, True)
    state = h0.clone()
    o2, _ = ccv.gated_linear_recurrence_fwd(x, g, cu, state, True, final_state_out=state)
    assert torch.equal(o, o2) and torch.equal(state, ht)


def test_decays_at_the_ends():
    """0 keeps a state, -inf and very large ones drop it, and what normalises x goes to 0 and 1 with them."""
    x, g, h0 = ref.inputs(1, 260, 64, seed=13)
    g[:, ::7] = 0.0
    g[:, 3::50] = -1000.0
    g[:, 5::50] = -1e-30
    g[:, 6::60] = -104.0
    check("ends", x, g, None, h0, True)
    check("ends", x, g, None, h0, False)
    gi = g.clone()
    gi[:, 3::50] = -float("inf")
    for normalize in (False, True):
        a = ccv.gated_linear_recurrence_fwd(x.cuda(), g.cuda(), initial_state=h0.cuda(), normalize=normalize)
        b = ccv.gated_linear_recurrence_fwd(x.cuda(), gi.cuda(), initial_state=h0.cuda(), normalize=normalize)
        assert torch.equal(a, b)


def test_growing():
    """Log decays above 0 grow; the input's weight is then 0 and so are its gradients."""
    x, g, h0 = ref.inputs(2, 140, 30, seed=14)
    g[:, 10:40] = 0.1
    for normalize in (False, True):
        check("growing", x, g, None, h0, normalize)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("nan")])
@pytest.mark.parametrize("where", ["x", "g", "h0", "dout", "dht"])
def test_bad_values_stay_in_their_sequence_and_channel(where, bad):
    lengths = [200, 100, 0, 250]
    x, g, h0 = (t.cuda() for t in ref.inputs(1, 560, 66, seed=15, seqs=4))
    cu, dout, dht = cu_of(lengths).cuda(), torch.randn(1, 560, 66).cuda(), torch.randn(4, 66).cuda()

    def all_of():
        o, ht, ca = ccv.gated_linear_recurrence_fwd(x, g, cu, h0, True, True, return_carries=True)
        return {"out": o[0], "ht": ht, **dict(zip(("dx", "dg", "dh0"), (t.squeeze(0) for t in ccv.gated_linear_recurrence_bwd(
            x, g, dout, cu, h0, dht, True, ca, True))))}
    clean = all_of()
    t = {"x": x, "g": g, "dout": dout}.get(where)
    if t is not None:
        t[0, 250, 7] = bad                                # the second sequence: steps 200 .. 299
    else:
        {"h0": h0, "dht": dht}[where][1, 7] = bad
    got = all_of()
    for n in clean:
        same = torch.ones_like(clean[n], dtype=torch.bool)
        same[(1 if n in ("ht", "dh0") else slice(200, 300)), 7] = False
        assert torch.equal(got[n][same], clean[n][same]), n
    if where in ("x", "g", "h0"):
        assert not bool(torch.isfinite(got["out"][250 if where != "h0" else 200:300, 7]).any())
        if where != "h0":
            assert torch.equal(got["out"][200:250, 7], clean["out"][200:250, 7])


def test_empty():
    for B, L, C in ((2, 0, 5), (0, 4, 5), (2, 4, 0)):
        x, g = torch.zeros(B, L, C).cuda(), torch.zeros(B, L, C).cuda()
        h0 = torch.randn(B, C).cuda()
        o, ht, ca = ccv.gated_linear_recurrence_fwd(x, g, None, h0, True, return_carries=True)
        assert o.shape == x.shape
        if L == 0:
            assert torch.equal(ht, h0)
        dx, dg, dh = ccv.gated_linear_recurrence_bwd(x, g, x, None, h0, h0, False, ca, True)
        assert dx.shape == x.shape
        if L == 0:
            assert torch.equal(dh, h0)
    o, ht = ccv.gated_linear_recurrence_fwd(torch.zeros(1, 0, 5).cuda(), torch.zeros(1, 0, 5).cuda(), torch.zeros(4, dtype=torch.int32).cuda(),
                                            None, True)
    assert torch.equal(ht, torch.zeros(3, 5).cuda())


def test_repeats_bit_for_bit():
    x, g, h0 = (t.cuda() for t in ref.inputs(2, 20000, 130, "bf16", "f32", seed=16, slow=0.9999))
    dout = torch.randn_like(x)
    first = None
    for _ in range(4):
        o, ht, ca = ccv.gated_linear_recurrence_fwd(x, g, None, h0, True, True, return_carries=True)
        res = (o, ht, *ccv.gated_linear_recurrence_bwd(x, g, dout, None, h0, ht, True, ca, True),
               *ccv.gated_linear_recurrence_bwd(x, g, dout, None, h0, ht, True, None, True))
        if first is None:
            first = res
        assert all(torch.equal(a, b) for a, b in zip(res, first))
    assert all(torch.equal(a, b) for a, b in zip(first[2:5], first[5:]))


def test_parts_continue_each_other():
    x, g, h0 = (t.cuda() for t in ref.inputs(2, 700, 66, seed=17))
    o, ht = ccv.gated_linear_recurrence_fwd(x, g, None, h0, True, True)
    s, parts = h0.clone(), []
    for t0, t1 in ((0, 1), (1, 333), (333, 700)):
        p, _ = ccv.gated_linear_recurrence_fwd(x[:, t0:t1], g[:, t0:t1], None, s, True, True, final_state_out=s)
        parts.append(p)
    want = ref.linrec(x.cpu(), g.cpu(), None, h0.cpu(), True)
    ref.assert_within("out", torch.cat(parts, 1), want["out"])
    ref.assert_within("ht", s, want["ht"])


# ---- decoding -------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,gate", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("B,T,C", [(1, 1, 1), (3, 1, 65), (2, 5, 64), (7, 2, 130), (4, 1, 3)])
@pytest.mark.parametrize("normalize", [False, True])
def test_update(B, T, C, dtype, gate, normalize):
    x, g, _ = ref.inputs(B, T, C, dtype, gate, seed=B + T + C, slow=0.99)
    state = torch.randn(B + 4, C)
    slots = torch.randperm(B + 4)[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, B + 4
    live = ((slots >= 0) & (slots < B + 4)).nonzero()[:, 0]
    cache = torch.full((B + 4, C + 9), 5.0)
    cache[:, 4:4 + C] = state
    cache = cache.cuda()
    view = cache[:, 4:4 + C]
    o = ccv.gated_linear_recurrence_update(x.cuda() if T > 1 else x[:, 0].cuda(), g.cuda() if T > 1 else g[:, 0].cuda(), view,
                                           slots.cuda(), normalize)
    o = o if T > 1 else o[:, None]
    want = ref.linrec(x[live], g[live], None, state[slots[live].long()], normalize)
    ref.assert_within("out", o[live.cuda()], want["out"])
    ref.assert_within("state", view[slots[live].long().cuda()], want["ht"])
    idle = torch.ones(B, dtype=torch.bool)
    idle[live] = False
    assert not bool(o[idle.cuda()].any())
    rest = torch.ones(B + 4, dtype=torch.bool)
    rest[slots[live].long()] = False
    assert torch.equal(view[rest.cuda()].cpu(), state[rest])
    assert bool((cache[:, :4] == 5).all()) and bool((cache[:, 4 + C:] == 5).all())


def test_update_is_the_forward():
    """Bit for bit: a step is the same three roundings; without slots, row b has state b."""
    x, g, h0 = (t.cuda() for t in ref.inputs(3, 8, 66, "bf16", "bf16", seed=18))
    o, ht = ccv.gated_linear_recurrence_fwd(x, g, None, h0, True, True)
    s = torch.cat([h0, h0[:1]])
    rows = [ccv.gated_linear_recurrence_update(x[:, t], g[:, t], s, normalize=True) for t in range(8)]
    assert torch.equal(torch.stack(rows, 1), o) and torch.equal(s[:3], ht) and torch.equal(s[3], h0[0])


# ---- autograd, streams, graphs ------------------------------------------------------------------------

def test_autograd():
    lengths = [150, 0, 140]
    x, g, h0 = (t.cuda().requires_grad_() for t in ref.inputs(1, 300, 66, seed=19, seqs=3))
    cu = cu_of(lengths).cuda()
    dout, dht = torch.randn(1, 300, 66).cuda(), torch.randn(3, 66).cuda()
    want = ref.linrec(x.detach().cpu(), g.detach().cpu(), lengths, h0.detach().cpu(), True, dout.cpu(), dht.cpu())
    o, ht = ccv.gated_linear_recurrence_fn(x, g, cu, h0, True, True)
    for n, t in zip(("dx", "dg", "dh0"), torch.autograd.grad([o, ht], [x, g, h0], [dout, dht], retain_graph=True)):
        ref.assert_within(n, t, want[n])
    # the states' gradient alone, and the outputs' alone
    only = ref.linrec(x.detach().cpu(), g.detach().cpu(), lengths, h0.detach().cpu(), True, dout.cpu() * 0, dht.cpu())
    ref.assert_within("dg", torch.autograd.grad(ht, g, dht)[0], only["dg"])
    o = ccv.gated_linear_recurrence_fn(x, g, cu, None, normalize=True)
    only = ref.linrec(x.detach().cpu(), g.detach().cpu(), lengths, None, True, dout.cpu())
    ref.assert_within("dx", torch.autograd.grad(o, x, dout)[0], only["dx"])


def test_broadcast_decays_get_their_sum():
    """One decay a head of channels: an expanded view's gradient is the sum over the head."""
    x, _, _ = ref.inputs(2, 90, 64, seed=20)
    gh = -0.3 * torch.rand(2, 90, 4)
    dout = torch.randn(2, 90, 64)
    gd = gh.cuda().requires_grad_()
    o = ccv.gated_linear_recurrence_fn(x.cuda(), gd[..., None].expand(-1, -1, -1, 16).flatten(2))
    got, = torch.autograd.grad(o, gd, dout.cuda())
    v, e = ref.linrec(x, gh.repeat_interleave(16, -1), dout=dout)["dg"]
    total = v.unflatten(2, (4, 16)).sum(-1)
    ref.assert_within("dg", got, (total, e.unflatten(2, (4, 16)).sum(-1) + 16 * ref.U * v.unflatten(2, (4, 16)).abs().sum(-1)))


def test_another_stream():
    x, g, h0 = (t.cuda() for t in ref.inputs(2, 9000, 66, seed=21))
    want, wt = ccv.gated_linear_recurrence_fwd(x, g, None, h0, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = [ccv.gated_linear_recurrence_fwd(x, g, None, h0, True) for _ in range(3)]
    b = [ccv.gated_linear_recurrence_fwd(x, g, None, h0, True) for _ in range(3)]         # at the same time
    torch.cuda.synchronize()
    for o, ht in a + b:
        assert torch.equal(o, want) and torch.equal(ht, wt)


def test_graphs():
    """Two captured calls, replayed in turn with eager work between; inputs change between replays."""
    lengths = [3000, 0, 1700]
    x, g, h0 = (t.cuda() for t in ref.inputs(1, 4800, 66, "bf16", "f32", seed=22, seqs=3))
    cu, dout = cu_of(lengths).cuda(), torch.randn(1, 4800, 66).cuda().bfloat16()

    def both():
        o, ht, ca = ccv.gated_linear_recurrence_fwd(x, g, cu, h0, True, True, return_carries=True)
        return (o, ht, *ccv.gated_linear_recurrence_bwd(x, g, dout, cu, h0, ht, True, ca, True))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = both()
        graphs.append((graph, res))
    for i in range(3):
        x.copy_(torch.randn_like(x))
        want = [t.clone() for t in both()]
        for graph, res in graphs:
            for t in res:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(res, want)), i
            torch.randn(1000, device="cuda").sum().item()
