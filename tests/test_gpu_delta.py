"""The gated delta rule on the GPU against its 64-bit step-by-step reference: forward, gradients
and the update, over head layouts, widths, lengths, dtypes, strides, packed rows and states."""
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
import layer_reference as ref
from gpu_support import log

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    ccv.lib()

NAN = float("nan")


def gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def check_fwd(q, k, v, g, beta, h0=None, lengths=None, scale=None, what="", views=None):
    log(f"  delta fwd {what} q {tuple(q.shape)} v {tuple(v.shape)} {q.dtype} lengths {lengths and len(lengths)}")
    cu = None if lengths is None else ref.cu_of(lengths).cuda()
    args = views or gpu(q, k, v, g, beta)
    out, ht = ccv.gated_delta_rule_fwd(*args, scale=scale, cu_seqlens=cu, initial_state=gpu(h0)[0], return_final_state=True)
    torch.cuda.synchronize()
    want, wht = ref.delta_reference(q, k, v, g, beta, scale, lengths, h0)
    ref.assert_near("out", out, want, 1, what)
    ref.assert_near("final_state", ht, wht, 1, what)
    return out, ht


def check_bwd(q, k, v, g, beta, h0=None, lengths=None, what="", dht=True, views=None, dout=None):
    log(f"  delta bwd {what} q {tuple(q.shape)} v {tuple(v.shape)} {q.dtype} lengths {lengths and len(lengths)}")
    gen = torch.Generator().manual_seed(99)
    dout = torch.randn(v.shape, generator=gen).to(v.dtype) if dout is None else dout
    n = q.shape[0] if lengths is None else len(lengths)
    dht = torch.randn(n, v.shape[2], q.shape[3], v.shape[3], generator=gen) * 0.2 if dht else None
    cu = None if lengths is None else ref.cu_of(lengths).cuda()
    args = views or gpu(q, k, v, g, beta)
    got = ccv.gated_delta_rule_bwd(*args, dout.cuda(), cu_seqlens=cu, initial_state=gpu(h0)[0], dfinal_state=gpu(dht)[0],
                                   return_dinitial_state=h0 is not None)
    torch.cuda.synchronize()
    want = ref.delta_gradients(q, k, v, g, beta, dout, None, lengths, h0, dht)
    for name, t in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got):
        if t is not None:
            ref.assert_near(name, t, want[name], 2, what)
    return got


LENGTHS = [1, 2, 63, 64, 65, 128, 130, 257]
WIDTHS = [(64, 64), (128, 128), (1, 1), (3, 5), (72, 96), (96, 40), (128, 33), (65, 130), (127, 17)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("L", LENGTHS)
def test_forward_lengths(dtype, L):
    q, k, v, g, beta, h0 = ref.delta_inputs(2, L, 1, 2, 64, 32, dtype, seed=L)
    check_fwd(q, k, v, g, beta, h0, what=f"L={L}")
    check_fwd(q, k, v, g, beta, None, what=f"L={L} no state")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Dk,Dv", WIDTHS)
def test_forward_widths(dtype, Dk, Dv):
    q, k, v, g, beta, h0 = ref.delta_inputs(1, 100, 2, 4, Dk, Dv, dtype, "bf16", "f16", seed=Dk)
    check_fwd(q, k, v, g, beta, h0, what=f"{Dk}x{Dv}")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 64, 65, 130])
def test_gradients_lengths(dtype, L):
    q, k, v, g, beta, h0 = ref.delta_inputs(2, L, 1, 2, 64, 32, dtype, "f32", "bf16", seed=L)
    check_bwd(q, k, v, g, beta, h0, what=f"L={L}")
    check_bwd(q, k, v, g, beta, None, what=f"L={L} no state")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Dk,Dv", WIDTHS)
def test_gradients_widths(dtype, Dk, Dv):
    q, k, v, g, beta, h0 = ref.delta_inputs(1, 70, 2, 6, Dk, Dv, dtype, "f32", "f32", seed=Dv)
    check_bwd(q, k, v, g, beta, h0, what=f"{Dk}x{Dv}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_heads_take_the_wider_slices(dtype):
    """Enough heads for workgroups of 32 values, and a value width that is no multiple of them."""
    q, k, v, g, beta, h0 = ref.delta_inputs(9, 66, 16, 16, 64, 72, dtype, seed=3)
    check_fwd(q, k, v, g, beta, h0, what="144 heads")
    check_bwd(q, k, v, g, beta, h0, what="144 heads")


# rows, key heads, value heads, widths: at least 1024 blocks of 16 values, where 16-bit inputs take whole
# columns a wave
WAVES = [(16, 4, 16, 64, 64), (16, 16, 16, 128, 50), (11, 4, 16, 72, 96), (64, 1, 8, 1, 17), (4, 16, 32, 128, 128)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("i", range(len(WAVES)))
@pytest.mark.parametrize("L", [1, 64, 130])
def test_whole_columns(dtype, i, L):
    B, Hk, Hv, Dk, Dv = WAVES[i]
    q, k, v, g, beta, h0 = ref.delta_inputs(B, L, Hk, Hv, Dk, Dv, dtype, "f32", "bf16", seed=i)
    check_fwd(q, k, v, g, beta, h0, what="columns")
    check_bwd(q, k, v, g, beta, h0 if L > 1 else None, what="columns")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("few", [False, True])
def test_columns_of_different_size(dtype, few):
    """Values and states of 1e-5 to 3e4 side by side: each column keeps its own precision."""
    B, H = (1, 2) if few else (16, 16)
    q, k, v, g, beta, h0 = ref.delta_inputs(B, 100, H, H, 64, 64, dtype, seed=5)
    size = 10.0 ** torch.linspace(-3 if dtype == "f16" else -5, 4, 64)
    v, h0 = (v.float() * size).to(v.dtype), h0 * size
    dout = torch.randn(v.shape, generator=torch.Generator().manual_seed(1)).to(v.dtype)
    out, ht = ccv.gated_delta_rule_fwd(*gpu(q, k, v, g, beta), initial_state=h0.cuda(), return_final_state=True)
    got = ccv.gated_delta_rule_bwd(*gpu(q, k, v, g, beta, dout), initial_state=h0.cuda(), return_dinitial_state=True)
    want = ref.delta_gradients(q, k, v, g, beta, dout, None, None, h0)
    for c in range(0, 64, 9):
        ref.assert_near("out", out[..., c], want["out"][..., c], 1, f"column {c}")
        ref.assert_near("final_state", ht[..., c], want["ht"][..., c], 1, f"column {c}")
        ref.assert_near("dv", got[2][..., c], want["dv"][..., c], 2, f"column {c}")
        ref.assert_near("dh0", got[5][..., c], want["dh0"][..., c], 2, f"column {c}")


def test_nan_stays_in_its_column_of_values():
    q, k, v, g, beta, h0 = ref.delta_inputs(16, 70, 16, 16, 64, 64, "f16", seed=6)
    clean, _ = ccv.gated_delta_rule_fwd(*gpu(q, k, v, g, beta), initial_state=h0.cuda(), return_final_state=True)
    v[3, 20, 5, 7], v[2, 20, 5, 8] = NAN, float("inf")
    out, _ = ccv.gated_delta_rule_fwd(*gpu(q, k, v, g, beta), initial_state=h0.cuda(), return_final_state=True)
    same = torch.ones(16, 70, 16, 64, dtype=torch.bool)
    same[3, :, 5, 7] = same[2, :, 5, 8] = False
    assert torch.equal(out.cpu()[same], clean.cpu()[same])
    assert torch.isnan(out[3, 20:, 5, 7]).all() and not torch.isfinite(out[2, 20:, 5, 8]).any()


def test_many_sequences_of_one_row():
    """Packed rows of whole-column waves: 130 sequences, longest first whatever their order."""
    gen = torch.Generator().manual_seed(3)
    lengths = torch.randint(0, 40, (130,), generator=gen).tolist()
    lengths[17], lengths[100] = 200, 129
    for dtype in ("f16", "bf16"):
        q, k, v, g, beta, h0 = ref.delta_inputs(1, sum(lengths), 1, 2, 64, 64, dtype, seed=4, seqs=130)
        check_fwd(q, k, v, g, beta, h0, lengths, what="130 sequences")
        check_bwd(q, k, v, g, beta, h0, lengths, what="130 sequences")


# few heads and many chunks: the passes take the sequences in parts
LONG = [(1, 1, 64, 64, [1030]), (1, 2, 128, 40, [2048]), (2, 4, 72, 33, [1500]), (1, 1, 64, 64, [1100, 0, 3, 1500]),
        (1, 3, 20, 130, [0, 64, 2500, 0]), (1, 2, 64, 64, [4096 + 64])]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("i", range(len(LONG)))
def test_long_sequences_of_few_heads(dtype, i):
    Hk, Hv, Dk, Dv, lengths = LONG[i]
    one = len(lengths) == 1
    q, k, v, g, beta, h0 = ref.delta_inputs(1, sum(lengths) + (0 if one else 7), Hk, Hv, Dk, Dv, dtype, seed=i, seqs=len(lengths),
                                            decay=0.01)
    check_fwd(q, k, v, g, beta, h0, None if one else lengths, what="long")
    check_bwd(q, k, v, g, beta, h0, None if one else lengths, what="long")
    g[:, 700] = -float("inf")
    g[:, 64:300] = 0.01
    check_fwd(q, k, v, g.clamp(min=-1e4), beta, None, None if one else lengths, what="long, forgotten", views=gpu(q, k, v, g, beta))


def test_nan_in_a_part_stays_behind_it():
    q, k, v, g, beta, _ = ref.delta_inputs(1, 2048, 1, 2, 64, 64, "bf16", seed=1)
    clean = ccv.gated_delta_rule_fwd(*gpu(q, k, v, g, beta))
    v[0, 1000, 1, 5], k[0, 1500, 0, 3] = NAN, NAN
    out = ccv.gated_delta_rule_fwd(*gpu(q, k, v, g, beta))
    same = torch.ones(1, 2048, 2, 64, dtype=torch.bool)
    same[0, 960:, 1, 5] = False             # from its chunk on
    same[0, 1472:] = False
    assert torch.equal(out.cpu()[same], clean.cpu()[same])
    assert torch.isnan(out[0, 1000:, 1, 5]).all() and torch.isnan(out[0, 1500:]).all()


PACKED = [[5, 0, 64, 1, 130], [0, 0, 7], [64, 64], [200], [0], [1] * 20, [65, 0]]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(PACKED)))
@pytest.mark.parametrize("rest", [0, 3, 70])
def test_packed_rows(dtype, i, rest):
    """Sequences of a row, empty ones among them; the steps behind them are not looked at."""
    lengths = PACKED[i]
    T = sum(lengths) + rest
    if T == 0:
        return
    q, k, v, g, beta, h0 = ref.delta_inputs(1, T, 2, 4, 64, 40, dtype, seed=i, seqs=len(lengths))
    dout = torch.randn(v.shape, generator=torch.Generator().manual_seed(1)).to(v.dtype)
    bad = [t.clone() for t in (q, k, v, g, beta, dout)]
    for t in bad:
        t[:, sum(lengths):] = NAN
    cu = ref.cu_of(lengths).cuda()
    out, ht = ccv.gated_delta_rule_fwd(*gpu(*bad[:5]), cu_seqlens=cu, initial_state=h0.cuda(), return_final_state=True)
    got = ccv.gated_delta_rule_bwd(*gpu(*bad), cu_seqlens=cu, initial_state=h0.cuda(), return_dinitial_state=True)
    want = ref.delta_gradients(q, k, v, g, beta, dout, None, lengths, h0)
    log(f"  packed {lengths} + {rest}")
    ref.assert_near("out", out, want["out"])
    ref.assert_near("final_state", ht, want["ht"])
    for name, t in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got):
        ref.assert_near(name, t, want[name], 2)
        if name != "dh0":
            assert not t[:, sum(lengths):].any(), name


def test_offsets_are_clamped():
    """Offsets that fall, or lead outside the row, count as their running maximum in [0, L]."""
    q, k, v, g, beta, _ = ref.delta_inputs(1, 100, 1, 2, 64, 32, seed=1)
    cu = torch.tensor([7, 30, 20, -5, 400], dtype=torch.int32, device="cuda")
    out, ht = ccv.gated_delta_rule_fwd(*gpu(q, k, v, g, beta), cu_seqlens=cu, return_final_state=True)
    want, wht = ref.delta_reference(q, k, v, g, beta, None, [30, 0, 0, 70])
    ref.assert_near("out", out, want)
    ref.assert_near("final_state", ht, wht)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_strided_views(dtype):
    """Views of one wider buffer at odd offsets, heads before steps, and gates broadcast over heads."""
    B, L, Hk, Hv, Dk, Dv = 2, 90, 2, 4, 64, 48
    q, k, v, g, beta, h0 = ref.delta_inputs(B, L, Hk, Hv, Dk, Dv, dtype, seed=4)
    for off, pad in ((0, 8), (3, 1), (1, 0)):
        buf = torch.full((B, L, off + 2 * Hk * Dk + Hv * Dv + pad), NAN, dtype=q.dtype, device="cuda")
        a, b = off + Hk * Dk, off + 2 * Hk * Dk
        views = [buf[..., off:a].unflatten(2, (Hk, Dk)), buf[..., a:b].unflatten(2, (Hk, Dk)),
                 buf[..., b:b + Hv * Dv].unflatten(2, (Hv, Dv))]
        for view, t in zip(views, (q, k, v)):
            view.copy_(t)
        views += gpu(g, beta)
        check_fwd(q, k, v, g, beta, h0, what=f"fused at {off}", views=views)
        check_bwd(q, k, v, g, beta, h0, what=f"fused at {off}", views=views)
    views = [t.cuda().transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    gb, bb = g[:, :, :1].expand(B, L, Hv), beta[:1, :1].expand(B, L, Hv)
    views += [g[:, :, :1].cuda().expand(B, L, Hv), beta[:1, :1].cuda().expand(B, L, Hv)]
    check_fwd(q, k, v, gb, bb, h0, what="heads first", views=views)
    check_bwd(q, k, v, gb, bb, h0, what="heads first", views=views)
    info = {}
    odd = q.cuda().transpose(2, 3).contiguous().transpose(2, 3)      # no unit stride inside a head: copied
    out = ccv.gated_delta_rule_fwd(odd, *gpu(k, v, g, beta), info=info)
    assert info["copied"] == ["q"]
    ref.assert_near("out", out, ref.delta_reference(q, k, v, g, beta)[0])


def test_one_step_rows_with_any_stride():
    """A single step whose step stride is never used, zero or huge."""
    q, k, v, g, beta, h0 = ref.delta_inputs(3, 1, 1, 2, 64, 32, "bf16", seed=8)
    for s in (0, 1 << 40):
        views = [t.cuda().as_strided(t.shape, (t.stride(0), s, t.stride(2)) + ((1,) if t.dim() == 4 else ())) for t in (q, k, v, g, beta)]
        check_fwd(q, k, v, g, beta, h0, what=f"stride {s}", views=views)
        check_bwd(q, k, v, g, beta, h0, what=f"stride {s}", views=views)


def test_offsets_past_32_bits():
    """Rows whose elements lie more than 2^32 bytes into their buffer."""
    q, k, v, g, beta, h0 = ref.delta_inputs(2, 70, 1, 1, 64, 32, "bf16", seed=2)
    big = 1 << 32
    buf = torch.empty(big + 70 * 64 * 4, dtype=torch.bfloat16, device="cuda")
    views = []
    for t in (q, k, v):
        x = buf.as_strided(t.shape, (big, t.stride(1), t.stride(2), 1), len(views) * 70 * 64)
        x.copy_(t)
        views.append(x)
    check_fwd(q, k, v, g, beta, h0, what="far rows", views=views + gpu(g, beta))
    check_bwd(q, k, v, g, beta, h0, what="far rows", views=views + gpu(g, beta))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_at_their_ends(dtype):
    """Forgotten states (-inf and far below 0), strengths of 0 and of 2, growth, strong decay."""
    B, L, H = 1, 140, 2
    q, k, v, g, beta, h0 = ref.delta_inputs(B, L, H, H, 64, 32, dtype, seed=6)
    beta[:, 10:20] = 0
    beta[:, 30] = 2
    check_fwd(q, k, v, g, beta, h0, what="beta ends")
    check_bwd(q, k, v, g, beta, h0, what="beta ends")
    g[:, 5:9] = 0.05
    g[:, 70:100] = -3.0
    check_fwd(q, k, v, g, beta, h0, what="growth and strong decay")
    check_bwd(q, k, v, g, beta, h0, what="growth and strong decay")
    g[:, 40] = -float("inf")
    g[:, 64, 0] = -1e30
    g[:, 101:103] = -float("inf")
    finite = g.clamp(min=-1e4)      # e^-1e4 is 0 in 64 bits too, without inf - inf in the reference's gradients
    out, ht = ccv.gated_delta_rule_fwd(*gpu(q, k, v, g, beta), initial_state=h0.cuda(), return_final_state=True)
    want, wht = ref.delta_reference(q, k, v, finite, beta, None, None, h0)
    ref.assert_near("out", out, want)
    ref.assert_near("final_state", ht, wht)
    check_bwd(q, k, v, finite, beta, h0, what="forgotten")
    got = ccv.gated_delta_rule_bwd(*gpu(q, k, v, g, beta), torch.ones_like(v).cuda(), initial_state=h0.cuda())
    assert all(torch.isfinite(t).all() for t in got[:5])


def test_gradients_that_are_zero():
    """The first step of a sequence without a state decays nothing: its dg is exactly 0."""
    q, k, v, g, beta, _ = ref.delta_inputs(1, 90, 1, 2, 64, 32, "bf16", seed=7)
    got = ccv.gated_delta_rule_bwd(*gpu(q, k, v, g, beta), torch.ones_like(v).cuda())
    assert not got[3][:, 0].any() and got[3][:, 1:].any()
    cu = ref.cu_of([1] * 90).cuda()
    got = ccv.gated_delta_rule_bwd(*gpu(q, k, v, g, beta), torch.ones_like(v).cuda(), cu_seqlens=cu)
    assert not got[3].any()


def test_nan_stays_in_its_sequence_and_head():
    lengths = [70, 66, 64]
    q, k, v, g, beta, h0 = ref.delta_inputs(1, 200, 2, 4, 64, 32, "bf16", seed=9, seqs=3)
    clean = ccv.gated_delta_rule_fwd(*gpu(q, k, v, g, beta), cu_seqlens=ref.cu_of(lengths).cuda(), initial_state=h0.cuda(),
                                     return_final_state=True)
    v2, k2 = v.clone(), k.clone()
    v2[0, 100, 1] = NAN                     # sequence 1, value head 1
    k2[0, 10, 1] = float("inf")             # sequence 0, key head 1: value heads 2 and 3
    out, ht = ccv.gated_delta_rule_fwd(*gpu(q, k2, v2, g, beta), cu_seqlens=ref.cu_of(lengths).cuda(), initial_state=h0.cuda(),
                                       return_final_state=True)
    same = torch.ones(1, 200, 4, dtype=torch.bool)
    same[0, 70:136, 1] = False
    same[0, :70, 2:] = False
    assert torch.equal(out.cpu()[same], clean[0].cpu()[same])
    assert torch.isnan(out[0, 100:136, 1]).any(-1).all()
    keep = torch.ones(3, 4, dtype=torch.bool)
    keep[1, 1] = keep[0, 2] = keep[0, 3] = False
    assert torch.equal(ht.cpu()[keep], clean[1].cpu()[keep])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_row_in_two_calls(dtype):
    """A prompt split anywhere: the first call's final state is the second's initial one, in place."""
    q, k, v, g, beta, h0 = ref.delta_inputs(2, 150, 1, 2, 64, 32, dtype, seed=11)
    whole, ht = ref.delta_reference(q, k, v, g, beta, None, None, h0)
    for cut in (1, 64, 77, 149):
        state, outs = h0.cuda(), []
        for part in (slice(0, cut), slice(cut, 150)):
            a = [t[:, part] for t in gpu(q, k, v, g, beta)]
            o, s = ccv.gated_delta_rule_fwd(*a, initial_state=state, return_final_state=True, final_state_out=state)
            assert s is state
            outs.append(o)
        ref.assert_near("out", torch.cat(outs, 1), whole, 1, f"cut {cut}")
        ref.assert_near("state", state, ht, 1, f"cut {cut}")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Dk,Dv", WIDTHS)
@pytest.mark.parametrize("T", [1, 3])
def test_update(dtype, Dk, Dv, T):
    """New steps against a cache: slots in any order, idle rows, one step with and without its dimension."""
    B, slots = 5, 9
    q, k, v, g, beta, _ = ref.delta_inputs(B, T, 2, 4, Dk, Dv, dtype, "f32", "bf16", seed=Dk + T)
    state = torch.randn(slots, 4, Dk, Dv, generator=torch.Generator().manual_seed(3)) * 0.3
    idx = [7, -1, 0, 9, 3]                   # -1 and 9 name no slot
    cache = state.cuda()
    args = gpu(q, k, v, g, beta)
    if T == 1:
        args = [t[:, 0] for t in args]
    out = ccv.gated_delta_rule_update(*args, cache, state_indices=torch.tensor(idx, dtype=torch.int32).cuda())
    log(f"  update {dtype} {Dk}x{Dv} T={T}")
    live = [b for b in range(B) if 0 <= idx[b] < slots]
    want, wht = ref.delta_reference(*(t[live] for t in (q, k, v, g, beta)), None, None, state[[idx[b] for b in live]])
    out = out if T > 1 else out[:, None]
    ref.assert_near("out", out[live], want)
    assert not out[[1, 3]].any()
    ref.assert_near("state", cache[[idx[b] for b in live]], wht)
    rest = [s for s in range(slots) if s not in idx]
    assert torch.equal(cache[rest].cpu(), state[rest])
    # without indices row b is slot b
    cache = state.cuda()
    out = ccv.gated_delta_rule_update(*gpu(q, k, v, g, beta), cache)
    want, wht = ref.delta_reference(q, k, v, g, beta, None, None, state[:B])
    ref.assert_near("out", out, want)
    ref.assert_near("state", cache[:B], wht)


def test_update_in_a_cache_past_32_bits():
    """A slot whose state lies more than 2^32 elements into the cache."""
    q, k, v, g, beta, h0 = ref.delta_inputs(2, 1, 1, 2, 64, 32, "bf16", seed=5)
    far = (1 << 32) + 64
    buf = torch.empty(far + 2 * 64 * 32, dtype=torch.float32, device="cuda")
    cache = buf.as_strided((2, 2, 64, 32), (far, 64 * 32, 32, 1))
    cache.copy_(h0)
    out = ccv.gated_delta_rule_update(*gpu(q, k, v, g, beta), cache)
    want, wht = ref.delta_reference(q, k, v, g, beta, None, None, h0)
    ref.assert_near("out", out, want)
    ref.assert_near("state", cache, wht)


def test_decoding_continues_a_prompt():
    """Prefill, then steps one by one, as one long row."""
    q, k, v, g, beta, _ = ref.delta_inputs(2, 80, 1, 2, 64, 32, "bf16", "f32", "bf16", seed=12)
    want, wht = ref.delta_reference(q, k, v, g, beta)
    a = gpu(q, k, v, g, beta)
    out, state = ccv.gated_delta_rule_fwd(*(t[:, :70] for t in a), return_final_state=True)
    outs = [out] + [ccv.gated_delta_rule_update(*(t[:, i:i + 1] for t in a), state) for i in range(70, 80)]
    ref.assert_near("out", torch.cat(outs, 1), want)
    ref.assert_near("state", state, wht)


def test_empty_calls():
    for B, L in ((0, 5), (2, 0)):
        q, k, v, g, beta, h0 = ref.delta_inputs(B, L, 1, 2, 64, 32)
        out, ht = ccv.gated_delta_rule_fwd(*gpu(q, k, v, g, beta), initial_state=h0.cuda(), return_final_state=True)
        assert out.shape == (B, L, 2, 32) and torch.equal(ht.cpu(), h0)
        got = ccv.gated_delta_rule_bwd(*gpu(q, k, v, g, beta, v), initial_state=h0.cuda(), dfinal_state=h0.cuda(),
                                       return_dinitial_state=True)
        assert torch.equal(got[5].cpu(), h0)
    q, k, v, g, beta, h0 = ref.delta_inputs(1, 0, 1, 2, 64, 32, seqs=3)
    _, ht = ccv.gated_delta_rule_fwd(*gpu(q, k, v, g, beta), cu_seqlens=torch.zeros(4, dtype=torch.int32).cuda(),
                                     initial_state=h0.cuda(), return_final_state=True)
    assert torch.equal(ht.cpu(), h0)


@pytest.mark.parametrize("packed", [False, True])
def test_autograd(packed):
    q, k, v, g, beta, h0 = ref.delta_inputs(1 if packed else 2, 75, 1, 3, 64, 32, "f32", seed=13, seqs=2 if packed else None)
    lengths = [40, 35] if packed else None
    leaves = [t.cuda().requires_grad_() for t in (q, k, v, g, beta, h0)]
    out, ht = ccv.gated_delta_rule_fn(*leaves[:5], cu_seqlens=ref.cu_of(lengths).cuda() if packed else None,
                                      initial_state=leaves[5], return_final_state=True)
    gen = torch.Generator().manual_seed(2)
    dout, dht = torch.randn(v.shape, generator=gen), torch.randn(h0.shape, generator=gen)
    grads = torch.autograd.grad([out, ht], leaves, [dout.cuda(), dht.cuda()])
    want = ref.delta_gradients(q, k, v, g, beta, dout, None, lengths, h0, dht)
    for n, t in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), grads):
        ref.assert_near(n, t, want[n], 2)
    # only the final state is used
    out, ht = ccv.gated_delta_rule_fn(*leaves[:5], cu_seqlens=ref.cu_of(lengths).cuda() if packed else None,
                                      initial_state=leaves[5], return_final_state=True)
    grads = torch.autograd.grad(ht, leaves, dht.cuda())
    want = ref.delta_gradients(q, k, v, g, beta, torch.zeros_like(v), None, lengths, h0, dht)
    for n, t in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), grads):
        if n != "dq":
            ref.assert_near(n, t, want[n], 2)
    assert not grads[0].any()


def test_gradients_against_differences():
    """The kernel's gradients against differences of the kernel's own forward, along random
    directions.  A difference over 2 e = 0.02 has the outputs' rounding (2^-19 of |out| |dout|,
    over 0.02) and a curvature of e^2 times a third derivative of order 1: 2e-3 of the scale."""
    q, k, v, g, beta, h0 = ref.delta_inputs(1, 70, 1, 2, 64, 32, seed=21)
    x = gpu(q, k, v, g, beta, h0)
    gen = torch.Generator().manual_seed(4)
    dout, dht = torch.randn(v.shape, generator=gen).cuda(), torch.randn(h0.shape, generator=gen).cuda()
    got = ccv.gated_delta_rule_bwd(*x[:5], dout, initial_state=x[5], dfinal_state=dht, return_dinitial_state=True)

    def loss(a):
        o, s = ccv.gated_delta_rule_fwd(*a[:5], initial_state=a[5], return_final_state=True)
        return float((o.double() * dout).sum() + (s.double() * dht).sum())

    e = 0.01
    for i in range(6):
        d = torch.randn(x[i].shape, generator=gen).cuda()
        d = d / d.norm()
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + e * d, x[i] - e * d
        slope = (loss(up) - loss(down)) / (2 * e)
        want = float((got[i].double() * d).sum())
        assert abs(slope - want) <= 2e-3 * float(got[i].double().norm()) + 1e-3, (i, slope, want)


def test_repeats_bit_for_bit_and_on_another_stream():
    q, k, v, g, beta, h0 = ref.delta_inputs(2, 200, 2, 4, 128, 128, "bf16", seed=14)
    a = gpu(q, k, v, g, beta)
    dout = torch.randn(v.shape, generator=torch.Generator().manual_seed(1)).to(v.dtype).cuda()
    run = lambda: [*ccv.gated_delta_rule_fwd(*a, initial_state=h0.cuda(), return_final_state=True),  # noqa: E731
                   *ccv.gated_delta_rule_bwd(*a, dout, initial_state=h0.cuda(), return_dinitial_state=True)]
    first = run()
    for t, u in zip(first, run()):
        assert torch.equal(t, u)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run()
    side.synchronize()
    for t, u in zip(first, other):
        assert torch.equal(t, u)


def test_graph_replays_equal_eager():
    """Forward, backward and update captured in a graph, replayed with new inputs in between."""
    lengths = [100, 0, 50]
    cu = ref.cu_of(lengths).cuda()
    first = ref.delta_inputs(1, 160, 1, 2, 64, 32, "bf16", seed=30, seqs=3)
    a = gpu(*first)
    dout = torch.ones_like(a[2])
    cache = torch.zeros(1, 2, 64, 32, device="cuda")

    def work():
        o, s = ccv.gated_delta_rule_fwd(*a[:5], cu_seqlens=cu, initial_state=a[5], return_final_state=True)
        gr = ccv.gated_delta_rule_bwd(*a[:5], dout, cu_seqlens=cu, initial_state=a[5], return_dinitial_state=True)
        u = ccv.gated_delta_rule_update(*(t[:, 0] for t in a[:5]), cache)
        return [o, s, *gr, u]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = work()
    for r in range(3):
        for t, n in zip(a, ref.delta_inputs(1, 160, 1, 2, 64, 32, "bf16", seed=31 + r, seqs=3)):
            t.copy_(n)
        before = torch.randn(cache.shape, generator=torch.Generator().manual_seed(r)).cuda()
        cache.copy_(before)
        graph.replay()
        torch.cuda.synchronize()
        got, after = [t.clone() for t in static], cache.clone()
        cache.copy_(before)
        for t, u in zip(got, work()):
            assert torch.equal(t, u), r
        assert torch.equal(after, cache)


@pytest.mark.parametrize("heads", [2, 256])
def test_fp16_subnormals(heads):
    """Keys below fp16's normal range count in every product."""
    gen = torch.Generator().manual_seed(2)
    q, k, v, g, beta, h0 = ref.delta_inputs(1, 70, heads, heads, 64, 64, "f16", seed=3)
    k = (torch.randint(-60, 60, k.shape, generator=gen) * 2.0 ** -24).to(torch.float16)
    q = (q.float() * 3e4).to(torch.float16)
    check_fwd(q, k, v, g, beta, None, what="subnormal keys")
    check_fwd(k, q * 2.0 ** -15, v, g, beta, h0 * 2.0 ** -18, what="subnormal queries and small states")
    dout = (torch.randint(-60, 60, v.shape, generator=gen) * 2.0 ** -24).to(torch.float16)
    got = ccv.gated_delta_rule_bwd(*gpu(q, k, v, g, beta, dout), initial_state=h0.cuda(), return_dinitial_state=True)
    want = ref.delta_gradients(q, k, v, g, beta, dout, None, None, h0)
    for name, t in (("dq", got[0]), ("dg", got[3]), ("dbeta", got[4]), ("dh0", got[5])):
        ref.assert_near(name, t, want[name], 2)


# the same calls where 16-bit inputs take whole columns a wave, and where a sequence runs in parts
FORMS = [("columns", 16, 64, [5, 0, 64, 1, 130]), ("parts", 1, 2, [1100, 0, 1500])]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_padding_of_either_form(dtype, form):
    """Steps behind the last sequence are not looked at, and give zeros."""
    what, Hk, Hv, lengths = FORMS[form]
    live = sum(lengths)
    q, k, v, g, beta, h0 = ref.delta_inputs(1, live + 70, Hk, Hv, 64, 48, dtype, seed=form, seqs=len(lengths), decay=0.05)
    dout = torch.randn(v.shape, generator=torch.Generator().manual_seed(1)).to(v.dtype)
    bad = [t.clone() for t in (q, k, v, g, beta, dout)]
    for t in bad:
        t[:, live:] = NAN
    cu = ref.cu_of(lengths).cuda()
    out, ht = ccv.gated_delta_rule_fwd(*gpu(*bad[:5]), cu_seqlens=cu, initial_state=h0.cuda(), return_final_state=True)
    got = ccv.gated_delta_rule_bwd(*gpu(*bad), cu_seqlens=cu, initial_state=h0.cuda(), return_dinitial_state=True)
    want = ref.delta_gradients(q, k, v, g, beta, dout, None, lengths, h0)
    ref.assert_near("out", out, want["out"], 1, what)
    ref.assert_near("final_state", ht, want["ht"], 1, what)
    for name, t in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got):
        ref.assert_near(name, t, want[name], 2, what)
        if name != "dh0":
            assert not t[:, live:].any(), name


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,L,Hk,Hv", [(16, 70, 8, 16), (1, 1100, 1, 2)])
def test_strides_of_either_form(dtype, B, L, Hk, Hv):
    """Views of one wider buffer at odd offsets, heads first, outputs with a stride of their own, in place states."""
    Dk, Dv = 64, 61
    q, k, v, g, beta, h0 = ref.delta_inputs(B, L, Hk, Hv, Dk, Dv, dtype, seed=4, decay=0.05)
    off = 3
    buf = torch.full((B, L, off + 2 * Hk * Dk + Hv * Dv + 1), NAN, dtype=q.dtype, device="cuda")
    a, b = off + Hk * Dk, off + 2 * Hk * Dk
    views = [buf[..., off:a].unflatten(2, (Hk, Dk)), buf[..., a:b].unflatten(2, (Hk, Dk)), buf[..., b:b + Hv * Dv].unflatten(2, (Hv, Dv))]
    for view, t in zip(views, (q, k, v)):
        view.copy_(t)
    check_fwd(q, k, v, g, beta, h0, what="fused", views=views + gpu(g, beta))
    check_bwd(q, k, v, g, beta, h0, what="fused", views=views + gpu(g, beta))
    views = [t.cuda().transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v, g, beta)]
    check_bwd(q, k, v, g, beta, h0, what="heads first", views=views)
    state = h0.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    out, s = ccv.gated_delta_rule_fwd(*views, initial_state=state, return_final_state=True, final_state_out=state)
    want, wht = ref.delta_reference(q, k, v, g, beta, None, None, h0)
    ref.assert_near("out", out, want)
    ref.assert_near("final_state", state, wht)


@pytest.mark.parametrize("B,L,H", [(16, 130, 16), (1, 1300, 1)])
def test_either_form_repeats_and_replays(B, L, H):
    """Bit for bit: again, on another stream, and in a graph replayed with new inputs."""
    first = ref.delta_inputs(B, L, H, H, 64, 64, "f16", seed=30, decay=0.05)
    a = gpu(*first)
    dout = torch.ones_like(a[2])

    def work():
        o, s = ccv.gated_delta_rule_fwd(*a[:5], initial_state=a[5], return_final_state=True)
        return [o, s, *ccv.gated_delta_rule_bwd(*a[:5], dout, initial_state=a[5], return_dinitial_state=True)]

    once = work()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t, u in zip(once, work()):
            assert torch.equal(t, u)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = work()
    for r in range(3):
        for t, n in zip(a, ref.delta_inputs(B, L, H, H, 64, 64, "f16", seed=31 + r, decay=0.05)):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        for t, u in zip([t.clone() for t in static], work()):
            assert torch.equal(t, u), r
