"""Group norm with an activation or a gate on the GPU against its 64-bit form, element by element within the
bounds derived in recurrent_reference."""
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
import recurrent_reference as ref
from gpu_support import log
from layer_reference import DT

pytestmark = pytest.mark.gpu

# of a width's threads and vectors: narrower than one, each number of lanes, whole and partial vectors, wider than 256 threads hold
WIDTHS = [1, 2, 3, 5, 7, 8, 9, 15, 16, 31, 32, 33, 64, 65, 100, 128, 129, 200, 256, 257, 500, 512, 600, 1000, 1024, 1500, 2048,
          2100, 4096, 5000, 8192, 9001]


def inputs(rows, C, dtype, weight, gated, seed):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = (rand(rows, C) * 1.5 + 0.3).to(DT[dtype])
    w, b = (None, None) if weight is None else ((1 + 0.2 * rand(C)).to(DT[weight]), (0.3 * rand(C)).to(DT[weight]))
    return x, w, b, (2 * rand(rows, C)).to(DT[dtype]) if gated else None, rand(rows, C).to(DT[dtype])


def cuda(t):
    return None if t is None else t.cuda()


def check(what, x, groups, w, b, z, dout, activation, eps=1e-5, views=None):
    want = ref.group_norm(x, groups, w, b, z, activation is not None, eps, dout)
    xs, zs, ds = views or (x.cuda(), cuda(z), dout.cuda())
    o, mean, rstd = ccv.group_norm_fwd(xs, groups, cuda(w), cuda(b), zs, activation, eps, return_stats=True)
    dx, dw, db, dz = ccv.group_norm_bwd(xs, groups, cuda(w), cuda(b), ds, mean, rstd, zs, activation)
    got = {"out": o, "mean": mean, "rstd": rstd, "dx": dx, "dw": dw, "db": db, "dz": dz}
    for n in want:
        ref.assert_within(n, got[n].reshape(want[n][0].shape), want[n], what)
    log(f"  {what}: within the bounds")
    return got


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype,weight", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16")])
def test_widths(width, dtype, weight):
    for groups, gated, activation in ((3, True, "silu"), (2, False, "silu")):
        x, w, b, z, dout = inputs(5, groups * width, dtype, weight, gated, width)
        check(f"width {width} {dtype}", x, groups, w, b, z, dout, activation)


@pytest.mark.parametrize("rows", [1, 2, 3, 63, 500, 4099])
@pytest.mark.parametrize("groups", [1, 2, 5, 16, 20, 33])
def test_rows_and_groups(rows, groups):
    x, w, b, z, dout = inputs(rows, groups * 24, "bf16", "f32", True, rows + groups)
    check(f"{rows} rows {groups} groups", x, groups, w, b, z, dout, "swish")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("weight", [None, "f32", "f16", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("activation", [None, "silu"])
def test_forms(dtype, weight, gated, activation):
    x, w, b, z, dout = inputs(70, 4 * 64, dtype, weight, gated, 3)
    check("both", x, 4, w, b, z, dout, activation)
    if weight:
        check("weight alone", x, 4, w, None, z, dout, activation)
        check("bias alone", x, 4, None, b, z, dout, activation)


def test_strides():
    x, w, b, z, dout = inputs(6 * 7, 90, "f16", "f16", True, 4)
    buf = torch.zeros(6, 7, 300, dtype=torch.float16).cuda()
    buf[..., 1:91], buf[..., 95:185], buf[..., 201:291] = (t.view(6, 7, 90).cuda() for t in (x, z, dout))
    views = buf[..., 1:91], buf[..., 95:185], buf[..., 201:291]
    a = check("slices", x, 3, w, b, z, dout, "silu", views=views)
    assert a["out"].shape == (6, 7, 90) and a["mean"].shape == (6, 7, 3)
    # leading dimensions that lie at no one stride, and channels at none: copied
    t = [v.transpose(0, 1) for v in views]
    o = ccv.group_norm_fwd(t[0], 3, w.cuda(), b.cuda(), t[1], "silu")
    assert torch.equal(o, a["out"].transpose(0, 1))
    c = [v.transpose(1, 2).contiguous().transpose(1, 2) for v in views]
    assert torch.equal(ccv.group_norm_fwd(c[0], 3, w.cuda(), b.cuda(), c[1], "silu"), a["out"])
    # one gate for all rows
    one = z[:1].expand(42, -1)
    check("broadcast gate", x, 3, w, b, one, dout, "silu", views=(x.cuda(), z[:1].cuda().expand(42, -1), dout.cuda()))


def test_constant_groups():
    """A variance of 0: n is 0 (or what rounding of the mean leaves), and rstd is eps^-1/2."""
    x, w, b, z, dout = inputs(4, 64, "f32", "f32", True, 5)
    x[:, :32] = 3.0
    got = check("constant", x, 2, w, b, z, dout, "silu", eps=1e-3)
    assert bool(torch.isfinite(got["dx"]).all())


def test_far_from_zero():
    """The variance is summed from deviations: a mean a thousand times the spread costs what its rounding does."""
    x, w, b, z, dout = inputs(9, 256, "f32", "f32", False, 6)
    check("far", x + 1000, 2, w, b, z, dout, None)


def test_saturated_gates():
    x, w, b, z, dout = inputs(9, 256, "f32", "f32", True, 7)
    z *= 60
    got = check("saturated", x, 2, w, b, z, dout, "silu")
    z[0, :4] = torch.tensor([1e4, -1e4, 1e30, -1e30])
    o = ccv.group_norm_fwd(x.cuda(), 2, w.cuda(), b.cuda(), z.cuda(), "silu")
    assert torch.equal(o[1:], got["out"][1:]) and bool((o[0, [1, 3]] == 0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_group(bad):
    x, w, b, z, dout = (t.cuda() for t in inputs(9, 96, "f32", "f32", True, 8))
    clean = ccv.group_norm_fwd(x, 3, w, b, z, "silu")
    x[4, 40] = bad
    o, mean, rstd = ccv.group_norm_fwd(x, 3, w, b, z, "silu", return_stats=True)
    dx = ccv.group_norm_bwd(x, 3, w, b, dout, mean, rstd, z, "silu")[0]
    same = torch.ones_like(clean, dtype=torch.bool)
    same[4, 32:64] = False
    assert torch.equal(o[same], clean[same]) and not bool(torch.isfinite(o[~same]).any())
    assert bool(torch.isfinite(dx[same]).all())


def test_empty():
    for shape, groups in (((0, 8), 2), ((3, 0, 8), 1)):
        x = torch.zeros(shape).cuda()
        w = torch.ones(8).cuda()
        o, mean, rstd = ccv.group_norm_fwd(x, groups, w, w, return_stats=True)
        dx, dw, db, dz = ccv.group_norm_bwd(x, groups, w, w, x, mean, rstd)
        assert o.shape == dx.shape == x.shape and dz is None
        assert torch.equal(dw, torch.zeros(8).cuda()) and torch.equal(db, dw)


def test_wanted_alone():
    x, w, b, z, dout = (t.cuda() for t in inputs(100, 96, "bf16", "f32", True, 9))
    o, mean, rstd = ccv.group_norm_fwd(x, 3, w, b, z, "silu", return_stats=True)
    every = ccv.group_norm_bwd(x, 3, w, b, dout, mean, rstd, z, "silu")
    for i in range(4):
        want = [i == j for j in range(4)]
        one = ccv.group_norm_bwd(x, 3, w, b, dout, mean, rstd, z, "silu", *want)
        for j in range(4):
            assert (one[j] is None) if j != i else torch.equal(one[j], every[j])


def test_long_sums_and_repeats():
    """dweight and dbias over many rows, the same bits each time."""
    x, w, b, z, dout = inputs(70000, 4 * 8, "f32", "f32", True, 10)
    first = check("70000 rows", x, 4, w, b, z, dout, "silu")
    again = check("70000 rows", x, 4, w, b, z, dout, "silu")
    assert all(torch.equal(first[n], again[n]) for n in first)


def test_autograd_streams_and_graphs():
    x, w, b, z, dout = inputs(300, 5 * 40, "f32", "f32", True, 11)
    want = ref.group_norm(x, 5, w, b, z, True, 1e-5, dout)
    leaves = [t.cuda().requires_grad_() for t in (x, w, b, z)]

    def run():
        y = ccv.group_norm_fn(leaves[0], 5, leaves[1], leaves[2], leaves[3], "silu")
        return (y.detach(), *torch.autograd.grad(y, leaves, dout_gpu))
    dout_gpu = dout.cuda()
    eager = run()
    for n, t in zip(("out", "dx", "dw", "db", "dz"), eager):
        ref.assert_within(n, t, want[n])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(other, eager))
    args = [t.detach() for t in leaves]

    def call():
        o, mean, rstd = ccv.group_norm_fwd(args[0], 5, *args[1:3], args[3], "silu", return_stats=True)
        return (o, *ccv.group_norm_bwd(args[0], 5, *args[1:3], dout_gpu, mean, rstd, args[3], "silu"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = call()
    for _ in range(3):
        args[0].copy_(torch.randn_like(args[0]))
        now = [t.clone() for t in call()]
        for t in res:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(res, now))
