"""Layer norm and the sequence tables on the GPU against their 64-bit forms.

Tolerances: a row of width w is summed in fp32 by at most 512 threads, each over at most w / 16
elements, then by a tree: the statistics are within 2^-20 of the row's largest deviation plus
2^-22 of its mean (rounding of x - mean), so an fp32 element is within 2^-18 (|n w| + |w|), and
rounds once more in 16 bits.  dx has three such terms with |dout w rstd| as their scale; column
sums over r rows are within 2^-20 sqrt(r) of the largest term, plus their own rounding."""
import ctypes

import numpy as np
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
import layer_reference as ref
from gpu_support import log

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    ccv.lib()

WIDTHS = [1, 2, 3, 7, 8, 9, 16, 63, 64, 65, 100, 128, 129, 511, 512, 2048, 2560, 4096, 5000, 8192, 16384, 16385, 20001]


def data(rows, width, dtype, wdt, seed=0, shift=0.3):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, width, generator=g) * 1.5 + shift).to(ref.DT[dtype])
    w = (1 + 0.2 * torch.randn(width, generator=g)).to(ref.DT[wdt])
    b = (0.3 * torch.randn(width, generator=g)).to(ref.DT[wdt])
    d = torch.randn(rows, width, generator=g).to(x.dtype)
    return x, w, b, d


def close(name, got, want, scale, what=""):
    """|got - want| within rounding of the result plus 2^-18 of `scale`, element by element."""
    g = got.detach().cpu().double()
    assert g.shape == want.shape
    lim = ref.half_spacing(got.dtype, want) + 2.0 ** -18 * scale
    over = ((g - want).abs() - lim)
    assert bool((over <= 0).all()), f"{what} {name}: {float(over.max()):.3g} over the limit"


def reference(x, w, b, d, eps):
    x, d = x.double(), d.double()
    mean = x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + eps)
    n = (x - mean) * r
    wd = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    a = d * wd
    dx = r * (a - a.mean(-1, keepdim=True) - n * (a * n).mean(-1, keepdim=True))
    flat = lambda t: t.reshape(-1, x.shape[-1])  # noqa: E731
    return {"out": n * wd + (0 if b is None else b.double()), "n": n, "mean": mean[..., 0], "rstd": r[..., 0], "dx": dx, "a": a,
            "dw": flat(d * n).sum(0), "db": flat(d).sum(0), "dn": flat(d * n), "d": flat(d), "wd": wd, "r": r}


def check(x, w, b, d, eps=1e-5, what="", xv=None, dv=None):
    log(f"  norm {what} {tuple(x.shape)} {x.dtype}")
    R = reference(x, w, b, d, eps)
    wg, bg = (None if t is None else t.cuda() for t in (w, b))
    xv = x.cuda() if xv is None else xv
    dv = d.cuda() if dv is None else dv
    out, mean, rstd = ccv.layer_norm_fwd(xv, wg, bg, eps, return_stats=True)
    assert torch.equal(out, ccv.layer_norm_fwd(xv, wg, bg, eps))
    scale = (R["n"].abs() + 1) * R["wd"].abs() + (0 if b is None else b.double().abs())
    close("out", out, R["out"], scale, what)
    close("mean", mean, R["mean"], x.double().abs().amax(-1), what)
    close("rstd", rstd, R["rstd"], R["rstd"], what)
    dx, dw, db = ccv.layer_norm_bwd(xv, wg, dv, mean, rstd)
    s = R["r"] * (R["a"].abs().amax(-1, keepdim=True) * (1 + R["n"].abs())) * 4
    close("dx", dx, R["dx"], s, what)
    rows = max(1, x.numel() // x.shape[-1])
    for name, t, terms in (("dw", dw, R["dn"].abs() + R["d"].abs()), ("db", db, R["d"].abs())):
        close(name, t, R[name], terms.amax(0) * rows ** 0.5, what)
    return dx, dw, db


@pytest.mark.parametrize("dtype,wdt", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(dtype, wdt, width):
    for rows in (1, 5, 70):
        check(*data(rows, width, dtype, wdt, seed=width + rows), what=f"{rows} rows")


@pytest.mark.parametrize("rows", [2, 255, 256, 1025, 5000, 40000])
def test_many_rows(rows):
    check(*data(rows, 128, "bf16", "f32", seed=rows), what="heads")
    if rows <= 5000:
        check(*data(rows, 300, "f32", "f32", seed=rows), what="odd")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_views(dtype):
    """Rows inside wider buffers, at odd offsets, heads before steps, one row for all, more dimensions."""
    x, w, b, d = data(6 * 10, 72, dtype, "f32", seed=1)
    x3, d3 = x.view(6, 10, 72), d.view(6, 10, 72)
    for off, pad in ((0, 8), (3, 1), (1, 0)):
        buf = torch.full((6, 10, off + 72 + pad), float("nan"), dtype=x.dtype, device="cuda")
        dbuf = buf.clone()
        xv, dv = buf[..., off:off + 72], dbuf[..., off:off + 72]
        xv.copy_(x3)
        dv.copy_(d3)
        check(x3, w, b, d3, what=f"offset {off}", xv=xv, dv=dv)
    xv = x3.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    check(x3, w, b, d3, what="heads first", xv=xv, dv=d3.cuda().transpose(0, 1).contiguous().transpose(0, 1))
    check(x3[:1, :1].expand(6, 10, 72), w, b, d3, what="broadcast", xv=x3[:1, :1].cuda().expand(6, 10, 72))
    check(x.view(2, 3, 10, 72), w, b, d.view(2, 3, 10, 72), what="4 dims")
    check(x[0], w, b, d[0], what="1 dim")
    xt = x.t().contiguous().t().cuda()            # no unit stride along the width: copied
    check(x, w, b, d, what="transposed", xv=xt)


def test_without_weight_or_bias():
    x, w, b, d = data(20, 200, "bf16", "f32")
    check(x, None, None, d, what="plain")
    check(x, w, None, d, what="no bias")
    check(x, None, b, d, what="no weight")
    _, mean, rstd = ccv.layer_norm_fwd(x.cuda(), return_stats=True)
    dx, dw, db = ccv.layer_norm_bwd(x.cuda(), None, d.cuda(), mean, rstd, True, False, False)
    assert dw is None and db is None and dx is not None
    dx, dw, db = ccv.layer_norm_bwd(x.cuda(), None, d.cuda(), mean, rstd, False, True, True, torch.float32)
    assert dx is None and dw.dtype == torch.float32


def test_rows_at_their_ends():
    """Constant rows, rows far from zero, values of the type's ends, NaN and infinities in one row."""
    x, w, b, d = data(8, 256, "f32", "f32")
    x[1] = 3.25                                    # no variance: out is the bias
    x[2] += 1000.0                                 # the deviations still count: they are summed, not squares
    out, mean, rstd = ccv.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda(), return_stats=True)
    assert torch.equal(out[1].cpu(), b)
    R = reference(x, w, b, d, 1e-5)
    # x - mean is exact to 2^-24 of 1000, a deviation of 1.5 then to 2^-15
    assert (out[2].cpu().double() - R["out"][2]).abs().max() < 2.0 ** -14 * 8
    y = x.clone()
    y[5, 100], y[6, 7] = float("nan"), float("inf")
    bad, _, _ = ccv.layer_norm_fwd(y.cuda(), w.cuda(), b.cuda(), return_stats=True)
    keep = [0, 1, 2, 3, 4, 7]
    assert torch.equal(bad[keep], out[keep]) and torch.isnan(bad[5:7]).all()
    z = torch.full((2, 256), 65504.0, dtype=torch.float16)
    z[1, ::2] = -65504.0
    out = ccv.layer_norm_fwd(z.cuda())
    assert torch.equal(out.cpu()[0], torch.zeros(256, dtype=torch.float16))
    assert torch.equal(out.cpu()[1].float().abs(), torch.ones(256))


def test_no_rows_and_no_width():
    w = torch.ones(16, device="cuda")
    x = torch.empty(0, 16, device="cuda")
    out, mean, rstd = ccv.layer_norm_fwd(x, w, w, return_stats=True)
    assert out.shape == (0, 16) and mean.shape == (0,)
    dx, dw, db = ccv.layer_norm_bwd(x, w, x, mean, rstd)
    assert dx.shape == (0, 16) and not dw.any() and not db.any()
    assert ccv.layer_norm_fwd(torch.empty(3, 0, device="cuda")).shape == (3, 0)


def test_autograd_differences_repeats_and_streams():
    x, w, b, d = data(30, 200, "f32", "f32", seed=8)
    xs, ws, bs = (t.cuda().requires_grad_() for t in (x, w, b))
    grads = torch.autograd.grad(ccv.layer_norm_fn(xs, ws, bs), [xs, ws, bs], d.cuda())
    R = reference(x, w, b, d, 1e-5)
    for t, n in zip(grads, ("dx", "dw", "db")):
        assert (t.cpu().double() - R[n]).norm() <= 2.0 ** -18 * R[n].norm()
    loss = lambda a: float((ccv.layer_norm_fwd(*a).double() * d.cuda()).sum())  # noqa: E731
    gen, e = torch.Generator().manual_seed(1), 0.01
    args = [x.cuda(), w.cuda(), b.cuda()]
    for i in range(3):      # rounding 2^-19 |out| |d| / 0.02 and curvature e^2
        u = torch.randn(args[i].shape, generator=gen).cuda()
        u = u / u.norm()
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + e * u, args[i] - e * u
        want = float((grads[i].double() * u).sum())
        assert abs((loss(up) - loss(down)) / (2 * e) - want) <= 2e-3 * float(grads[i].double().norm()) + 1e-2
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        xt, wt, bt = (t.cuda().requires_grad_() for t in (x, w, b))
        other = torch.autograd.grad(ccv.layer_norm_fn(xt, wt, bt), [xt, wt, bt], d.cuda())
    side.synchronize()
    for t, u in zip(grads, other):
        assert torch.equal(t, u)


def test_norm_graph_replays_equal_eager():
    x, w, b, d = (t.cuda() for t in data(300, 512, "bf16", "f32", seed=2))

    def work():
        o, m, r = ccv.layer_norm_fwd(x, w, b, return_stats=True)
        return [o, *ccv.layer_norm_bwd(x, w, d, m, r)]

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
        for t, n in zip((x, w, b, d), data(300, 512, "bf16", "f32", seed=3 + r)):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        for t, u in zip([t.clone() for t in static], work()):
            assert torch.equal(t, u)


TABLES = [([], 0), ([], 5), ([0], 1), ([3], 3), ([3], 10), ([0, 0, 4, 0], 4), ([5, -2, 5], 8), ([4, 4, 4], 6),
          ([1] * 3000, 3000), ([1, 0] * 1500, 5000), ([100000], 100000), ([4095, 1, 4096, 3], 9000), ([2 ** 31 - 1, 5], 5000)]


@pytest.mark.parametrize("i", range(len(TABLES)))
def test_tables(i):
    lengths, total = TABLES[i]
    cu, seq, pos = ccv.sequence_tables(torch.tensor(lengths, dtype=torch.int32).cuda(), total)
    want = ref.tables_reference(lengths, total)
    for got, w in zip((cu, seq[0], pos[0]), want):
        assert np.array_equal(got.cpu().numpy(), w)


def test_tables_of_a_random_row():
    g = np.random.default_rng(5)
    for n, total in ((1, 7), (1023, 70000), (1024, 70000), (1025, 300000), (5000, 1 << 20)):
        lengths = g.integers(0, 2 * total // n + 1, n).astype(np.int32)
        lengths[g.integers(0, n, n // 8)] = 0
        cu, seq, pos = ccv.sequence_tables(torch.from_numpy(lengths).cuda(), total)
        for got, w in zip((cu, seq[0], pos[0]), ref.tables_reference(lengths.tolist(), total)):
            assert np.array_equal(got.cpu().numpy(), w), (n, total)


def test_tables_at_any_address():
    """The low-level call with outputs 4 bytes off a 16-byte boundary."""
    lengths = torch.tensor([70, 0, 5000, 3, 4096], dtype=torch.int32).cuda()
    total = 9300
    buf = [torch.full((total + 8,), -7, dtype=torch.int32, device="cuda") for _ in range(3)]
    a = ccv.ccv_seq_tables_args_t(struct_size=ctypes.sizeof(ccv.ccv_seq_tables_args_t), N=5, total=total, lengths=lengths.data_ptr(),
                                  cu_seqlens=buf[0].data_ptr() + 4, seq_idx=buf[1].data_ptr() + 4, positions=buf[2].data_ptr() + 12)
    assert ccv.ccv_seq_tables(a) == 0
    torch.cuda.synchronize()
    cu, seq, pos = ref.tables_reference(lengths.tolist(), total)
    for t, at, w in ((buf[0], 1, cu), (buf[1], 1, seq), (buf[2], 3, pos)):
        got = t.cpu().numpy()
        assert np.array_equal(got[at:at + len(w)], w)
        assert (got[:at] == -7).all() and (got[at + len(w):] == -7).all()
