"""Layer norm's dweight and dbias over very many rows, of terms of one sign: the sums are split often enough that no
chain of fp32 additions is long.

A chain of n additions of terms of one sign is within n 2^-24 of its sum.  Where rows are held in registers, a sum
passes through at most 1024 additions of rows, 16 over a workgroup's rows, 128 + 8 over partial rows, 5 over the threads
that share them, and a rounding: fewer than 1200.  Where they are not, 128 of rows, then 25 more for such runs, 128, 5
and 1: fewer than 320.  dweight's terms are rounded too, and n has rstd's error, 2^-18 as in the other tests of
layer norm."""
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
from gpu_support import log

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    ccv.lib()


@pytest.mark.parametrize("width,rows,dtype,chain", [(3, 1_000_000, torch.float32, 320), (1, 3_000_000, torch.float32, 320), (7, 3_000_001, torch.bfloat16, 320),
                                                    (8, 1 << 28, torch.float16, 1200), (200, 20_000_000, torch.float16, 1200),
                                                    (20001, 200_000, torch.bfloat16, 320), (12000, 200_000, torch.float32, 320)])
def test_sums_of_one_sign(width, rows, dtype, chain):
    log(f"  {rows} rows of {width} in {dtype}")
    x = torch.linspace(-1, 2, width).to(dtype).cuda().expand(rows, width)       # one row, seen `rows` times
    d = torch.full((width,), 0.7, dtype=dtype, device="cuda").expand(rows, width)
    one = x[0].double()
    mean = one.mean()
    rstd = ((one - mean).square().mean() + 1e-5).rsqrt()
    stats = [t.float().expand(rows).contiguous() for t in (mean, rstd)]
    _, dw, db = ccv.layer_norm_bwd(x, None, d, *stats, want_dx=False, weight_dtype=torch.float32)
    db0 = rows * d[0].double()
    assert bool(((db.double() - db0).abs() <= chain * 2.0 ** -24 * db0).all()), ((db.double() / db0 - 1).abs().max() * 2 ** 24)
    dw0 = db0 * (one - stats[0][0].double()) * stats[1][0].double()
    assert bool(((dw.double() - dw0).abs() <= (chain * 2.0 ** -24 + 2.0 ** -18) * dw0.abs() + 2.0 ** -24 * rows).all())
