"""Corners of the gated linear recurrence, group norm and rotary positions on the GPU, against their 64-bit
forms, element by element within the bounds derived in recurrent_reference."""
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
from test_gpu_group_norm import check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,groups,width,dtype,weight,gated", [(64, 131072, 1, "bf16", "f32", True), (66, 140001, 2, "f32", "f32", False),
                                                                  (65, 131073, 3, "f16", "f16", True)])
def test_group_norm_of_very_many_narrow_groups(rows, groups, width, dtype, weight, gated):
    x, w, b, z, dout = inputs(rows, groups * width, dtype, weight, gated, groups)
    check(f"{rows} rows of {groups} groups of {width}", x, groups, w, b, z, dout, "silu")


def test_norms_without_values():
    x = torch.zeros(2, 3, 0).cuda()
    out, mean, rstd = ccv.group_norm_fwd(x, 4, gate=x, activation="silu", return_stats=True)
    assert out.shape == x.shape and mean.shape == rstd.shape == (2, 3, 4) and bool((mean.isnan() & rstd.isnan()).all())
    y = x.clone().requires_grad_()
    ccv.group_norm_fn(y, 4).sum().backward()
    assert y.grad.shape == y.shape
    out, mean, rstd = ccv.layer_norm_fwd(x, return_stats=True)
    assert out.shape == x.shape and mean.shape == rstd.shape == (2, 3) and bool((mean.isnan() & rstd.isnan()).all())


@pytest.mark.parametrize("wanted", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("weight", ["f32", "f16", "bf16"])
def test_gradients_in_a_type_of_the_callers(weight, wanted):
    """The 32-bit sums of a call with the weight's values in 32 bits, rounded once."""
    x, w, b, z, dout = (t.cuda() for t in inputs(300, 96, "bf16", weight, True, 5))
    o, mean, rstd = ccv.group_norm_fwd(x, 3, w, b, z, "silu", return_stats=True)
    wide = ccv.group_norm_bwd(x, 3, w.float(), b.float(), dout, mean, rstd, z, "silu")
    got = ccv.group_norm_bwd(x, 3, w, b, dout, mean, rstd, z, "silu", weight_dtype=wanted)
    assert torch.equal(got[0], wide[0]) and torch.equal(got[3], wide[3])
    assert torch.equal(got[1], wide[1].to(wanted)) and torch.equal(got[2], wide[2].to(wanted))
    o, mean, rstd = ccv.layer_norm_fwd(x, w, b, return_stats=True)
    wide = ccv.layer_norm_bwd(x, w.float(), dout, mean, rstd)
    got = ccv.layer_norm_bwd(x, w, dout, mean, rstd, weight_dtype=wanted)
    assert torch.equal(got[0], wide[0]) and torch.equal(got[1], wide[1].to(wanted)) and torch.equal(got[2], wide[2].to(wanted))
