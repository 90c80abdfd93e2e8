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


def test_group_norm_without_channels():
    x = torch.zeros(2, 3, 0).cuda()
    out, mean, rstd = ccv.group_norm_fwd(x, 4, gate=x, activation="silu", return_stats=True)
    assert out.shape == x.shape and mean.shape == rstd.shape == (2, 3, 4) and bool((mean.isnan() & rstd.isnan()).all())
    y = x.clone().requires_grad_()
    ccv.group_norm_fn(y, 4).sum().backward()
    assert y.grad.shape == y.shape
