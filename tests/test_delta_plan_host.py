"""The delta rule's choice of kernels, which the backward's workspace shows: it holds partial sums for every slice of
the values, of 16 or 32 in the pass from the end and in the forward one.  (CPU)"""
import pytest

import causal_depthwise_conv1d_amd as ccv
from test_layer_host import bwd


def size(B, H, dtype, chunks=96):
    """Backward workspace of B rows of H heads with `chunks` groups of 64 steps in all."""
    need = ccv.ccv_delta_bwd_workspace_size(bwd(B=B, L=64 * chunks // B, Hk=H, Hv=H, Dk=128, Dv=128, x_dtype=dtype))
    assert need > 0
    return need


def slices(B, H, dtype):
    """(slices of the pass from the end, of the forward one) by what the workspace has beside the rest, whose size is that of
    fp32, which takes 8 slices of each."""
    rest = size(B, H, ccv.CCV_F32) - 96 * H * 4 * 8 * (192 + 64)
    left = (size(B, H, dtype) - rest) // (96 * H * 4)
    return next((p, q) for p in (4, 8) for q in (4, 8) if 192 * p + 64 * q == left)


@pytest.mark.parametrize("dtype", [ccv.CCV_BF16, ccv.CCV_F16])
@pytest.mark.parametrize("heads", [16, 24, 32, 40, 64, 72, 96, 128, 192])
def test_rows_and_heads_count_alike(dtype, heads):
    """One row of many heads is as many blocks of values as several rows of fewer."""
    assert len({slices(B, heads // B, dtype) for B in (1, 2, 4)}) == 1


@pytest.mark.parametrize("B", [1, 2, 8])
def test_bounds(B):
    """Blocks of 16 values: 32 a workgroup from 257 blocks on, whole columns a wave forward from 513 on."""
    for blocks, forward, back in ((128, 8, 8), (256, 8, 8), (320, 4, 4), (512, 4, 4), (576, 8, 4), (1024, 8, 4)):
        assert slices(B, blocks // 8 // B, ccv.CCV_BF16) == (back, forward), blocks
