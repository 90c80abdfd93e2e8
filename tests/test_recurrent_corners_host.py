"""Corners of the gated linear recurrence, group norm and rotary positions, on the CPU."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
from test_recurrent_host import CALLS, calls_do_nothing  # noqa: F401


# ---- the frequencies of stretched contexts ---------------------------------------------------

def plain(turned, base):
    return torch.tensor([base ** (-2 * i / turned) for i in range(turned // 2)], dtype=torch.float64)


@pytest.mark.parametrize("turned,base,length", [
    (128, 10000.0, 2048), (128, 10000.0, 54000), (128, 10000.0, 65536), (128, 10000.0, 131072), (128, 10000.0, 1 << 24),
    (64, 500000.0, 8192), (64, 500000.0, 1 << 23), (4, 10000.0, 2048), (2, 10000.0, 2048), (16, 100.0, 4096), (128, 10000.0, 100)])
def test_parts_is_a_ramp_over_pairs(turned, base, length):
    """The share of a frequency that stays: 1 up to the last whole pair before the one of 32 turns, 0 from the first whole pair behind
    that of one turn on, wherever these lie, and straight between."""
    factor = 8.0
    f, scale = ccv.rotary_frequencies(turned, base, "parts", factor, length, device="cpu")
    assert math.isclose(scale, 0.1 * math.log(factor) + 1)
    at = [turned * math.log(length / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32.0, 1.0)]
    first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), turned - 1)
    for i, w in enumerate(plain(turned, base).tolist()):
        stays = 1.0 if i <= first else 0.0 if i >= last else 1 - (i - first) / (last - first)
        assert math.isclose(float(f[i]), w * (stays + (1 - stays) / factor), rel_tol=1e-13), (i, first, last)


def test_parts_divides_no_pair_whole_that_makes_a_turn():
    """131072 steps: the slowest of 64 pairs makes 2.4 turns, so it keeps a share; over 2^24 steps it makes more than 32, and every pair stays."""
    want = plain(128, 10000.0)
    f, _ = ccv.rotary_frequencies(128, scaling="parts", factor=8, original_length=131072, device="cpu")
    turns = 131072 * want / (2 * math.pi)
    assert float(turns[-1]) > 2 and bool((f[turns > 1.4] > want[turns > 1.4] / 8 * 1.01).all())
    f, _ = ccv.rotary_frequencies(128, scaling="parts", factor=8, original_length=1 << 24, device="cpu")
    assert torch.equal(f, want)


# ---- the recurrence's sizes ------------------------------------------------------------------

@pytest.mark.parametrize("B,C", [(2 ** 30, 256), (2 ** 26, 4096), (2 ** 31 - 1, 2 ** 24), (2 ** 31 - 1, 1), (1, 1)])
@pytest.mark.parametrize("call", ["ccv_linrec_fwd", "ccv_linrec_bwd"])
def test_no_steps_of_many_rows(call, B, C):
    """Without steps there are no tiles, so that no number of rows and channels is too many for them: the calls need no workspace and do nothing."""
    args = CALLS[call](B=B, L=0, C=C, workspace=None, workspace_bytes=0)
    assert ccv.STATUS[getattr(ccv, call + "_check")(args)] == "CCV_OK"
    assert getattr(ccv, call + "_workspace_size")(args) == 0
    assert getattr(ccv.lib(), call)(ctypes.byref(args), None) == 0


@pytest.mark.parametrize("B,L,C", [(2 ** 23 - 1, 1, 64), (2 ** 22 - 1, 128, 65), (65535, 1, 8192), (1, 128 * (2 ** 23 - 1), 1), (31, 128 * 31, 64 * 8729)])
@pytest.mark.parametrize("call", ["ccv_linrec_fwd", "ccv_linrec_bwd"])
def test_most_tiles(call, B, L, C):
    """B ceil(L / 128) ceil(C / 64) below 2^23, as the header has it."""
    tiles = lambda B, L, C: B * -(-L // 128) * -(-C // 64)  # noqa: E731
    for more in ((0, 0, 0), (1, 0, 0), (0, 128, 0), (0, 0, 64)):
        b, n, c = (i + j for i, j in zip((B, L, C), more))
        want = "CCV_OK" if tiles(b, n, c) < 2 ** 23 else "CCV_E_SHAPE"
        args = CALLS[call](B=b, L=n, C=c, workspace_bytes=1 << 62)
        assert ccv.STATUS[getattr(ccv, call + "_check")(args)] == want, (b, n, c)
        assert (getattr(ccv, call + "_workspace_size")(args) >= 0) == (want == "CCV_OK")


@pytest.mark.parametrize("B,C,want", [(2 ** 31 - 257, 1, "CCV_OK"), (2 ** 31 - 256, 2, "CCV_E_SHAPE"), (2 ** 31 - 257, 3, "CCV_E_SHAPE"),
                                      (2 ** 20, 4094, "CCV_OK"), (2 ** 20, 4095, "CCV_E_SHAPE"), (255, 2 ** 24, "CCV_OK"), (256, 2 ** 24, "CCV_E_SHAPE")])
def test_most_rows_of_a_step(B, C, want):
    """B ceil(C / 2) below 2^31 - 256, as the header has it."""
    assert ccv.STATUS[ccv.ccv_linrec_update_check(CALLS["ccv_linrec_update"](B=B, C=C, slots=B))] == want


def test_the_decays_polynomial():
    """The coefficients in the kernels' header against expm1 in 64 bits: within 1.9e-8 of e^r - 1, and so within an eighth of 2^-24 of e^r, over
    |r| <= ln 2 / 2.  The bounds that the kernels are held to allow two units of 2^-24 for it and its rounding."""
    path = os.path.join(os.path.dirname(ccv.__file__), "csrc", "ccv_linrec_device.hpp")
    with open(path) as f:
        body = f.read().split("inline float expm1_near(float r) {")[1].split("}")[0]
    c = [np.float64(np.float32(v)) for v in re.findall(r"(\d+\.\d+)f", body)]
    assert len(c) == 6 and c[-1] == 1.0
    r = np.linspace(-math.log(2) / 2, math.log(2) / 2, 1000000)          # an even number: 0 is none of them
    q = c[0]
    for k in c[1:]:
        q = r * q + k
    off = np.abs(r * q - np.expm1(r))
    assert (off / np.abs(np.expm1(r))).max() < 1.9e-8 and (off / np.exp(r)).max() < 2.0 ** -24 / 8


# ---- group norm's sizes ----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [ccv.CCV_F32, ccv.CCV_F16, ccv.CCV_BF16])
@pytest.mark.parametrize("rows,groups,width", [
    (64, 131071, 1), (64, 131072, 1), (100, 200000, 4), (1, 2 ** 24, 1), (2 ** 31 - 1, 2 ** 24, 1), (2 ** 31 - 1, 2 ** 22, 4), (2 ** 31 - 1, 2 ** 21, 8),
    (2 ** 31 - 1, 5, 64), (2 ** 20, 2 ** 15, 512), (2 ** 31 - 1, 2 ** 16, 256), (2 ** 31 - 1, 1, 2 ** 24), (2 ** 31 - 1, 2, 2 ** 23)])
def test_group_norm_differentiates_what_it_takes(dtype, rows, groups, width):
    """Every size that the forward takes, the backward takes too: all up to 2^31 - 1 rows and 2^24 channels."""
    sizes = dict(rows=rows, groups=groups, width=width, x_dtype=dtype)
    C, back = groups * width, CALLS["ccv_group_norm_bwd"](**sizes, workspace_bytes=1 << 62)
    assert ccv.STATUS[ccv.ccv_group_norm_fwd_check(CALLS["ccv_group_norm_fwd"](**sizes))] == "CCV_OK"
    need = ccv.ccv_group_norm_bwd_workspace_size(back)
    assert need > 0 and need % (8 * C) == 0, need
    assert ccv.STATUS[ccv.ccv_group_norm_bwd_check(back)] == "CCV_OK"
    walkers, vector = need // (8 * C), 4 if dtype == ccv.CCV_F32 else 8
    assert 1 <= walkers <= rows
    if vector <= width <= 1024 * vector:                     # in vectors, by at least 4 threads each, of which a launch has fewer than 2^32
        assert walkers * groups * 4 <= 2 ** 31
    else:
        assert walkers <= 64


@pytest.mark.parametrize("shape", [(0,), (5, 0), (2, 3, 0), (2, 0, 0), (2, 3, 4, 0)])
def test_group_norm_without_channels(calls_do_nothing, shape):  # noqa: F811
    """As the C entries take it: nothing to normalise, and statistics of nothing."""
    x = torch.zeros(3, *shape)
    out, mean, rstd = ccv.group_norm_fwd(x, 2, gate=x, return_stats=True)
    assert out.shape == x.shape and mean.shape == rstd.shape == (*x.shape[:-1], 2)
    assert bool(mean.isnan().all()) and bool(rstd.isnan().all())
    dx, dw, db, dz = ccv.group_norm_bwd(x, 2, None, None, x, mean, rstd, x)
    assert dx.shape == dz.shape == x.shape and dw.shape == db.shape == (0,)
    y = torch.zeros(3, *shape, requires_grad=True)
    ccv.group_norm_fn(y, 2).sum().backward()
    assert y.grad.shape == y.shape


@pytest.mark.parametrize("shape", [(0,), (5, 0), (2, 3, 4, 0)])
def test_layer_norm_without_values(monkeypatch, shape):
    """Statistics of nothing here too."""
    monkeypatch.setattr(ccv, "_same_device", lambda x, **others: x.device)
    monkeypatch.setitem(ccv._CALLS, "ccv_norm_fwd", lambda *values: None)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: torch.full(*a, 7.0, **kw))
    out, mean, rstd = ccv.layer_norm_fwd(torch.zeros(shape), return_stats=True)
    assert out.shape == shape and mean.shape == rstd.shape == shape[:-1]
    assert bool(mean.isnan().all()) and bool(rstd.isnan().all())


# ---- rotary positions ------------------------------------------------------------------------

def test_rotary_refuses_frequencies_that_want_gradients(calls_do_nothing):  # noqa: F811
    q, pos = torch.zeros(2, 5, 3, 8), torch.zeros(2, 5, dtype=torch.int32)
    freq = torch.ones(2, dtype=torch.float64, requires_grad=True)
    for leaf in (q, q.clone().requires_grad_()):
        with pytest.raises(ValueError, match="frequencies"):
            ccv.rotary_fn(leaf, None, pos, freq)
        with pytest.raises(ValueError, match="frequencies"):
            ccv.rotary_fn(leaf, None, pos, freq * 2)
        with torch.no_grad():
            ccv.rotary_fn(leaf, None, pos, freq)
        assert ccv.rotary_fn(leaf, None, pos, freq.detach())[0].requires_grad == leaf.requires_grad


# ---- the parameters' gradients in a type of the caller's --------------------------------------

TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.mark.parametrize("wanted", [None, *TYPES])
@pytest.mark.parametrize("weight", [None, *TYPES])
@pytest.mark.parametrize("norm", ["group", "layer"])
def test_weight_dtype_is_that_of_the_gradients(calls_do_nothing, monkeypatch, norm, weight, wanted):  # noqa: F811
    """dweight and dbias come in weight_dtype, whatever the weight's own."""
    monkeypatch.setattr(ccv, "_same_device", lambda x, **others: x.device)
    monkeypatch.setitem(ccv._CALLS, "ccv_norm_bwd", lambda *values: None)
    x, w = torch.zeros(5, 8, dtype=torch.bfloat16), None if weight is None else torch.ones(8, dtype=weight)
    if norm == "group":
        _, dw, db, _ = ccv.group_norm_bwd(x, 2, w, None, x, torch.zeros(5, 2), torch.ones(5, 2), weight_dtype=wanted)
        _, _, alone, _ = ccv.group_norm_bwd(x, 2, None, w, x, torch.zeros(5, 2), torch.ones(5, 2), want_dweight=False, weight_dtype=wanted)
    else:
        _, dw, db = ccv.layer_norm_bwd(x, w, x, torch.zeros(5), torch.ones(5), weight_dtype=wanted)
        _, _, alone = ccv.layer_norm_bwd(x, w, x, torch.zeros(5), torch.ones(5), want_dweight=False, weight_dtype=wanted)
    assert dw.dtype == db.dtype == alone.dtype == (wanted or weight or x.dtype)
