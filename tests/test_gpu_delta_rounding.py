"""16-bit results of the delta rule are those of a 32-bit computation, rounded once.

A result y that is d off before its rounding falls to the other side of a rounding boundary with the
probability |d| / s, s the spacing of the type at y, and is then s from the rounded 64-bit result: a mean square of
|d| s.  With |d| = e |y| and s between 2^-8 and 2^-7 of y in bf16 (2^-11 and 2^-10 in fp16), on average 2^-7.5
(2^-10.5), the 2-norm of the difference from the *rounded* reference is about sqrt(e 2^-7.5) of the result's.
fp32 sums over 128 terms, their roundings of random sign, are within e = sqrt(128) 2^-24 = 2^-20.5: 2^-14 in bf16
and 2^-15.5 in fp16; two such sums one after the other, as in a gradient, sqrt(2) times the e.  An operand of 16
significant bits (e about 2^-18.5) gives 2^-13 and 2^-14.5.
"""
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
import layer_reference as ref
from gpu_support import log

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    ccv.lib()


def check(name, got, want, chains):
    want = want.to(got.dtype).double()
    d = got.cpu().double() - want
    per = 2.0 ** (-7.5 if got.dtype == torch.bfloat16 else -10.5)
    limit, off = (chains ** 0.5 * 2.0 ** -20.5 * per) ** 0.5, float(d.norm() / want.norm())
    log(f"  {name}: {off:.3g} from the rounded reference, allowed {limit:.3g}")
    assert off <= limit, f"{name}: {off:.3g} from the rounded reference, allowed {limit:.3g}"


# B, L, Hk, Hv, Dk, Dv, packed lengths: few heads, heads for wider slices, for whole columns, packed, in parts
SHAPES = {"few": (2, 400, 2, 4, 128, 128, None), "wide": (2, 130, 16, 32, 128, 64, None), "columns": (2, 130, 32, 64, 64, 128, None),
          "packed": (1, 500, 2, 4, 72, 96, [201, 0, 1, 250]), "parts": (1, 1100, 1, 1, 64, 128, None)}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_outputs(shape, dtype):
    *sizes, lengths = SHAPES[shape]
    q, k, v, g, beta, h0 = ref.delta_inputs(*sizes, dtype, seed=3, seqs=lengths and len(lengths))
    cu = None if lengths is None else ref.cu_of(lengths).cuda()
    out = ccv.gated_delta_rule_fwd(*(t.cuda() for t in (q, k, v, g, beta)), cu_seqlens=cu, initial_state=h0.cuda())
    torch.cuda.synchronize()
    check(f"{shape} out", out, ref.delta_reference(q, k, v, g, beta, None, lengths, h0)[0], 1)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", ["few", "packed", "parts"])
def test_gradients(shape, dtype):
    *sizes, lengths = SHAPES[shape]
    q, k, v, g, beta, h0 = ref.delta_inputs(*sizes, dtype, seed=4, seqs=lengths and len(lengths))
    dout = torch.randn(v.shape, generator=torch.Generator().manual_seed(5)).to(v.dtype)
    cu = None if lengths is None else ref.cu_of(lengths).cuda()
    got = ccv.gated_delta_rule_bwd(*(t.cuda() for t in (q, k, v, g, beta, dout)), cu_seqlens=cu, initial_state=h0.cuda())
    torch.cuda.synchronize()
    want = ref.delta_gradients(q, k, v, g, beta, dout, None, lengths, h0)
    for name, t in zip(("dq", "dk", "dv"), got):
        check(f"{shape} {name}", t, want[name], 2)
