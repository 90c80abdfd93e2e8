"""Steps that write nothing (beta 0): what is a multiple of beta is 0 itself, and every gradient is the reference's."""
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
import layer_reference as ref
from gpu_support import log

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    ccv.lib()


# few heads, heads for 32 values a workgroup, for whole columns forward and in both passes, in parts
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,L,Hk,Hv,Dv", [(1, 150, 2, 4, 40), (9, 70, 16, 16, 64), (10, 70, 16, 16, 96), (1, 1100, 1, 1, 64)])
def test_steps_without_a_write(dtype, B, L, Hk, Hv, Dv):
    log(f"  beta 0 {dtype} {B} x {L}, {Hv} heads")
    q, k, v, g, beta, h0 = ref.delta_inputs(B, L, Hk, Hv, 64, Dv, dtype, seed=9, decay=0.05)
    beta[:, ::3] = 0
    beta[:, L // 2:, 0] = 0
    gen = torch.Generator().manual_seed(3)
    dout, dht = torch.randn(v.shape, generator=gen).to(v.dtype), torch.randn(h0.shape, generator=gen) * 0.2
    got = ccv.gated_delta_rule_bwd(*(t.cuda() for t in (q, k, v, g, beta, dout)), initial_state=h0.cuda(), dfinal_state=dht.cuda(),
                                   return_dinitial_state=True)
    want = ref.delta_gradients(q, k, v, g, beta, dout, None, None, h0, dht)
    assert not got[2].cpu()[beta == 0].any()
    for name, t in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got):
        ref.assert_near(name, t, want[name], 2, "beta 0")
