"""Steps of v so far apart that 64 of them pass 32 bits: they are copied, heads first, and the results are those of
arrays whose steps lie together."""
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
from gpu_support import log

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    ccv.lib()


def test_steps_far_apart():
    L, H, D = 64, 17, 1 << 20                     # 71 MB from step to step, 4.6 GB in all
    log(f"  {L} steps of {H} heads of {D}")
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, g, beta = rand(1, L, 1, 1), rand(1, L, 1, 1), -0.2 * rand(1, L, H), rand(1, L, H)
    v = rand(1, L, H, D)
    near = v.transpose(1, 2).contiguous().transpose(1, 2)           # the same values, steps of a head together
    outs = [torch.empty_like(near).copy_(near) for _ in range(2)]
    for x, out in zip((v, near), outs):
        assert out.stride(1) == D
        ccv.gated_delta_rule_fwd(q, k, x, g, beta, out=out)
    torch.cuda.synchronize()
    assert torch.equal(*outs)
    # and the recurrence itself, whose state is one row a head
    S = torch.zeros(H, D, device="cuda", dtype=torch.float64)
    for t in range(L):
        S = g[0, t].double().exp()[:, None] * S
        S = S + k[0, t, 0].double() * beta[0, t].double()[:, None] * (v[0, t].double() - k[0, t, 0].double() * S)
        y = q[0, t, 0].double() * S
        assert float((outs[0][0, t].double() - y).abs().max()) <= 2.0 ** -16 * float(y.abs().max()), t
