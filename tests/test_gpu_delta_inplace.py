"""States written over the states they came from: the results are those of separate arrays, bit for bit, whether a
sequence is one workgroup's or goes through the call in parts."""
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
import layer_reference as ref
from gpu_support import log

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    ccv.lib()

# B, L, Hk, Hv, Dk, Dv, packed lengths.  In parts: a last part of one chunk, of several, more parts than the chip takes at
# once, parts beside whole sequences; whole: chains and columns
SHAPES = {"parts": (1, 64 * 33, 1, 2, 64, 32, None), "rows in parts": (3, 64 * 48 - 5, 1, 1, 128, 64, None),
          "many parts": (1, 27 * 64 * 17, 1, 1, 128, 32, [64 * 17] * 27),
          "parts and whole": (1, 64 * 80, 1, 2, 64, 64, [64 * 60, 0, 1, 100]),
          "whole": (3, 200, 2, 4, 72, 40, None), "packed": (1, 300, 2, 4, 128, 64, [129, 0, 65, 64]),
          "columns": (8, 70, 16, 16, 64, 128, None)}


def inputs(shape, dtype, seed):
    *sizes, lengths = SHAPES[shape]
    q, k, v, g, beta, h0 = ref.delta_inputs(*sizes, dtype, seed=seed, seqs=lengths and len(lengths), decay=0.01)
    log(f"  {shape} {dtype}")
    return [t.cuda() for t in (q, k, v, g, beta)], h0.cuda(), None if lengths is None else ref.cu_of(lengths).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_final_state_over_the_initial_one(shape, dtype):
    x, h0, cu = inputs(shape, dtype, 1)
    want, final = ccv.gated_delta_rule_fwd(*x, cu_seqlens=cu, initial_state=h0, return_final_state=True)
    for _ in range(3):
        cache = h0.clone()
        out, ht = ccv.gated_delta_rule_fwd(*x, cu_seqlens=cu, initial_state=cache, return_final_state=True, final_state_out=cache)
        assert ht is cache
        assert torch.equal(out, want) and torch.equal(cache, final)
