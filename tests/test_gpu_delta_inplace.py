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


def strides(t):
    return (ccv.ctypes.c_int64 * 3)(*t.stride()[:3])


def backward(x, cu, scale, h0, dout, dht, dh0):
    """The C call with everything given: [dq, dk, dv, dg, dbeta]."""
    q, k, v, g, beta = x
    d = [torch.full_like(t, float("nan")) for t in x]
    a = ccv.ccv_delta_bwd_args_t(B=q.shape[0], L=q.shape[1], N=0 if cu is None else len(cu) - 1, Hk=q.shape[2], Hv=v.shape[2],
                                 Dk=q.shape[3], Dv=v.shape[3], x_dtype=ccv.DTYPE_CODE[q.dtype], g_dtype=ccv.DTYPE_CODE[g.dtype],
                                 beta_dtype=ccv.DTYPE_CODE[beta.dtype], scale=scale, cu_seqlens=None if cu is None else cu.data_ptr())
    for n, s, t in (("q", "q", q), ("k", "k", k), ("v", "v", v), ("g", "g", g), ("beta", "beta", beta), ("dout", "dout", dout),
                    ("initial_state", "init", h0), ("dfinal_state", "dfinal", dht), ("dinitial_state", "dinit", dh0),
                    ("dq", "dq", d[0]), ("dk", "dk", d[1]), ("dv", "dv", d[2]), ("dg", "dg", d[3]), ("dbeta", "dbeta", d[4])):
        setattr(a, n, t.data_ptr())
        setattr(a, s + "_stride", strides(t) if t.dim() == 4 else (ccv.ctypes.c_int64 * 3)(*t.stride()))
    need = ccv.ccv_delta_bwd_workspace_size(a)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    a.workspace, a.workspace_bytes = ws.data_ptr(), need
    assert ccv.ccv_delta_bwd(a) == 0
    torch.cuda.synchronize()
    return d


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_state_gradient_over_the_one_it_came_from(shape, dtype):
    x, h0, cu = inputs(shape, dtype, 2)
    gen = torch.Generator().manual_seed(3)
    dout = torch.randn(x[2].shape, generator=gen).to(x[2].dtype).cuda()
    dht = (torch.randn(h0.shape, generator=gen) * 0.2).cuda()
    dh0 = torch.empty_like(h0)
    want = backward(x, cu, 0.125, h0, dout, dht.clone(), dh0)
    for _ in range(3):
        both = dht.clone()
        got = backward(x, cu, 0.125, h0, dout, both, both)
        assert torch.equal(both, dh0)
        for n, t, w in zip(("dq", "dk", "dv", "dg", "dbeta"), got, want):
            assert torch.equal(t, w), n
