"""What the layer's differentiable operators tell torch's autograd: on the CPU with the C calls' results in the place of
the calls, and on the GPU."""
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
import layer_reference as ref


def delta_by_reference(monkeypatch):
    """gated_delta_rule_fwd and _bwd from the 64-bit reference, in the shapes and dtypes of the calls."""
    def fwd(q, k, v, g, beta, scale=None, cu_seqlens=None, initial_state=None, return_final_state=False, **kw):
        out, ht = ref.delta_reference(q, k, v, g, beta, scale, None, initial_state)
        return (out.to(v.dtype), ht.float()) if return_final_state else out.to(v.dtype)

    def bwd(q, k, v, g, beta, dout, scale=None, cu_seqlens=None, initial_state=None, dfinal_state=None, return_dinitial_state=False):
        with torch.enable_grad():
            r = ref.delta_gradients(*(t.detach() for t in (q, k, v, g, beta, dout)), scale, None,
                                    None if initial_state is None else initial_state.detach(), dfinal_state)
        dh = r["dh0"].float() if return_dinitial_state else None
        return (*(r[n].to(t.dtype) for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta))), dh)

    monkeypatch.setattr(ccv, "gated_delta_rule_fwd", fwd)
    monkeypatch.setattr(ccv, "gated_delta_rule_bwd", bwd)


def norm_by_formula(monkeypatch):
    def fwd(x, weight=None, bias=None, eps=1e-5, return_stats=False, out=None):
        d = x - x.mean(-1, keepdim=True)
        rstd = (d.square().mean(-1, keepdim=True) + eps).rsqrt()
        y = d * rstd * (1 if weight is None else weight) + (0 if bias is None else bias)
        return y, x.mean(-1), rstd[..., 0]

    def bwd(x, weight, dout, mean, rstd, want_dx=True, want_dweight=True, want_dbias=True, weight_dtype=None):
        n = (x - mean[..., None]) * rstd[..., None]
        a = dout * (1 if weight is None else weight)
        dx = rstd[..., None] * (a - a.mean(-1, keepdim=True) - n * (a * n).mean(-1, keepdim=True))
        return (dx if want_dx else None, (dout * n).sum(0) if want_dweight else None, dout.sum(0) if want_dbias else None)

    monkeypatch.setattr(ccv, "layer_norm_fwd", fwd)
    monkeypatch.setattr(ccv, "layer_norm_bwd", bwd)


def delta(device="cpu", states=True):
    x = ref.delta_inputs(1, 6, 1, 2, 8, 8, states=states)
    leaves = [t.to(device).requires_grad_() for t in x if t is not None]
    return leaves, lambda: ccv.gated_delta_rule_fn(*leaves[:5], initial_state=leaves[5] if states else None)


def norm(device="cpu", states=True):
    gen = torch.Generator().manual_seed(0)
    leaves = [t.to(device).requires_grad_() for t in (torch.randn(5, 16, generator=gen), torch.rand(16, generator=gen), torch.rand(16, generator=gen))]
    leaves = leaves if states else leaves[:1]
    return leaves, lambda: ccv.layer_norm_fn(*leaves)


def check_second_derivative(make, states):
    """Refused whatever the incoming gradient is, a constant too; first derivatives are as without create_graph."""
    leaves, run = make
    plain = torch.autograd.grad(run().sum(), leaves)
    for loss in (lambda: run().sum(), lambda: run().square().sum()):
        grads = torch.autograd.grad(loss(), leaves, create_graph=True)
        for g in grads:
            assert g.requires_grad
            with pytest.raises(RuntimeError, match="second derivative"):
                torch.autograd.grad(g.square().sum(), leaves, retain_graph=True, allow_unused=True)
        # a penalty on the gradient beside a loss of its own
        with pytest.raises(RuntimeError, match="second derivative"):
            (loss() + grads[0].square().sum()).backward()
    for g, p in zip(torch.autograd.grad(run().sum(), leaves, create_graph=True), plain):
        assert torch.equal(g, p)
    frozen = run().sum()
    for g, p in zip(torch.autograd.grad(frozen, leaves[:1]), plain):
        assert torch.equal(g, p) and not g.requires_grad


@pytest.mark.parametrize("states", [True, False])
def test_second_derivatives_of_the_delta_rule_are_refused(monkeypatch, states):
    delta_by_reference(monkeypatch)
    check_second_derivative(delta(states=states), states)


@pytest.mark.parametrize("states", [True, False])
def test_second_derivatives_of_layer_norm_are_refused(monkeypatch, states):
    norm_by_formula(monkeypatch)
    check_second_derivative(norm(states=states), states)


@pytest.mark.gpu
@pytest.mark.parametrize("states", [True, False])
@pytest.mark.parametrize("make", [delta, norm])
def test_second_derivatives_on_the_gpu(make, states):
    check_second_derivative(make("cuda", states), states)


def step_inputs(x, state):
    """One step's q, k, v, g, beta of the sequences' inputs, and the state."""
    return [*(t.detach()[:, 0].contiguous() for t in x[:5]), state]


def calls_do_nothing(monkeypatch):
    monkeypatch.setattr(ccv, "_same_device", lambda x, **others: x.device)
    for name in ("ccv_delta_fwd", "ccv_delta_update", "ccv_norm_fwd"):
        monkeypatch.setitem(ccv._CALLS, name, lambda *values: None)


def test_written_tensors_have_new_versions(monkeypatch):
    calls_do_nothing(monkeypatch)
    q, k, v, g, beta, h0 = ref.delta_inputs(1, 6, 1, 2, 8, 8)
    out, one = torch.empty_like(v), torch.empty_like(v[:, 0])
    given = {"state": h0, "out": out, "one": one, "q": q}
    before = {n: t._version for n, t in given.items()}
    ccv.gated_delta_rule_fwd(q, k, v, g, beta, initial_state=h0, return_final_state=True)
    ccv.gated_delta_rule_fwd(q, k, v, g, beta, initial_state=h0)
    assert {n: t._version for n, t in given.items()} == before
    ccv.gated_delta_rule_fwd(q, k, v, g, beta, initial_state=h0, return_final_state=True, final_state_out=h0, out=out)
    assert h0._version > before["state"] and out._version > before["out"]
    at = h0._version
    ccv.gated_delta_rule_update(*step_inputs((q, k, v, g, beta), h0), out=one)
    assert h0._version > at and one._version > before["one"] and q._version == before["q"]
    y = torch.empty(3, 8)
    at = y._version
    ccv.layer_norm_fwd(torch.ones(3, 8), out=y)
    assert y._version > at
    with torch.inference_mode():
        ccv.gated_delta_rule_update(*step_inputs((q, k, v, g, beta), torch.zeros(1, 2, 8, 8)))


def check_advanced_state(x, advance):
    """A cache that was the initial state of a differentiable call, advanced before its backward: torch raises."""
    leaves, cache = x[:5], x[5].detach().clone()
    loss = ccv.gated_delta_rule_fn(*leaves, initial_state=cache).sum()
    advance(leaves, cache)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def by_update(leaves, cache):
    ccv.gated_delta_rule_update(*step_inputs(leaves, cache))


def by_prefill(leaves, cache):
    with torch.no_grad():
        ccv.gated_delta_rule_fwd(*leaves, initial_state=cache, return_final_state=True, final_state_out=cache)


def test_a_state_advanced_before_the_backward(monkeypatch):
    calls_do_nothing(monkeypatch)
    for advance in (by_update, by_prefill):
        leaves, _ = delta()
        forward = ccv.gated_delta_rule_fwd
        with monkeypatch.context() as m:
            delta_by_reference(m)
            reference = ccv.gated_delta_rule_fwd
            m.setattr(ccv, "gated_delta_rule_fwd", lambda *a, **kw: (forward if "final_state_out" in kw else reference)(*a, **kw))
            check_advanced_state(leaves, advance)


@pytest.mark.gpu
@pytest.mark.parametrize("advance", [by_update, by_prefill])
def test_a_state_advanced_before_the_backward_on_the_gpu(advance):
    check_advanced_state(delta("cuda")[0], advance)
