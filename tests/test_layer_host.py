"""The layer's operators on the CPU: the args structs, every check that needs no device, the
binding's refusals, and the 64-bit reference itself against finite differences."""
import ctypes

import numpy as np
import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
import layer_reference as ref

Q, K, V, G, BETA, OUT, H0, HT, WS, CU, DO, DQ, DK, DV, DG, DB, DH0, DHT = (0x1000000 * (i + 1) for i in range(18))


def s3(*v):
    return (ctypes.c_int64 * 3)(*v)


def fwd(B=2, L=100, Hk=2, Hv=4, Dk=64, Dv=32, **over):
    a = ccv.ccv_delta_fwd_args_t()
    a.B, a.L, a.Hk, a.Hv, a.Dk, a.Dv = B, L, Hk, Hv, Dk, Dv
    a.x_dtype, a.g_dtype, a.beta_dtype, a.scale = ccv.CCV_BF16, ccv.CCV_F32, ccv.CCV_BF16, 0.125
    a.q, a.k, a.v, a.g, a.beta, a.out = Q, K, V, G, BETA, OUT
    a.q_stride = a.k_stride = s3(L * Hk * Dk, Hk * Dk, Dk)
    a.v_stride = a.out_stride = s3(L * Hv * Dv, Hv * Dv, Dv)
    a.g_stride = a.beta_stride = s3(L * Hv, Hv, 1)
    a.init_stride = a.final_stride = s3(Hv * Dk * Dv, Dk * Dv, Dv)
    a.workspace, a.workspace_bytes = WS, 1 << 40
    for n, x in over.items():
        setattr(a, n, s3(*x) if n.endswith("stride") else x)
    return a


def bwd(B=2, L=100, Hk=2, Hv=4, Dk=64, Dv=32, **over):
    a = ccv.ccv_delta_bwd_args_t()
    f = fwd(B, L, Hk, Hv, Dk, Dv)
    for n in ("B", "L", "Hk", "Hv", "Dk", "Dv", "x_dtype", "g_dtype", "beta_dtype", "scale", "q", "k", "v", "g", "beta",
              "q_stride", "k_stride", "v_stride", "g_stride", "beta_stride", "init_stride", "workspace", "workspace_bytes"):
        setattr(a, n, getattr(f, n))
    a.dout, a.dq, a.dk, a.dv, a.dg, a.dbeta = DO, DQ, DK, DV, DG, DB
    a.dout_stride = a.dv_stride = f.v_stride
    a.dq_stride = a.dk_stride = f.q_stride
    a.dg_stride = a.dbeta_stride = f.g_stride
    a.dfinal_stride = a.dinit_stride = f.init_stride
    for n, x in over.items():
        setattr(a, n, s3(*x) if n.endswith("stride") else x)
    return a


def upd(B=3, L=1, slots=8, Hk=2, Hv=4, Dk=64, Dv=32, **over):
    a = ccv.ccv_delta_update_args_t()
    f = fwd(B, L, Hk, Hv, Dk, Dv)
    for n in ("B", "L", "Hk", "Hv", "Dk", "Dv", "x_dtype", "g_dtype", "beta_dtype", "scale", "q", "k", "v", "g", "beta", "out",
              "q_stride", "k_stride", "v_stride", "g_stride", "beta_stride", "out_stride"):
        setattr(a, n, getattr(f, n))
    a.slots, a.state, a.state_stride = slots, H0, f.init_stride
    for n, x in over.items():
        setattr(a, n, s3(*x) if n.endswith("stride") else x)
    return a


def name(call, a):
    return ccv.STATUS[getattr(ccv, call + "_check")(a)]


CALLS = {"ccv_delta_fwd": fwd, "ccv_delta_bwd": bwd, "ccv_delta_update": upd}


@pytest.mark.parametrize("call", sorted(ccv._LAYER_CALLS))
def test_packed_args_are_the_struct(call):
    """What the binding packs in one go has the size and the field places of the ctypes mirror."""
    t = ccv._LAYER_CALLS[call][0]
    values, fields = [], []
    for i, (n, ty) in enumerate(t._fields_[1:]):
        if ty in (ccv._I64x2, ccv._I64x3):
            v = [1000 * (i + 1) + j for j in range(ty._length_)]
            values += v
        else:
            v = 0.5 + i if ty is ctypes.c_float else 1000 * (i + 1)
            values.append(v)
        fields.append((n, v))
    c = ccv._CALLS[call]
    raw = c.pack(c.size, *values)
    a = t.from_buffer_copy(raw)
    assert len(raw) == ctypes.sizeof(t) and a.struct_size == ctypes.sizeof(t)
    for n, v in fields:
        got = getattr(a, n)
        assert (list(got) if isinstance(v, list) else got) == v, n


@pytest.mark.parametrize("call", sorted(CALLS))
def test_valid_and_malformed(call):
    make = CALLS[call]
    assert name(call, make()) == "CCV_OK"
    assert getattr(ccv.lib(), call + "_check")(None) == -1
    a = make()
    a.struct_size -= 8
    assert name(call, a) == "CCV_E_ABI"
    for over in ({"Hk": 3}, {"Dk": 0}, {"Dv": 0}, {"Hk": 0}, {"B": -1}, {"L": -1}, {"L": 2 ** 31}):
        a = make()
        for n, x in over.items():
            setattr(a, n, x)
        assert name(call, a) == "CCV_E_SHAPE", over
    a = make()
    a.Dk = 129
    assert name(call, a) == "CCV_E_UNSUPPORTED"
    for f in ("x_dtype", "g_dtype", "beta_dtype"):
        assert name(call, make(**{f: 3})) == "CCV_E_DTYPE"
    for f in ("q", "k", "v", "g", "beta"):
        assert name(call, make(**{f: None})) == "CCV_E_NULL", f
    assert name(call, make(q_stride=(12800, -128, 64))) == "CCV_E_LAYOUT"
    assert name(call, make(v_stride=(2 ** 62, 128, 32))) == "CCV_E_SHAPE"


def test_forward_errors():
    c = "ccv_delta_fwd"
    assert name(c, fwd(out=None)) == "CCV_E_NULL"
    assert name(c, fwd(out=V)) == "CCV_E_ALIAS"
    assert name(c, fwd(out_stride=(12800, 16, 32))) == "CCV_E_LAYOUT"      # steps overlap
    assert name(c, fwd(out_stride=(12800, 0, 32))) == "CCV_E_LAYOUT"
    assert name(c, fwd(B=1, out_stride=(2 ** 40, 2 ** 26, 32))) == "CCV_E_LAYOUT"   # steps too far apart
    assert name(c, fwd(final_state=HT, final_stride=(8192, 0, 32))) == "CCV_E_LAYOUT"
    assert name(c, fwd(final_state=HT, initial_state=HT)) == "CCV_OK"
    assert name(c, fwd(final_state=HT, initial_state=HT, init_stride=(0, 2048, 32))) == "CCV_E_ALIAS"
    assert name(c, fwd(final_state=Q)) == "CCV_E_ALIAS"
    assert name(c, fwd(cu_seqlens=CU, N=3)) == "CCV_E_SHAPE"               # packed needs one row
    assert name(c, fwd(N=3)) == "CCV_E_SHAPE"
    assert name(c, fwd(B=1, cu_seqlens=CU, N=3)) == "CCV_OK"
    need = ccv.ccv_delta_fwd_workspace_size(fwd())
    assert need > 0
    assert name(c, fwd(workspace_bytes=need)) == "CCV_OK"
    assert name(c, fwd(workspace_bytes=need - 1)) == "CCV_E_SHAPE"
    assert name(c, fwd(workspace=None)) == "CCV_E_NULL"
    assert name(c, fwd(workspace=WS + 8)) == "CCV_E_LAYOUT"
    # zero strides of inputs (broadcast) are fine, and rows that need a copy take more workspace
    assert name(c, fwd(g_stride=(0, 0, 0), beta_stride=(0, 0, 0), q_stride=(0, 0, 0))) == "CCV_OK"
    assert ccv.ccv_delta_fwd_workspace_size(fwd(q=Q + 2)) > need


def test_nothing_to_do_needs_no_pointers():
    for c, make in CALLS.items():
        nul = dict(q=None, k=None, v=None, g=None, beta=None)
        assert name(c, make(L=0, **nul)) == "CCV_OK"
        assert name(c, make(B=0, **nul)) == "CCV_OK"
    assert ccv.ccv_delta_fwd_workspace_size(fwd(L=0)) == 0
    assert ccv.ccv_delta_bwd_workspace_size(bwd(B=0)) == 0


def test_backward_errors():
    c = "ccv_delta_bwd"
    for f in ("dout", "dq", "dk", "dv", "dg", "dbeta"):
        assert name(c, bwd(**{f: None})) == "CCV_E_NULL", f
    assert name(c, bwd(dinitial_state=DH0)) == "CCV_E_UNSUPPORTED"
    assert name(c, bwd(dinitial_state=DH0, initial_state=H0)) == "CCV_OK"
    assert name(c, bwd(dinitial_state=H0, initial_state=H0)) == "CCV_E_ALIAS"
    assert name(c, bwd(dinitial_state=DHT, initial_state=H0, dfinal_state=DHT)) == "CCV_OK"
    assert name(c, bwd(dq=Q)) == "CCV_E_ALIAS"
    assert name(c, bwd(dq=DK)) == "CCV_E_ALIAS"
    assert name(c, bwd(dg=DB)) == "CCV_E_ALIAS"
    assert name(c, bwd(dv_stride=(12800, 1, 32))) == "CCV_E_LAYOUT"
    need = ccv.ccv_delta_bwd_workspace_size(bwd())
    assert need > ccv.ccv_delta_fwd_workspace_size(fwd())
    assert name(c, bwd(workspace_bytes=need - 1)) == "CCV_E_SHAPE"


def test_update_errors():
    c = "ccv_delta_update"
    assert name(c, upd(state=None)) == "CCV_E_NULL"
    assert name(c, upd(slots=2)) == "CCV_E_SHAPE"                          # row b is slot b
    assert name(c, upd(slots=2, state_indices=CU)) == "CCV_OK"
    assert name(c, upd(slots=-1)) == "CCV_E_SHAPE"
    assert name(c, upd(out=H0)) == "CCV_E_ALIAS"
    assert name(c, upd(out=Q)) == "CCV_E_ALIAS"
    assert name(c, upd(state_stride=(8192, 0, 32))) == "CCV_E_LAYOUT"


def norm_fwd(**over):
    a = ccv.ccv_norm_fwd_args_t()
    a.n0, a.n1, a.width, a.x_dtype, a.w_dtype, a.eps = 4, 5, 96, ccv.CCV_BF16, ccv.CCV_F32, 1e-5
    a.x, a.weight, a.bias, a.out, a.mean, a.rstd = Q, K, V, OUT, G, BETA
    a.x_stride = a.out_stride = (ctypes.c_int64 * 2)(480, 96)
    for n, x in over.items():
        setattr(a, n, (ctypes.c_int64 * 2)(*x) if n.endswith("stride") else x)
    return a


def norm_bwd(**over):
    a = ccv.ccv_norm_bwd_args_t()
    a.n0, a.n1, a.width, a.x_dtype, a.w_dtype = 4, 5, 96, ccv.CCV_BF16, ccv.CCV_F32
    a.x, a.weight, a.dout, a.mean, a.rstd, a.dx, a.dweight, a.dbias = Q, K, DO, G, BETA, DQ, DK, DV
    a.x_stride = a.dout_stride = a.dx_stride = (ctypes.c_int64 * 2)(480, 96)
    a.workspace, a.workspace_bytes = WS, 1 << 30
    for n, x in over.items():
        setattr(a, n, (ctypes.c_int64 * 2)(*x) if n.endswith("stride") else x)
    return a


def test_norm_errors():
    f, b = "ccv_norm_fwd", "ccv_norm_bwd"
    assert name(f, norm_fwd()) == name(b, norm_bwd()) == "CCV_OK"
    assert name(f, norm_fwd(weight=None, bias=None, mean=None, rstd=None)) == "CCV_OK"
    assert name(f, norm_fwd(x=None)) == name(f, norm_fwd(out=None)) == "CCV_E_NULL"
    assert name(f, norm_fwd(out=Q)) == name(f, norm_fwd(mean=Q)) == name(f, norm_fwd(mean=BETA)) == "CCV_E_ALIAS"
    for eps in (-1.0, float("nan"), float("inf")):
        assert name(f, norm_fwd(eps=eps)) == "CCV_E_UNSUPPORTED"
    assert name(f, norm_fwd(width=-1)) == name(f, norm_fwd(n0=2 ** 20, n1=2 ** 20)) == "CCV_E_SHAPE"
    assert name(f, norm_fwd(x_dtype=4)) == name(b, norm_bwd(w_dtype=-1)) == "CCV_E_DTYPE"
    assert name(f, norm_fwd(out_stride=(480, 90))) == name(f, norm_fwd(x_stride=(-480, 96))) == "CCV_E_LAYOUT"
    assert name(f, norm_fwd(x_stride=(0, 0))) == "CCV_OK"                  # one row for all
    assert name(f, norm_fwd(n0=0, x=None, out=None)) == "CCV_OK"
    for p in ("x", "dout", "mean", "rstd"):
        assert name(b, norm_bwd(**{p: None})) == "CCV_E_NULL"
    assert name(b, norm_bwd(dx=None, dweight=None, dbias=None, workspace=None)) == "CCV_OK"
    assert name(b, norm_bwd(dx=DO)) == name(b, norm_bwd(dbias=DK)) == "CCV_E_ALIAS"
    need = ccv.ccv_norm_bwd_workspace_size(norm_bwd())
    assert need > 0 and need % (2 * 96 * 4) == 0
    assert name(b, norm_bwd(workspace=None)) == "CCV_E_NULL"
    assert name(b, norm_bwd(workspace_bytes=need - 1)) == "CCV_E_SHAPE"


def test_table_errors():
    a = ccv.ccv_seq_tables_args_t()
    a.N, a.total, a.lengths, a.cu_seqlens, a.seq_idx, a.positions = 3, 10, Q, K, V, G
    c = "ccv_seq_tables"
    assert name(c, a) == "CCV_OK"
    for f, x, want in (("lengths", None, "CCV_E_NULL"), ("cu_seqlens", None, "CCV_E_NULL"), ("seq_idx", None, "CCV_OK"),
                       ("seq_idx", Q, "CCV_E_ALIAS"), ("positions", K, "CCV_E_ALIAS"), ("N", -1, "CCV_E_SHAPE"),
                       ("total", 2 ** 31, "CCV_E_SHAPE")):
        b = ccv.ccv_seq_tables_args_t.from_buffer_copy(a)
        setattr(b, f, x)
        assert name(c, b) == want, (f, x)


def test_binding_refuses_cpu_tensors_and_shapes():
    q, k, v, g, beta, h0 = ref.delta_inputs(1, 5, 1, 2, 8, 8)
    with pytest.raises(ValueError, match="GPU"):
        ccv.gated_delta_rule_fwd(q, k, v, g, beta)
    with pytest.raises(ValueError, match="GPU"):
        ccv.gated_delta_rule_update(q, k, v, g, beta, h0)
    with pytest.raises(ValueError, match="GPU"):
        ccv.layer_norm_fwd(q)
    with pytest.raises(ValueError, match="GPU"):
        ccv.sequence_tables(torch.ones(3, dtype=torch.int32), 5)
    with pytest.raises(ValueError, match="multiple"):
        ccv.gated_delta_rule_fwd(q.expand(1, 5, 3, 8), k.expand(1, 5, 3, 8), v, g, beta)
    with pytest.raises(ValueError, match="one dtype"):
        ccv.gated_delta_rule_fwd(q, k, v.half(), g, beta)
    with pytest.raises(ValueError, match=r"\[B, L, Hv\]"):
        ccv.gated_delta_rule_fwd(q, k, v, g[..., :1], beta)
    with pytest.raises(ValueError, match="return_final_state"):
        ccv.gated_delta_rule_fwd(q, k, v, g, beta, final_state_out=h0)
    with pytest.raises(ValueError, match="int32"):
        ccv.sequence_tables(torch.ones(3), 5)
    with pytest.raises(ValueError, match="weight's dtype"):
        ccv.layer_norm_fwd(q, torch.ones(8), torch.ones(8).half())


@pytest.mark.parametrize("lengths", [None, [3, 0, 4]])
def test_reference_gradients_against_differences(lengths):
    """The 64-bit reference's gradients against central differences of its outputs."""
    L = 8
    q, k, v, g, beta, h0 = ref.delta_inputs(1, L, 1, 2, 3, 2, seed=5, seqs=3 if lengths else 1)
    gen = torch.Generator().manual_seed(6)
    dout, dht = torch.randn(1, L, 2, 2, generator=gen), torch.randn(h0.shape, generator=gen)
    got = ref.delta_gradients(q, k, v, g, beta, dout, lengths=lengths, h0=h0, dht=dht)
    x = [t.double() for t in (q, k, v, g, beta, h0)]

    def loss(args):
        o, s = ref.delta_reference(*args[:5], None, lengths, args[5])
        return float((o * dout.double()).sum() + (s * dht.double()).sum())

    e = 1e-5      # differences: rounding 1e-16 / 1e-5 and e^2 curvature, far below the 1e-7 allowed
    for i, n in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dh0")):
        flat, want = x[i].reshape(-1), got[n].reshape(-1)
        for j in range(0, flat.numel(), max(1, flat.numel() // 10)):
            keep = float(flat[j])
            flat[j] = keep + e
            up = loss(x)
            flat[j] = keep - e
            down = loss(x)
            flat[j] = keep
            assert abs((up - down) / (2 * e) - float(want[j])) < 1e-7, (n, j)


def test_reference_tables():
    cu, seq, pos = ref.tables_reference([2, 0, 3, -4, 9], 8)
    assert cu.tolist() == [0, 2, 2, 5, 5, 8]
    assert seq.tolist() == [0, 0, 2, 2, 2, 4, 4, 4]
    assert pos.tolist() == [0, 1, 0, 1, 2, 0, 1, 2]
    assert np.array_equal(ref.tables_reference([], 2)[1], [-1, -1])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 70])
def test_rounded_reference_is_within_the_limits(dtype, L):
    """The 64-bit results, rounded once to the type, pass the limits that the kernels are held to,
    whatever the number of elements; results one spacing off do not."""
    q, k, v, g, beta, h0 = ref.delta_inputs(2, L, 1, 2, 64, 32, dtype, seed=L)
    want = ref.delta_gradients(q, k, v, g, beta, v, None, None, h0)
    for name in ("out", "dq", "dk", "dv", "dg", "dbeta"):
        ref.assert_near(name, want[name].to(ref.DT[dtype]), want[name])
    with pytest.raises(AssertionError):
        ref.assert_near("out", (want["out"] * (1 + 2.0 ** -7)).to(ref.DT[dtype]), want["out"])
    tiny = torch.linspace(-1e-5, 1e-5, 999, dtype=torch.float64)
    assert bool(((tiny.to(ref.DT[dtype]).double() - tiny).abs() <= ref.half_spacing(ref.DT[dtype], tiny)).all())
