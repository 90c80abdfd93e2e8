"""The gated linear recurrence, group norm and rotary positions on the CPU: every check that needs no
device, the binding's refusals, what torch's autograd is told, the frequencies' formulas, and the
64-bit references themselves against finite differences."""
import ctypes
import math

import pytest
import torch

import causal_depthwise_conv1d_amd as ccv
import recurrent_reference as ref

X, G, OUT, H0, HT, CAR, WS, CU, DO, DX, DG, DH0, DHT, W, B_, Z, MEAN, RSTD, DW, DB, DZ, POS, FREQ = (
    0x1000000 * (i + 1) for i in range(23))


def fill(t, base, over):
    a = t()
    for n, v in {**base, **over}.items():
        kind = dict(t._fields_)[n]
        setattr(a, n, kind(*v) if isinstance(v, tuple) else v)
    return a


def fwd(B=2, L=300, C=100, **over):
    s = (L * C, C)
    return fill(ccv.ccv_linrec_fwd_args_t, dict(B=B, L=L, C=C, x_dtype=ccv.CCV_BF16, g_dtype=ccv.CCV_F32, x=X, x_stride=s, g=G, g_stride=s,
                                                out=OUT, out_stride=s, init_stride=C, final_stride=C, workspace=WS, workspace_bytes=1 << 40), over)


def bwd(B=2, L=300, C=100, **over):
    s = (L * C, C)
    return fill(ccv.ccv_linrec_bwd_args_t, dict(B=B, L=L, C=C, x_dtype=ccv.CCV_BF16, g_dtype=ccv.CCV_F32, x=X, x_stride=s, g=G, g_stride=s,
                                                dout=DO, dout_stride=s, dx=DX, dx_stride=s, dg=DG, dg_stride=s, init_stride=C, dfinal_stride=C,
                                                dinit_stride=C, workspace=WS, workspace_bytes=1 << 40), over)


def upd(B=3, L=1, C=100, **over):
    s = (L * C, C)
    return fill(ccv.ccv_linrec_update_args_t, dict(B=B, L=L, C=C, slots=8, x_dtype=ccv.CCV_BF16, g_dtype=ccv.CCV_F32, x=X, x_stride=s, g=G,
                                                   g_stride=s, out=OUT, out_stride=s, state=H0, state_stride=C), over)


def gn_fwd(rows=20, groups=4, width=24, **over):
    C = groups * width
    return fill(ccv.ccv_group_norm_fwd_args_t, dict(rows=rows, groups=groups, width=width, x_dtype=ccv.CCV_BF16, w_dtype=ccv.CCV_F32, eps=1e-5, x=X,
                                                    x_stride=C, weight=W, bias=B_, gate=Z, gate_stride=C, out=OUT, out_stride=C,
                                                    mean=MEAN, rstd=RSTD), over)


def gn_bwd(rows=20, groups=4, width=24, **over):
    C = groups * width
    return fill(ccv.ccv_group_norm_bwd_args_t, dict(rows=rows, groups=groups, width=width, x_dtype=ccv.CCV_BF16, w_dtype=ccv.CCV_F32, x=X,
                                                    x_stride=C, weight=W, bias=B_, gate=Z, gate_stride=C, dout=DO, dout_stride=C,
                                                    mean=MEAN, rstd=RSTD, dx=DX, dx_stride=C, dgate=DZ, dgate_stride=C, dweight=DW,
                                                    dbias=DB, workspace=WS, workspace_bytes=1 << 30), over)


def rot(B=2, L=30, Hq=4, Hk=2, D=64, **over):
    qs, ks = (L * Hq * D, Hq * D, D), (L * Hk * D, Hk * D, D)
    return fill(ccv.ccv_rotary_args_t, dict(B=B, L=L, Hq=Hq, Hk=Hk, D=D, turned=32, x_dtype=ccv.CCV_BF16, scale=1.0, q=X, q_stride=qs, k=Z,
                                            k_stride=ks, positions=POS, pos_stride=(L, 1), frequencies=FREQ, q_out=OUT, q_out_stride=qs,
                                            k_out=DZ, k_out_stride=ks), over)


CALLS = {"ccv_linrec_fwd": fwd, "ccv_linrec_bwd": bwd, "ccv_linrec_update": upd, "ccv_group_norm_fwd": gn_fwd,
         "ccv_group_norm_bwd": gn_bwd, "ccv_rotary": rot}


def name(call, **over):
    return ccv.STATUS[getattr(ccv, call + "_check")(CALLS[call](**over))]


def cases(table):
    return [pytest.param(call, over, want, id=f"{call}-{want}-{'-'.join(f'{k}={v}' for k, v in over.items())}")
            for call, want, overs in table for over in overs]


LINREC = ("ccv_linrec_fwd", "ccv_linrec_bwd", "ccv_linrec_update")
GROUP = ("ccv_group_norm_fwd", "ccv_group_norm_bwd")

TABLE = [
    *((c, "CCV_OK", [{}, {"C": 0}, {"B": 0}]) for c in LINREC),
    *((c, "CCV_E_SHAPE", [{"B": -1}, {"L": -1}, {"C": -1}, {"L": 2 ** 31 - 8191}, {"C": 2 ** 24 + 1}, {"B": 2 ** 31},
                          {"x_stride": (2 ** 62, 100)}]) for c in LINREC),
    *((c, "CCV_E_DTYPE", [{"x_dtype": 3}, {"x_dtype": -1}, {"g_dtype": 3}]) for c in LINREC),
    *((c, "CCV_E_UNSUPPORTED", [{"normalize": 2}, {"normalize": -1}]) for c in LINREC),
    *((c, "CCV_E_NULL", [{"x": None}, {"g": None}]) for c in LINREC),
    *((c, "CCV_E_LAYOUT", [{"x_stride": (-1, 100)}, {"g_stride": (30000, -100)}, {"L": 2, "x_stride": (0, (16 << 20) + 1)},
                           {"L": 2, "g_stride": (0, (8 << 20) + 1)}]) for c in LINREC),
    *((c, "CCV_OK", [{"x_stride": (0, 0), "g_stride": (0, 0)}, {"L": 2, "x_stride": (0, 16 << 20)}]) for c in LINREC),
    *((c, "CCV_E_SHAPE", [{"N": 3}, {"cu_seqlens": CU, "N": 3}, {"B": 1, "cu_seqlens": CU, "N": -1}, {"B": 1, "cu_seqlens": CU, "N": 2 ** 31}])
      for c in LINREC[:2]),
    *((c, "CCV_OK", [{"B": 1, "cu_seqlens": CU, "N": 3}, {"B": 1, "cu_seqlens": CU, "N": 0}, {"L": 0, "x": None, "g": None}]) for c in LINREC[:2]),
    *((c, "CCV_E_NULL", [{"workspace": None}]) for c in LINREC[:2]),
    *((c, "CCV_E_LAYOUT", [{"workspace": WS + 8}, {"initial_state": H0, "init_stride": -1}]) for c in LINREC[:2]),
    ("ccv_linrec_fwd", "CCV_E_NULL", [{"out": None}]),
    ("ccv_linrec_fwd", "CCV_E_LAYOUT", [{"out_stride": (30000, 99)}, {"out_stride": (0, 100)}, {"out_stride": (30000, 0)},
                                        {"final_state": HT, "final_stride": 99}, {"final_state": HT, "final_stride": 0}]),
    ("ccv_linrec_fwd", "CCV_E_ALIAS", [{"out": X}, {"out": G}, {"initial_state": OUT}, {"final_state": OUT}, {"carries": OUT}, {"final_state": X},
                                       {"carries": G}, {"carries": H0, "initial_state": H0}, {"carries": HT, "final_state": HT},
                                       {"final_state": H0, "initial_state": H0, "init_stride": 0},
                                       {"B": 1, "cu_seqlens": OUT, "N": 3}, {"B": 1, "cu_seqlens": CAR, "N": 3, "carries": CAR}]),
    ("ccv_linrec_fwd", "CCV_OK", [{"final_state": H0, "initial_state": H0}, {"carries": CAR, "final_state": HT, "initial_state": H0},
                                  {"initial_state": H0, "init_stride": 0}, {"B": 1, "final_state": H0, "initial_state": H0, "init_stride": 0},
                                  {"L": 0, "out": None, "initial_state": H0, "final_state": HT, "workspace": None},
                                  {"L": 100, "workspace": None}]),
    ("ccv_linrec_fwd", "CCV_E_SHAPE", [{"B": 2 ** 20, "L": 2 ** 20, "C": 64, "x_stride": (0, 0), "g_stride": (0, 0), "out_stride": (2 ** 27, 64)},
                                       {"initial_state": H0, "init_stride": 2 ** 62}]),
    ("ccv_linrec_bwd", "CCV_E_NULL", [{"dout": None}, {"dx": None}, {"dg": None}]),
    ("ccv_linrec_bwd", "CCV_E_UNSUPPORTED", [{"dinitial_state": DH0}]),
    ("ccv_linrec_bwd", "CCV_E_LAYOUT", [{"dx_stride": (30000, 99)}, {"dg_stride": (0, 100)}, {"dinitial_state": DH0, "initial_state": H0, "dinit_stride": 0}]),
    ("ccv_linrec_bwd", "CCV_E_ALIAS", [{"dx": X}, {"dx": G}, {"dx": DO}, {"dg": G}, {"dx": DG}, {"carries": DX}, {"dfinal_state": DG},
                                       {"dinitial_state": H0, "initial_state": H0}, {"dinitial_state": DHT, "initial_state": H0, "dfinal_state": DHT},
                                       {"dinitial_state": DX, "initial_state": H0}, {"B": 1, "cu_seqlens": DG, "N": 3}]),
    ("ccv_linrec_bwd", "CCV_OK", [{"carries": CAR, "dfinal_state": DHT, "initial_state": H0, "dinitial_state": DH0}, {"dout_stride": (0, 0)},
                                  {"dfinal_state": DHT, "dfinal_stride": 0}]),
    ("ccv_linrec_update", "CCV_E_NULL", [{"state": None}, {"out": None}]),
    ("ccv_linrec_update", "CCV_E_SHAPE", [{"slots": 2}, {"slots": -1}, {"slots": 0, "state": None}]),
    ("ccv_linrec_update", "CCV_OK", [{"slots": 2, "state_indices": CU}, {"slots": 0, "state": None, "state_indices": CU}, {"L": 0, "x": None}, {"L": 5}]),
    ("ccv_linrec_update", "CCV_E_ALIAS", [{"out": X}, {"out": H0}, {"state": G}, {"out": CU, "state_indices": CU}, {"state": CU, "state_indices": CU}]),
    ("ccv_linrec_update", "CCV_E_LAYOUT", [{"out_stride": (99, 1)}, {"state_stride": 99}]),

    *((c, "CCV_OK", [{}, {"gate": None, "dgate": None} if c.endswith("bwd") else {"gate": None}, {"weight": None, "bias": None},
                     {"width": 0, "x": None}, {"x_stride": 0}, {"activation": ccv.CCV_ACT_SILU}]) for c in GROUP),
    *((c, "CCV_E_SHAPE", [{"rows": -1}, {"groups": 0}, {"width": -1}, {"rows": 2 ** 31}, {"groups": 2 ** 13, "width": 2 ** 12},
                          {"groups": 2 ** 25}, {"width": 2 ** 25, "groups": 1}, {"x_stride": 2 ** 60}]) for c in GROUP),
    *((c, "CCV_E_DTYPE", [{"x_dtype": 3}, {"w_dtype": -1}]) for c in GROUP),
    *((c, "CCV_E_UNSUPPORTED", [{"activation": 2}, {"activation": -1}]) for c in GROUP),
    *((c, "CCV_E_LAYOUT", [{"x_stride": -1}, {"gate_stride": -96}]) for c in GROUP),
    *((c, "CCV_E_NULL", [{"x": None}]) for c in GROUP),
    ("ccv_group_norm_fwd", "CCV_OK", [{"rows": 0, "x": None, "out": None}, {"mean": None, "rstd": None}, {"eps": 0.0}]),
    ("ccv_group_norm_fwd", "CCV_E_UNSUPPORTED", [{"eps": -1.0}, {"eps": math.inf}, {"eps": math.nan}]),
    ("ccv_group_norm_fwd", "CCV_E_NULL", [{"out": None}]),
    ("ccv_group_norm_fwd", "CCV_E_LAYOUT", [{"out_stride": 95}, {"out_stride": 0}]),
    ("ccv_group_norm_fwd", "CCV_E_ALIAS", [{"out": X}, {"out": Z}, {"mean": W}, {"mean": RSTD}, {"rstd": OUT}]),
    ("ccv_group_norm_bwd", "CCV_E_NULL", [{"dout": None}, {"mean": None}, {"rstd": None}, {"workspace": None}]),
    ("ccv_group_norm_bwd", "CCV_E_UNSUPPORTED", [{"gate": None}]),
    ("ccv_group_norm_bwd", "CCV_E_LAYOUT", [{"dx_stride": 95}, {"dgate_stride": 0}, {"workspace": WS + 4}]),
    ("ccv_group_norm_bwd", "CCV_E_ALIAS", [{"dx": X}, {"dx": DO}, {"dgate": Z}, {"dgate": DX}, {"dweight": W}, {"dbias": DW}, {"dweight": MEAN}]),
    ("ccv_group_norm_bwd", "CCV_OK", [{"dx": None, "dgate": None, "dweight": None, "dbias": None, "workspace": None},
                                      {"rows": 0, "x": None, "dout": None, "mean": None, "rstd": None, "workspace": None}]),

    ("ccv_rotary", "CCV_OK", [{}, {"Hk": 0, "k": None, "k_out": None}, {"Hq": 0, "q": None, "q_out": None}, {"B": 0, "q": None}, {"L": 0, "q": None},
                              {"turned": 0, "positions": None, "frequencies": None}, {"q_out": X}, {"q_out": X, "k_out": Z}, {"pos_stride": (0, 1)},
                              {"pos_stride": (0, 0)}, {"q_stride": (0, 0, 0)}, {"interleaved": 1, "inverse": 1}, {"scale": 0.0}]),
    ("ccv_rotary", "CCV_E_SHAPE", [{"B": -1}, {"L": -1}, {"Hq": -1}, {"Hk": -1}, {"D": 0}, {"turned": -2}, {"turned": 66}, {"turned": 3},
                                   {"Hq": 65537}, {"B": 2 ** 16, "L": 2 ** 15}, {"q_stride": (2 ** 62, 256, 64)}, {"pos_stride": (2 ** 62, 1)},
                                   {"B": 1, "L": 2 ** 24, "D": 2048, "Hk": 0}]),
    ("ccv_rotary", "CCV_E_DTYPE", [{"x_dtype": 3}]),
    ("ccv_rotary", "CCV_E_UNSUPPORTED", [{"D": 2049}, {"interleaved": 2}, {"inverse": -1}, {"scale": math.nan}, {"scale": math.inf}]),
    ("ccv_rotary", "CCV_E_NULL", [{"q": None}, {"k": None}, {"q_out": None}, {"k_out": None}, {"positions": None}, {"frequencies": None}]),
    ("ccv_rotary", "CCV_E_LAYOUT", [{"q_stride": (7680, 256, -64)}, {"q_out_stride": (7680, 256, 63)}, {"q_out_stride": (7680, 255, 64)},
                                    {"k_out_stride": (0, 128, 64)}, {"pos_stride": (-1, 1)}]),
    ("ccv_rotary", "CCV_E_ALIAS", [{"q_out": X, "q_stride": (0, 256, 64)}, {"q_out": Z}, {"k_out": X}, {"k_out": OUT}, {"q_out": POS}, {"k_out": FREQ}]),
]


@pytest.mark.parametrize("call,over,want", cases(TABLE))
def test_checks(call, over, want):
    assert name(call, **over) == want


@pytest.mark.parametrize("call", sorted(CALLS))
def test_malformed(call):
    assert getattr(ccv.lib(), call + "_check")(None) == -1
    a = CALLS[call]()
    a.struct_size -= 8
    assert ccv.STATUS[getattr(ccv, call + "_check")(a)] == "CCV_E_ABI"


@pytest.mark.parametrize("call", ["ccv_linrec_fwd", "ccv_linrec_bwd", "ccv_group_norm_bwd"])
def test_workspaces(call):
    make, size = CALLS[call], getattr(ccv, call + "_workspace_size")
    need = size(make(workspace=None, workspace_bytes=0))
    assert need > 0
    assert name(call, workspace_bytes=need) == "CCV_OK"
    assert name(call, workspace_bytes=need - 1) == "CCV_E_SHAPE"
    if call == "ccv_group_norm_bwd":
        assert need % (2 * 96 * 4) == 0
        assert size(make(dweight=None, dbias=None)) == size(make(rows=0)) == size(make(width=0)) == 0
        assert ccv.STATUS[size(make(rows=-1))] == "CCV_E_SHAPE"
    else:
        assert size(make(B=0)) == size(make(C=0)) == 0
        # packed rows: a number a step more
        assert size(make(B=1, cu_seqlens=CU, N=3)) >= size(make(B=1)) + 4 * 300
    if call == "ccv_linrec_bwd":
        # the states before the three chunks of both rows, and the words of a pass that makes them
        assert need >= size(make(carries=CAR)) + 2 * 3 * 100 * 4


def test_binding_refusals():
    x, g, h0 = ref.inputs(2, 5, 8)
    cu = torch.tensor([0, 5], dtype=torch.int32)
    f, b, u = ccv.gated_linear_recurrence_fwd, ccv.gated_linear_recurrence_bwd, ccv.gated_linear_recurrence_update
    for call in (lambda: f(x, g), lambda: ccv.gated_linear_recurrence_fn(x, g), lambda: b(x, g, x), lambda: u(x, g, h0), lambda: u(x[:, 0], g[:, 0], h0),
                 lambda: ccv.group_norm_fwd(x, 2), lambda: ccv.group_norm_fn(x, 2), lambda: ccv.group_norm_bwd(x, 2, None, None, x, h0, h0),
                 lambda: ccv.rotary_fwd(x, None, cu, torch.ones(2, dtype=torch.float64))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call, match in (
            (lambda: f(x[0], g[0]), r"\[B, L, C\]"), (lambda: f(x, g[:, :4]), r"\[B, L, C\]"), (lambda: f(x.double(), g), "float32, float16 or bfloat16"),
            (lambda: f(x, g, final_state_out=h0), "return_final_state"), (lambda: u(x[0, 0], g[0, 0], h0), r"\[B, L, C\]"),
            (lambda: ccv.group_norm_fwd(x, 3), "divide"), (lambda: ccv.group_norm_fwd(x, 0), "divide"), (lambda: ccv.group_norm_fwd(x[0, 0], 1), r"\.\.\., C"),
            (lambda: ccv.group_norm_fwd(x, 2, activation="gelu"), "activation"), (lambda: ccv.group_norm_fwd(x, 2, torch.ones(7)), r"\[C\]"),
            (lambda: ccv.group_norm_fwd(x, 2, torch.ones(8), torch.ones(8).half()), "weight's dtype"), (lambda: ccv.group_norm_fwd(x.double(), 2), "float32"),
            (lambda: ccv.group_norm_fwd(x, 2, gate=x.half()), "gate"), (lambda: ccv.group_norm_fwd(x, 2, gate=x[:1]), "gate"),
            (lambda: ccv.rotary_fwd(x[:1], None, cu, torch.ones(2, dtype=torch.float64)), "positions"),
            (lambda: ccv.rotary_fwd(h0, None, cu, torch.ones(2, dtype=torch.float64)), "expected q"),
            (lambda: ccv.rotary_fwd(x, x.half(), cu, torch.ones(2, dtype=torch.float64)), "k must"),
            (lambda: ccv.rotary_fwd(x, x[:1], cu, torch.ones(2, dtype=torch.float64)), "k must"),
            (lambda: ccv.rotary_fwd(x, None, cu.long(), torch.ones(2, dtype=torch.float64)), "positions"),
            (lambda: ccv.rotary_fwd(x, None, cu, torch.ones(2)), "frequencies"),
            (lambda: ccv.rotary_fwd(x, None, cu, torch.ones(5, dtype=torch.float64)), "frequencies")):
        with pytest.raises(ValueError, match=match):
            call()


# ---- what is checked once the tensors are on a GPU, with the calls left out

@pytest.fixture
def calls_do_nothing(monkeypatch):
    monkeypatch.setattr(ccv, "_one_device", lambda x, **others: x.device)
    for n in ("ccv_linrec_fwd", "ccv_linrec_bwd", "ccv_linrec_update", "ccv_group_norm_fwd", "ccv_group_norm_bwd", "ccv_rotary"):
        monkeypatch.setitem(ccv._CALLS, n, lambda *values: None)


def test_refusals_behind_the_device(calls_do_nothing):
    x, g, h0 = ref.inputs(2, 5, 8)
    f, b, u = ccv.gated_linear_recurrence_fwd, ccv.gated_linear_recurrence_bwd, ccv.gated_linear_recurrence_update
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    gn, gb = ccv.group_norm_fwd, ccv.group_norm_bwd
    stats = torch.zeros(2, 5, 2)
    freq = torch.ones(2, dtype=torch.float64)
    q, pos = torch.zeros(2, 5, 3, 8), torch.zeros(2, 5, dtype=torch.int32)
    for call, match in (
            (lambda: f(x, g, cu_seqlens=i32(0, 5)), "B = 1|one row"), (lambda: f(x[:1], g[:1], cu_seqlens=torch.zeros(2, dtype=torch.int64)), "int32"),
            (lambda: f(x, g, initial_state=h0[:1]), "initial_state"), (lambda: f(x, g, initial_state=h0.half()), "initial_state"),
            (lambda: f(x, g, return_final_state=True, final_state_out=h0[:, :4]), "final_state_out"),
            (lambda: f(x, g, return_final_state=True, final_state_out=torch.zeros(8, 2).t()), "unit stride"),
            (lambda: f(x, g, out=x.half()), "out"), (lambda: f(x, g, out=x[:1]), "out"), (lambda: f(x, g, out=torch.zeros(2, 8, 5).transpose(1, 2)), "out"),
            (lambda: b(x, g, x.half()), "dout"), (lambda: b(x, g, x[:1]), "dout"), (lambda: b(x, g, x, return_dinitial_state=True), "initial_state"),
            (lambda: b(x, g, x, carries=torch.zeros(2, 2, 8)), "carries"), (lambda: b(x, g, x, carries=torch.zeros(2, 1, 8).half()), "carries"),
            (lambda: b(x, g, x, dfinal_state=h0[:1]), "dfinal_state"),
            (lambda: u(x, g, h0[:1]), "more rows"), (lambda: u(x, g, h0[:, :4]), "state"), (lambda: u(x, g, h0.half()), "state"),
            (lambda: u(x, g, torch.zeros(8, 2).t()), "unit stride"), (lambda: u(x, g, h0, i32(0)), "state_indices"),
            (lambda: u(x, g, h0, torch.zeros(2, dtype=torch.int64)), "state_indices"), (lambda: u(x, g, h0, out=x[:, 0]), "out"),
            (lambda: gn(x, 2, out=x.half()), "out"), (lambda: gn(x, 2, out=torch.zeros(2, 5, 16)[..., ::2]), "out"),
            (lambda: gb(x, 2, None, None, x.half(), stats, stats), "dout"), (lambda: gb(x, 2, None, None, x, stats[:1], stats), "mean"),
            (lambda: gb(x, 2, None, None, x, stats, stats.half()), "rstd"), (lambda: gb(x, 2, None, None, x, stats, stats, weight_dtype=torch.int8), "weight_dtype"),
            (lambda: ccv.rotary_fwd(q, None, pos, freq, k_out=q), "k_out"), (lambda: ccv.rotary_fwd(q, None, pos, freq, q_out=q.half()), "q_out"),
            (lambda: ccv.rotary_fwd(q, q, pos, freq, k_out=q[:1]), "k_out"),
            (lambda: ccv.rotary_fwd(q, None, pos, freq, q_out=torch.zeros(2, 5, 8, 3).transpose(2, 3)), "unit stride"),
            (lambda: ccv.rotary_fwd(torch.zeros(2, 5, 3, 2049), None, pos, freq), "2048")):
        with pytest.raises(ValueError, match=match):
            call()


def test_copies_are_named(calls_do_nothing):
    x, g, h0 = ref.inputs(2, 5, 8)
    info = {}
    ccv.gated_linear_recurrence_fwd(x, torch.zeros(2, 8, 5).transpose(1, 2), initial_state=torch.zeros(8, 2).t(), info=info)
    assert info["copied"] == ["g", "initial_state"]
    ccv.gated_linear_recurrence_fwd(x, g[:, :1].expand(2, 5, 8), info=info)
    assert info["copied"] == []


def test_written_tensors_have_new_versions(calls_do_nothing):
    x, g, h0 = ref.inputs(2, 5, 8)
    q, pos, freq = torch.zeros(2, 5, 3, 8), torch.zeros(2, 5, dtype=torch.int32), torch.ones(2, dtype=torch.float64)
    read = (x, g, q, pos)
    at = [t._version for t in read]

    def writes(call, *given):
        before = [t._version for t in given]
        call()
        assert all(t._version > v for t, v in zip(given, before))

    out, out1, k = torch.empty_like(x), torch.empty_like(x), torch.empty_like(q)
    ccv.gated_linear_recurrence_fwd(x, g, initial_state=h0, return_final_state=True)
    assert h0._version == 0
    writes(lambda: ccv.gated_linear_recurrence_fwd(x, g, initial_state=h0, return_final_state=True, final_state_out=h0, out=out), h0, out)
    writes(lambda: ccv.gated_linear_recurrence_update(x, g, h0, out=out), h0, out)
    writes(lambda: ccv.group_norm_fwd(x, 2, out=out1), out1)
    writes(lambda: ccv.rotary_fwd(torch.zeros_like(q), k, pos, freq, q_out=torch.empty_like(q), k_out=k), k)
    assert [t._version for t in read] == at


# ---- autograd, with the C calls' results from the formulas

def linrec_by_reference(monkeypatch):
    def fwd(x, g, cu_seqlens=None, initial_state=None, return_final_state=False, normalize=False, return_carries=False, **kw):
        r = ref.linrec(x.detach(), g.detach(), None, None if initial_state is None else initial_state.detach(), normalize)
        return (r["out"][0].to(x.dtype),) + ((r["ht"][0].float(),) if return_final_state else ()) + ((torch.zeros(1),) if return_carries else ())

    def bwd(x, g, dout, cu_seqlens=None, initial_state=None, dfinal_state=None, normalize=False, carries=None, return_dinitial_state=False):
        with torch.no_grad():
            r = ref.linrec(x, g, None, initial_state, normalize, dout, dfinal_state)
        return r["dx"][0].to(x.dtype), r["dg"][0].to(g.dtype), r["dh0"][0].float() if return_dinitial_state else None

    monkeypatch.setattr(ccv, "gated_linear_recurrence_fwd", fwd)
    monkeypatch.setattr(ccv, "gated_linear_recurrence_bwd", bwd)


def group_norm_by_reference(monkeypatch):
    def fwd(x, num_groups, weight=None, bias=None, gate=None, activation=None, eps=1e-5, return_stats=False, out=None):
        r = ref.group_norm(x.detach(), num_groups, weight.detach(), bias.detach(), None if gate is None else gate.detach(), activation == "silu", eps)
        return tuple(r[n][0].float() for n in ("out", "mean", "rstd"))

    def bwd(x, num_groups, weight, bias, dout, mean, rstd, gate=None, activation=None, *want):
        r = ref.group_norm(x, num_groups, weight, bias, gate, activation == "silu", 1e-5, dout)
        return tuple(r[n][0].float() if n in r else None for n in ("dx", "dw", "db", "dz"))

    monkeypatch.setattr(ccv, "group_norm_fwd", fwd)
    monkeypatch.setattr(ccv, "group_norm_bwd", bwd)


def rotary_by_reference(monkeypatch):
    def fwd(q, k, positions, frequencies, interleaved=False, scale=1.0, inverse=False, q_out=None, k_out=None):
        turn = lambda t: None if t is None else ref.rotary(t.detach().cpu(), positions.cpu(), frequencies, interleaved, scale, inverse)[0].float()  # noqa: E731
        return turn(q), turn(k)

    monkeypatch.setattr(ccv, "rotary_fwd", fwd)


def linrec_call(device="cpu"):
    x, g, h0 = ref.inputs(2, 9, 6)
    leaves = [t.to(device).requires_grad_() for t in (x, g, h0)]
    return leaves, lambda: ccv.gated_linear_recurrence_fn(*leaves[:2], initial_state=leaves[2], normalize=True)


def group_norm_call(device="cpu"):
    gen = torch.Generator().manual_seed(3)
    leaves = [torch.randn(*s, generator=gen).to(device).requires_grad_() for s in ((5, 12), (12,), (12,), (5, 12))]
    return leaves, lambda: ccv.group_norm_fn(leaves[0], 3, *leaves[1:], activation="silu")


def rotary_call(device="cpu"):
    gen = torch.Generator().manual_seed(4)
    leaves = [torch.randn(2, 5, h, 8, generator=gen).to(device).requires_grad_() for h in (3, 1)]
    pos, freq = torch.arange(10, dtype=torch.int32).view(2, 5).to(device), torch.tensor([1.0, 0.1, 0.01], dtype=torch.float64, device=device)
    return leaves, lambda: torch.cat([t.flatten() for t in ccv.rotary_fn(*leaves, pos, freq)])


MADE = {"linrec": (linrec_call, linrec_by_reference), "group_norm": (group_norm_call, group_norm_by_reference),
        "rotary": (rotary_call, rotary_by_reference)}


def check_second_derivative(leaves, run, linear):
    """Refused where a gradient depends on anything (a linear call's only through the incoming one); first derivatives are
    as without create_graph."""
    plain = torch.autograd.grad(run().sum(), leaves)
    for loss in [lambda: run().square().sum()] + [lambda: run().sum()] * (not linear):
        grads = torch.autograd.grad(loss(), leaves, create_graph=True)
        for g in grads:
            assert g.requires_grad
            with pytest.raises(RuntimeError, match="second derivative"):
                torch.autograd.grad(g.square().sum(), leaves, retain_graph=True, allow_unused=True)
    for g, p in zip(torch.autograd.grad(run().sum(), leaves, create_graph=True), plain):
        assert torch.equal(g, p)


@pytest.mark.parametrize("made", sorted(MADE))
def test_second_derivatives_are_refused(monkeypatch, made):
    make, by = MADE[made]
    by(monkeypatch)
    check_second_derivative(*make(), made == "rotary")


@pytest.mark.gpu
@pytest.mark.parametrize("made", sorted(MADE))
def test_second_derivatives_on_the_gpu(made):
    check_second_derivative(*MADE[made][0]("cuda"), made == "rotary")


def advanced(x, advance):
    """A cache that was the initial state of a differentiable call, advanced before its backward: torch raises."""
    leaves, cache = x[:2], x[2].detach().clone()
    loss = ccv.gated_linear_recurrence_fn(*leaves, initial_state=cache).sum()
    advance(leaves, cache)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def by_update(leaves, cache):
    ccv.gated_linear_recurrence_update(*(t.detach()[:, 0] for t in leaves), cache)


def by_prefill(leaves, cache):
    with torch.no_grad():
        ccv.gated_linear_recurrence_fwd(*leaves, initial_state=cache, return_final_state=True, final_state_out=cache)


@pytest.mark.parametrize("advance", [by_update, by_prefill])
def test_a_state_advanced_before_the_backward(calls_do_nothing, advance):
    advanced(linrec_call()[0], advance)


@pytest.mark.gpu
@pytest.mark.parametrize("advance", [by_update, by_prefill])
def test_a_state_advanced_before_the_backward_on_the_gpu(advance):
    advanced(linrec_call("cuda")[0], advance)


# ---- the references and the frequencies

def differences(loss, args, got, names):
    """Central differences: rounding 1e-16 / 1e-5 and e^2 curvature, far below the 1e-7 allowed."""
    e = 1e-5
    for i, n in enumerate(names):
        flat, want = args[i].reshape(-1), got[n][0].reshape(-1)
        for j in range(0, flat.numel(), max(1, flat.numel() // 12)):
            keep = float(flat[j])
            flat[j] = keep + e
            up = loss(args)
            flat[j] = keep - e
            down = loss(args)
            flat[j] = keep
            assert abs((up - down) / (2 * e) - float(want[j])) < 1e-7 * (1 + abs(float(want[j]))), (n, j)


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("lengths", [None, [3, 0, 4]])
def test_recurrence_gradients_against_differences(lengths, normalize):
    x, g, h0 = (t.double() for t in ref.inputs(1, 8, 3, seed=7, seqs=3 if lengths else 1, slow=0.6))
    g = g - 0.05                            # the root's curvature grows as 1 / s^3
    gen = torch.Generator().manual_seed(8)
    dout, dht = torch.randn(1, 8, 3, generator=gen).double(), torch.randn(h0.shape, generator=gen).double()
    if lengths:
        dout[:, sum(lengths):] = 0
    got = ref.linrec(x, g, lengths, h0, normalize, dout, dht)

    def loss(args):
        r = ref.linrec(args[0], args[1], lengths, args[2], normalize)
        return float((r["out"][0] * dout).sum() + (r["ht"][0] * dht).sum())

    differences(loss, [x, g, h0], got, ("dx", "dg", "dh0"))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("silu", [False, True])
def test_group_norm_gradients_against_differences(silu, gated):
    gen = torch.Generator().manual_seed(9)
    x, w, b, z, dout = (torch.randn(*s, generator=gen).double() for s in ((4, 12), (12,), (12,), (4, 12), (4, 12)))
    got = ref.group_norm(x, 3, w, b, z if gated else None, silu, 1e-2, dout)

    def loss(args):
        return float((ref.group_norm(args[0], 3, args[1], args[2], args[3] if gated else None, silu, 1e-2)["out"][0] * dout).sum())

    differences(loss, [x, w, b] + [z] * gated, got, ("dx", "dw", "db") + ("dz",) * gated)


def test_rotary_reference():
    """A turn keeps a pair's length, the inverse takes it back, and differences of positions are what products see."""
    gen = torch.Generator().manual_seed(10)
    x, y = torch.randn(1, 6, 1, 8, generator=gen).double(), torch.randn(1, 6, 1, 8, generator=gen).double()
    freq = torch.tensor([1.0, 0.3, 0.01], dtype=torch.float64)
    pos = torch.arange(6, dtype=torch.int32)[None] * 7
    for inter in (False, True):
        t = ref.rotary(x, pos, freq, inter)[0]
        assert torch.allclose(t.norm(dim=-1), x.norm(dim=-1)) and torch.equal(t[..., 6:], x[..., 6:])
        assert torch.allclose(ref.rotary(t, pos, freq, inter, inverse=True)[0], x)
        far = (t * ref.rotary(y, pos + 3, freq, inter)[0]).sum(-1)
        assert torch.allclose(far, (ref.rotary(x, pos + 100, freq, inter)[0] * ref.rotary(y, pos + 103, freq, inter)[0]).sum(-1))


def test_frequencies():
    f, s = ccv.rotary_frequencies(64, device="cpu")
    want = torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64)
    assert f.dtype == torch.float64 and s == 1.0 and torch.allclose(f, want, rtol=1e-15, atol=0)
    f, s = ccv.rotary_frequencies(64, scaling="linear", factor=8, device="cpu")
    assert s == 1.0 and torch.allclose(f, want / 8, rtol=1e-15, atol=0)
    f, s = ccv.rotary_frequencies(64, scaling="base", factor=8, device="cpu")
    assert s == 1.0 and float(f[0]) == 1.0 and math.isclose(float(f[-1]), float(want[-1]) / 8, rel_tol=1e-13)
    f, s = ccv.rotary_frequencies(64, scaling="parts", factor=8, original_length=2048, device="cpu")
    assert math.isclose(s, 0.1 * math.log(8) + 1)
    turns = 2048 * want / (2 * math.pi)
    share = f / want
    assert torch.equal(f[turns > 32 * 1.4], want[turns > 32 * 1.4])          # a pair and more (10000^(1/32) = 1.33) from the ends
    assert torch.allclose(share[turns < 1 / 1.4], torch.full((), 1 / 8, dtype=torch.float64))
    assert bool((share[1:] <= share[:-1]).all()) and bool(((share < 1) & (share > 1 / 8)).any())
    f, _ = ccv.rotary_frequencies(2, scaling="base", factor=8, device="cpu")
    assert f.tolist() == [1.0]
    for kw in (dict(turned=0), dict(turned=3), dict(turned=8, scaling="other"), dict(turned=8, base=1.0), dict(turned=8, factor=0.5),
               dict(turned=8, scaling="parts"), dict(turned=8, scaling="parts", original_length=0), dict(turned=8, fast=1.0, slow=2.0),
               dict(turned=8, base=math.nan)):
        with pytest.raises(ValueError):
            ccv.rotary_frequencies(**kw, device="cpu")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("L", [1, 2, 70])
def test_rounded_references_are_within_their_bounds(dtype, L):
    """64-bit results rounded once pass the bounds that the kernels are held to; results two spacings off do not."""
    x, g, h0 = ref.inputs(1, L, 40, dtype, seed=L)
    want = ref.linrec(x, g, None, h0, True, x, h0)
    for n in ("out", "dx", "dg"):
        ref.assert_within(n, want[n][0].to(ref.DT[dtype]), want[n])
    with pytest.raises(AssertionError):
        ref.assert_within("out", (want["out"][0] * (1 + 2.0 ** -6)).to(ref.DT[dtype]), want["out"])
