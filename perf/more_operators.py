"""The operators of a recurrent layer beside the delta rule, as they are measured.

A layer whose state is one number a channel convolves its input (the causal conv1d of this package) and runs a gated
linear recurrence over the result; its heads leave it through a group norm and a gate.  Layers that keep queries and
keys turn them by the steps' positions, which the sequence tables of a packed row give.  Four kinds of case:

  "scan"    the gated linear recurrence over whole sequences ("fwd": outputs and final states; "train": these and every
            gradient)
  "step"    the same recurrence for a few new steps against states in a cache, advanced in place
  "gnorm"   group norm of each step's channels with an activation or a gate ("fwd", or "train": outputs and gradients)
  "rotary"  queries and keys turned by their positions ("fwd", or "train")

Where `own` is false everything is computed by elementary torch operations in 32 bits (angles in 64); where it is true
by this package's kernels.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-5


# ---- the cases ----------------------------------------------------------------------------

def _scan(name, mode, B, L, C, dtype, gate, normalize=False, seqs=0, states=True, fill=1.0, pad=0):
    return {"name": name, "op": "scan", "mode": mode, "B": B, "L": L, "C": C, "dtype": dtype, "gate": gate,
            "normalize": normalize, "seqs": seqs, "states": states, "fill": fill, "pad": pad}


def _step(name, B, T, slots, C, dtype, gate, normalize, idle):
    return {"name": name, "op": "step", "B": B, "T": T, "slots": slots, "C": C, "dtype": dtype, "gate": gate,
            "normalize": normalize, "idle": idle}


def _gnorm(name, mode, rows, C, groups, dtype, weight, activation, gated, pad=0):
    return {"name": name, "op": "gnorm", "mode": mode, "rows": rows, "C": C, "groups": groups, "dtype": dtype,
            "weight": weight, "activation": activation, "gated": gated, "pad": pad}


def _rotary(name, mode, B, L, Hq, Hk, D, turned, dtype, interleaved, scaling="none", far=0, fused=True):
    return {"name": name, "op": "rotary", "mode": mode, "B": B, "L": L, "Hq": Hq, "Hk": Hk, "D": D, "turned": turned,
            "dtype": dtype, "interleaved": interleaved, "scaling": scaling, "far": far, "fused": fused}


def listed():
    return [
        # a short prompt of one request in fp32, the 64 channels of the small conv workload: what a call costs at the least
        _scan("scan fwd f32 1x2048x64", "fwd", 1, 2048, 64, "f32", "f32", states=False),
        # prefill of the bf16 conv workload's batch (4 x 4096, 2048 channels) with carried states
        _scan("scan fwd bf16 4x4096x2048", "fwd", 4, 4096, 2048, "bf16", "bf16", normalize=True),
        # serving prefill: the packed conv workload (65536 steps, 64 requests, 2560 channels), decays in fp32
        _scan("scan fwd f16 packed 65536x2560", "fwd", 1, 65536, 2560, "f16", "f32", normalize=True, seqs=64),
        # the million-step conv workload: very long sequences of few channels
        _scan("scan fwd f32 2x1048576x128", "fwd", 2, 1048576, 128, "f32", "f32"),
        # a training step of the strided conv workload's 4096 channels
        _scan("scan train bf16 2x4096x4096", "train", 2, 4096, 4096, "bf16", "bf16", normalize=True, states=False),
        # training in fp32 on a packed row of odd lengths and an odd width, with steps behind the last sequence
        _scan("scan train f32 packed 3011x333", "train", 1, 3011, 333, "f32", "f32", seqs=7, fill=0.97),
        # decoding: the update workload's 256 requests and 4096 channels, one step each
        _step("step bf16 B256 C4096", 256, 1, 256, 4096, "bf16", "bf16", True, 0),
        # a few requests of a larger cache, one row idle
        _step("step f16 B5 C2560 of 64 slots", 5, 1, 64, 2560, "f16", "f32", True, 1),
        # the heads' norm and gate of a decode step
        _gnorm("gnorm fwd bf16 256x4096 g32", "fwd", 256, 4096, 32, "bf16", "bf16", "silu", True),
        # the same in training: 65536 tokens of 20 heads of 128, read out of a wider buffer
        _gnorm("gnorm train f16 65536x2560 g20", "train", 65536, 2560, 20, "f16", "f32", "silu", True, pad=512),
        # training on 4 x 4096 tokens: 16 query and 4 key heads of 128, views of the projections' buffer
        _rotary("rotary train bf16 4x4096 h16+4", "train", 4, 4096, 16, 4, 128, 128, "bf16", False),
        # decoding far into a long context: 256 requests, half of each head turned, adjacent pairs
        _rotary("rotary fwd f16 256x1 h32+8", "fwd", 256, 1, 32, 8, 128, 64, "f16", True, "parts", 1 << 20),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["scan", "scan", "scan", "step", "gnorm", "gnorm", "rotary"])
    mark = {"draw": rng.randrange(1 << 20)}
    dtype = rng.choice(["f32", "f16", "bf16"])
    gate = rng.choice([dtype, "f32", "bf16"])
    if kind == "scan":
        mode = rng.choice(["fwd", "train"])
        C = rng.choice([64, 128, 2048, 2560, 4096, _log(rng, 1, 8192), _log(rng, 1, 8192)])
        T = min(_log(rng, 1, 1 << 18), max(1, (1 << (26 if mode == "fwd" else 25)) // C))
        seqs = rng.choice([0, 0, rng.randint(1, 40)])
        B = 1 if seqs else max(1, min(rng.choice([1, 2, 4, 8]), T // 100))
        return _scan("", mode, B, max(1, T // B), C, dtype, gate, rng.random() < 0.5, seqs, rng.random() < 0.6,
                     rng.choice([1.0, 1.0, 0.9]), rng.choice([0, 0, 8, 3])) | mark
    if kind == "step":
        B = _log(rng, 1, 512)
        return _step("", B, rng.choice([1, 1, 1, 2, 4]), B + rng.randint(0, 64), _log(rng, 1, 8192), dtype, gate,
                     rng.random() < 0.5, rng.randint(0, min(B - 1, 3))) | mark
    if kind == "gnorm":
        groups = rng.choice([1, 2, 4, 8, 16, 20, 32, rng.randint(1, 40)])
        width = rng.choice([32, 64, 128, 256, _log(rng, 1, 1000)])
        rows = max(1, min(_log(rng, 1, 65536), (1 << 26) // (groups * width)))
        return _gnorm("", rng.choice(["fwd", "train"]), rows, groups * width, groups, dtype, rng.choice(["f32", dtype]),
                      rng.choice(["silu", "silu", "none"]), rng.random() < 0.6, rng.choice([0, 0, 8, 3])) | mark
    Hq = rng.choice([1, 2, 8, 16, 32, rng.randint(1, 40)])
    Hk = rng.choice([0, 1, Hq, max(1, Hq // 4)])
    D = rng.choice([64, 128, 128, 256, 2 * rng.randint(1, 100)])
    T = min(_log(rng, 1, 1 << 16), (1 << 25) // (Hq * D))
    B = max(1, min(rng.choice([1, 2, 4, 256]), T))
    return _rotary("", rng.choice(["fwd", "train"]), B, max(1, T // B), Hq, Hk, D, rng.choice([D, D, D // 4 * 2 or D]),
                   dtype, rng.random() < 0.5, rng.choice(["none", "linear", "base", "parts"]),
                   rng.choice([0, 0, _log(rng, 1, 1 << 24)]), rng.random() < 0.7) | mark


def _lengths(count, total, gen):
    """`count` lengths of sum `total`, some of them zero, as a list."""
    w = torch.empty(count, dtype=torch.float64).exponential_(generator=gen) + 0.1
    if count > 4:
        w[torch.randint(0, count, (max(1, count // 16),), generator=gen)] = 0.0
    edges = torch.floor(torch.cumsum(w / w.sum(), 0) * total + 1e-9).to(torch.int64)
    edges[-1] = total
    return torch.diff(edges, prepend=torch.zeros(1, dtype=torch.int64))


# ---- inputs -------------------------------------------------------------------------------

def _silu(x):
    return x / (1 + torch.exp(-x))


def _scan_inputs(case, lead, gen):
    """x as it leaves the conv (SiLU); log decays -8 softplus(c) sigmoid(r), with c such that a channel's slowest decay
    lies between 0.9 and 0.999 a step."""
    C, pad = case["C"], case.get("pad", 0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x = _silu(rand(*lead, C + pad)).to(_DT[case["dtype"]])[..., :C]
    slow = -torch.log(0.9 + 0.099 * torch.rand(C, device="cuda", generator=gen))
    g = rand(*lead, C).neg_().exp_().add_(1).reciprocal_().mul_(-slow).to(_DT[case["gate"]])
    return x, g


def _frequencies(case):
    """Radians a position of each pair, in 64 bits: base^(-2i/d), with the scalings for contexts eight times as long: every
    position divided, the base raised, or only the pairs divided that turn too slowly to have been seen whole."""
    d, base, factor, before = case["turned"], 10000.0, 8.0, 8192
    if case["scaling"] == "base":
        base *= factor ** (d / max(d - 2, 1))
    i = torch.arange(d // 2, dtype=torch.float64)
    f = base ** (-2 * i / d)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "parts":
        at = lambda turns: d * math.log(before / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), d // 2 - 1)
        whole = 1 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f / factor * (1 - whole) + f * whole
    return f.cuda(), 0.1 * math.log(factor) + 1 if case["scaling"] == "parts" else 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    rand = lambda *n: torch.randn(*n, device="cuda", generator=gen)  # noqa: E731
    if op == "scan":
        B, L, C, N = case["B"], case["L"], case["C"], case["seqs"]
        s["x"], s["g"] = _scan_inputs(case, (B, L), gen)
        s["cu"] = None
        if N:
            lengths = _lengths(N, max(1, int(L * case["fill"])), host)
            cu = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)])
            s["cu"] = cu.to(torch.int32).cuda()
            live = lengths > 0
            s["live"], s["first"], s["last"] = live.cuda(), cu[:-1][live].cuda(), (cu[1:][live] - 1).cuda()
            s["end"] = int(cu[-1])
        s["h0"] = rand(N or B, C) * 0.5 if case["states"] else None
        if case["mode"] == "train":
            s["dout"] = rand(B, L, C).to(s["x"].dtype)
            s["dht"] = rand(N or B, C) * 0.5 if case["states"] else None
            for n in ("x", "g", "h0"):
                if s[n] is not None:
                    s[n] = s[n].detach().requires_grad_()
    elif op == "step":
        s["x"], s["g"] = _scan_inputs(case, (case["B"], case["T"]), gen)
        s["state"] = rand(case["slots"], case["C"]) * 0.5
        slots = torch.randperm(case["slots"], device="cuda", generator=gen)[: case["B"]].to(torch.int32)
        if case["idle"]:
            slots[torch.randperm(case["B"], device="cuda", generator=gen)[: case["idle"]]] = -1
        s["slots"] = slots
    elif op == "gnorm":
        rows, C, dt, wd = case["rows"], case["C"], _DT[case["dtype"]], _DT[case["weight"]]
        s["x"] = (rand(rows, C + case["pad"]) * 1.5 + 0.3).to(dt)[..., :C]
        s["z"] = rand(rows, C).to(dt) if case["gated"] else None
        s["w"], s["b"] = (1 + 0.1 * rand(C)).to(wd), (0.1 * rand(C)).to(wd)
        if case["mode"] == "train":
            s["dout"] = rand(rows, C).to(dt)
            for n in ("x", "z", "w", "b"):
                if s[n] is not None:
                    s[n] = s[n].detach().requires_grad_()
    else:
        B, L, Hq, Hk, D, dt = (case[n] for n in ("B", "L", "Hq", "Hk", "D", "dtype"))
        q, k = (rand(B, L, h, D).to(_DT[dt]) if h else None for h in (Hq, Hk))
        if case["fused"] and Hk:   # views of one buffer, as the projections leave them
            buf = torch.cat([q.flatten(2), k.flatten(2)], -1)
            q, k = buf[..., : Hq * D].unflatten(2, (Hq, D)), buf[..., Hq * D:].unflatten(2, (Hk, D))
        s["q"], s["k"] = q, k
        s["pos"] = torch.arange(L, dtype=torch.int32, device="cuda").repeat(B, 1)
        if case["far"]:            # each request somewhere in its context
            s["pos"] += torch.randint(0, case["far"], (B, 1), device="cuda", generator=gen, dtype=torch.int32)
        s["freq"], s["scale"] = _frequencies(case)
        if case["mode"] == "train":
            s["dq"], s["dk"] = (None if t is None else rand(*t.shape).to(t.dtype) for t in (q, k))
            for n in ("q", "k"):
                if s[n] is not None:
                    s[n] = s[n].detach().requires_grad_()
    return s


# ---- plain forms --------------------------------------------------------------------------

def _doubling(a, b):
    """h[:, t] = a[:, t] h[:, t - 1] + b[:, t], by steps of doubled width."""
    k, L = 1, a.shape[1]
    while k < L:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        if 2 * k < L:
            a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _plain_scan(s, train):
    case = s["case"]
    x, g = s["x"].float(), s["g"].float()
    B, L, C = x.shape
    a = torch.exp(s["g"].double()).float()       # next to 1: a rounding that leans one way adds up over thousands of steps
    weight = torch.sqrt(-torch.expm1(2 * g)) if case["normalize"] else torch.ones_like(a)
    b = weight * x
    h0 = s["h0"]
    if s["cu"] is None:
        first, last, row = torch.zeros(B, dtype=torch.int64, device="cuda"), torch.full((B,), L - 1, device="cuda"), torch.arange(B, device="cuda")
        start = h0 if h0 is not None else x.new_zeros(B, C)
        live = torch.ones(B, dtype=torch.bool, device="cuda")
    else:
        first, last, live = s["first"], s["last"], s["live"]
        row = torch.zeros_like(first)
        start = h0[live] if h0 is not None else x.new_zeros(first.numel(), C)
    b[row, first] += a[row, first] * start
    keep = a.clone()
    keep[row, first] = 0
    inside = torch.ones(L, device="cuda") if s["cu"] is None else (torch.arange(L, device="cuda") < s["end"]).float()
    keep, b = keep * inside[:, None], b * inside[:, None]
    h = _doubling(keep, b)
    final = h0.clone() if h0 is not None else x.new_zeros(live.numel(), C)
    final[live] = h[row, last]
    ans = {"out": h.to(s["x"].dtype), "final_state": final}
    if not train:
        return ans
    d = s["dout"].float() * inside[:, None]
    if s["dht"] is not None:
        d[row, last] += s["dht"][live]
    back = torch.cat([keep[:, 1:], keep.new_zeros(B, 1, C)], 1)            # D[t] = d[t] + a[t + 1] D[t + 1]
    D = _doubling(back.flip(1), d.flip(1)).flip(1)
    before = torch.cat([h.new_zeros(B, 1, C), h[:, :-1]], 1)
    before[row, first] = start
    dg = a * before * D
    if case["normalize"]:
        dg = dg - a * a / weight * x * D
    ans["dx"], ans["dg"] = (weight * D).to(s["x"].dtype), (dg * inside[:, None]).to(s["g"].dtype)
    if h0 is not None:
        dh0 = s["dht"].clone()
        dh0[live] = a[row, first] * D[row, first]
        ans["dh0"] = dh0
    return ans


def _plain_step(s):
    case, state = s["case"], s["state"]
    live = s["slots"] >= 0
    slot = s["slots"][live].long()
    x, g = s["x"][live].float(), s["g"][live].float()
    out, h, rows = torch.zeros(s["x"].shape, device="cuda"), state[slot], []
    for t in range(case["T"]):   # one step after the other
        w = torch.sqrt(-torch.expm1(2 * g[:, t])) if case["normalize"] else 1.0
        h = torch.exp(g[:, t]) * h + w * x[:, t]
        rows.append(h)
    out[live] = torch.stack(rows, 1)
    state[slot] = h
    return {"out": out.to(s["x"].dtype), "state": state}


def _plain_gnorm(s, train):
    case = s["case"]
    G, act = case["groups"], case["activation"] == "silu"
    x, w, b = s["x"].float().unflatten(1, (G, -1)), s["w"].float(), s["b"].float()
    d = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(d.square().mean(-1, keepdim=True) + _EPS)
    n = d * r
    y = n.flatten(1) * w + b
    through = s["z"].float() if case["gated"] else y                       # what the activation is of
    sig = 1 / (1 + torch.exp(-through))
    value = through * sig if act else through
    out = y * value if case["gated"] else value
    ans = {"out": out.to(s["x"].dtype)}
    if not train:
        return ans
    dout = s["dout"].float()
    slope = sig * (1 + through * (1 - sig)) if act else torch.ones_like(sig)
    dy = dout * (value if case["gated"] else slope)
    if case["gated"]:
        ans["dz"] = (dout * y * slope).to(s["z"].dtype)
    e = (dy * w).unflatten(1, (G, -1))
    dx = r * (e - e.mean(-1, keepdim=True) - n * (e * n).mean(-1, keepdim=True))
    ans["dx"] = dx.flatten(1).to(s["x"].dtype)
    ans["dw"], ans["db"] = (dy * n.flatten(1)).sum(0).to(s["w"].dtype), dy.sum(0).to(s["b"].dtype)
    return ans


def _turn(x, cos, sin, turned, interleaved):
    """x [B, L, H, D]; cos and sin [B, L, 1, turned / 2]."""
    y = x.float()
    if interleaved:
        a, b = y[..., 0:turned:2], y[..., 1:turned:2]
        both = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., : turned // 2], y[..., turned // 2: turned]
        both = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([both, y[..., turned:]], -1).to(x.dtype)


def _plain_rotary(s, train):
    case = s["case"]
    angle = s["pos"].double()[..., None, None] * s["freq"]
    cos, sin = ((f(angle) * s["scale"]).float() for f in (torch.cos, torch.sin))
    names = [n for n in ("q", "k") if s[n] is not None]
    ans = {n: _turn(s[n], cos, sin, case["turned"], case["interleaved"]) for n in names}
    if train:
        ans.update({"d" + n: _turn(s["d" + n], cos, -sin, case["turned"], case["interleaved"]) for n in names})
    return ans


# ---- one pass -----------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op, train = case["op"], case.get("mode") == "train"
    if own:
        return _run_own(s, case, op, train)
    with torch.no_grad():
        if op == "scan":
            return _plain_scan(s, train)
        if op == "step":
            return _plain_step(s)
        return _plain_gnorm(s, train) if op == "gnorm" else _plain_rotary(s, train)


def _run_own(s, case, op, train):
    import causal_depthwise_conv1d_amd as ccv
    if op == "scan":
        call = ccv.gated_linear_recurrence_fn if train else ccv.gated_linear_recurrence_fwd
        o, ht = call(s["x"], s["g"], cu_seqlens=s["cu"], initial_state=s["h0"], return_final_state=True, normalize=case["normalize"])
        ans = {"out": o.detach(), "final_state": ht.detach()}
        if train:
            names = [n for n in ("x", "g", "h0") if s[n] is not None]
            ends, seeds = ([o, ht], [s["dout"], s["dht"]]) if case["states"] else ([o], [s["dout"]])
            ans.update({"d" + n: d for n, d in zip(names, torch.autograd.grad(ends, [s[n] for n in names], seeds))})
        return ans
    if op == "step":
        out = ccv.gated_linear_recurrence_update(s["x"], s["g"], s["state"], state_indices=s["slots"], normalize=case["normalize"])
        return {"out": out, "state": s["state"]}
    if op == "gnorm":
        act = None if case["activation"] == "none" else case["activation"]
        if not train:
            return {"out": ccv.group_norm_fwd(s["x"], case["groups"], s["w"], s["b"], gate=s["z"], activation=act, eps=_EPS)}
        out = ccv.group_norm_fn(s["x"], case["groups"], s["w"], s["b"], gate=s["z"], activation=act, eps=_EPS)
        names = [n for n in ("x", "z", "w", "b") if s[n] is not None]
        grads = torch.autograd.grad(out, [s[n] for n in names], s["dout"])
        return {"out": out.detach(), **{"d" + n: d for n, d in zip(names, grads)}}
    call = ccv.rotary_fn if train else ccv.rotary_fwd
    names = [n for n in ("q", "k") if s[n] is not None]
    out = call(s["q"], s["k"], s["pos"], s["freq"], interleaved=case["interleaved"], scale=s["scale"])[: len(names)]
    ans = {n: t.detach() for n, t in zip(names, out)}
    if train:
        grads = torch.autograd.grad(out, [s[n] for n in names], [s["d" + n] for n in names])
        ans.update({"d" + n: d for n, d in zip(names, grads)})
    return ans


# ---- from the definitions, in 64 bits -----------------------------------------------------

def _by_pieces(a, b):
    """h[t] = a[t] h[t - 1] + b[t] along dimension 0, h before the first step 0: step by step inside pieces side by side,
    then from piece to piece."""
    L = a.shape[0]
    T = max(1, math.isqrt(L))
    K = -(-L // T)
    a, b = (torch.cat([t, t.new_zeros(K * T - L, *t.shape[1:])]).unflatten(0, (K, T)) for t in (a, b))
    h, p = torch.empty_like(b), torch.empty_like(a)
    now, far = torch.zeros_like(b[:, 0]), torch.ones_like(a[:, 0])
    for t in range(T):
        now = torch.addcmul(b[:, t], a[:, t], now)
        far = far * a[:, t]
        h[:, t], p[:, t] = now, far
    carry = torch.zeros_like(b[0, 0])
    for k in range(K):
        h[k].addcmul_(p[k], carry)
        carry = h[k, -1]
    return h.flatten(0, 1)[:L]


def _exact_scan(s):
    case = s["case"]
    B, L, C = s["x"].shape
    train = case["mode"] == "train"
    cu = [0, L] if s["cu"] is None else s["cu"].tolist()
    spans = [(r, cu[i], cu[i + 1], r + i) for r in range(B) for i in range(len(cu) - 1)]
    ans = {"out": torch.zeros(B, L, C, dtype=torch.float64, device="cuda"), "final_state": torch.zeros(len(spans), C, dtype=torch.float64, device="cuda")}
    if train:
        ans.update({n: torch.zeros_like(ans["out"]) for n in ("dx", "dg")})
        if s["h0"] is not None:
            ans["dh0"] = torch.zeros_like(ans["final_state"])
    zero = torch.zeros(C, dtype=torch.float64, device="cuda")
    for r, t0, t1, i in spans:   # each sequence by itself
        h0 = s["h0"][i].double() if s["h0"] is not None else zero
        if t0 == t1:
            ans["final_state"][i] = h0
            if "dh0" in ans:
                ans["dh0"][i] = s["dht"][i].double()
            continue
        x, g = s["x"][r, t0:t1].double(), s["g"][r, t0:t1].double()
        a = g.exp()
        w = (1 - (2 * g).exp()).sqrt() if case["normalize"] else torch.ones_like(a)
        b = w * x
        b[0] += a[0] * h0
        h = _by_pieces(a, b)
        ans["out"][r, t0:t1], ans["final_state"][i] = h, h[-1]
        if not train:
            continue
        d = s["dout"][r, t0:t1].double().clone()
        if s["dht"] is not None:
            d[-1] += s["dht"][i].double()
        D = _by_pieces(torch.cat([a[1:], a[:1]]).flip(0), d.flip(0)).flip(0)
        ans["dx"][r, t0:t1] = w * D
        dg = a * torch.cat([h0[None], h[:-1]]) * D
        ans["dg"][r, t0:t1] = dg - x * D * (2 * g).exp() / w if case["normalize"] else dg
        if "dh0" in ans:
            ans["dh0"][i] = a[0] * D[0]
    return ans


def exact(case, seed):
    s = prepare(case, seed)
    op, train = case["op"], case.get("mode") == "train"
    with torch.no_grad():
        if op == "scan":
            return _exact_scan(s)
        if op == "step":
            state, out = s["state"].double(), torch.zeros(s["x"].shape, device="cuda", dtype=torch.float64)
            for r, slot in enumerate(s["slots"].tolist()):
                for t in range(case["T"] if slot >= 0 else 0):
                    g = s["g"][r, t].double()
                    w = (1 - (2 * g).exp()).sqrt() if case["normalize"] else 1.0
                    state[slot] = out[r, t] = g.exp() * state[slot] + w * s["x"][r, t].double()
            return {"out": out, "state": state}
        if op == "gnorm":
            with torch.enable_grad():                                      # differentiated in 64 bits
                x, w, b = (s[n].detach().double().requires_grad_(train) for n in ("x", "w", "b"))
                z = s["z"].detach().double().requires_grad_(train) if case["gated"] else None
                per = x.unflatten(1, (case["groups"], -1))
                var = per.var(-1, keepdim=True, unbiased=False)
                y = ((per - per.mean(-1, keepdim=True)) / (var + _EPS).sqrt()).flatten(1) * w + b
                f = (lambda t: t / (1 + (-t).exp())) if case["activation"] == "silu" else (lambda t: t)
                out = y * f(z) if case["gated"] else f(y)
                ans = {"out": out.detach()}
                if train:
                    leaves = {n: t for n, t in (("dz", z), ("dx", x), ("dw", w), ("db", b)) if t is not None}
                    ans.update(zip(leaves, torch.autograd.grad(out, list(leaves.values()), s["dout"].double())))
            return ans
        d, half = case["turned"], case["turned"] // 2
        turn = torch.polar(torch.full_like(s["freq"], s["scale"]).expand(*s["pos"].shape, half), s["pos"].double()[..., None] * s["freq"])[:, :, None]
        ans = {}
        for n in ("q", "k", "dq", "dk"):
            if s.get(n) is None:
                continue
            y = s[n].double()
            pairs = y[..., :d].unflatten(-1, (half, 2)) if case["interleaved"] else y[..., :d].unflatten(-1, (2, half)).transpose(-1, -2)
            z = torch.view_as_complex(pairs.contiguous()) * (turn.conj() if n[0] == "d" else turn)
            z = torch.view_as_real(z)
            z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
            ans[n] = torch.cat([z, y[..., d:]], -1)
        return ans


# ---- what a pass cannot do without --------------------------------------------------------

def work(case):
    op, train = case["op"], case.get("mode") == "train"
    es = _ES[case["dtype"]]
    if op == "scan":
        n, N = case["B"] * case["L"] * case["C"], case["seqs"] or case["B"]
        gs, state = _ES[case["gate"]], N * case["C"] * 4
        nbytes = n * (2 * es + gs) + state * (2 if case["states"] else 1)
        if train:                                           # dout in; dx, dg out; the states' gradients
            nbytes += n * (2 * es + gs) + (2 * state if case["states"] else 0)
        return {"bytes": nbytes, "flops": n * (12 if train else 4) + (n * (10 if train else 4) if case["normalize"] else 0)}
    if op == "step":
        live = case["B"] - case["idle"]
        per = case["C"] * (8 + case["T"] * (2 * es + _ES[case["gate"]]))
        return {"bytes": live * per, "flops": live * case["T"] * case["C"] * (8 if case["normalize"] else 4)}
    if op == "gnorm":
        n = case["rows"] * case["C"]
        arrays = (3 if case["gated"] else 2) + ((3 if case["gated"] else 2) if train else 0)   # dout; dx and dz
        return {"bytes": n * es * arrays, "flops": n * (40 if train else 14)}
    n = case["B"] * case["L"] * (case["Hq"] + case["Hk"]) * case["D"]
    return {"bytes": n * es * (4 if train else 2) + case["B"] * case["L"] * 4, "flops": n * (6 if train else 3)}
