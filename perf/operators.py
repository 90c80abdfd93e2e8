"""The operators of a gated linear-attention layer around the causal conv1d, as they are measured.

A layer of this kind normalises its input (layer norm), convolves the projections (the causal
conv1d of this package), runs the gated delta rule over queries, keys and values, and normalises
each head's output (layer norm again).  Serving packs requests of different lengths into one row,
so the row's sequence tables are built on the GPU from the lengths; decoding then advances each
request's state by a step.  Four kinds of case:

  "delta"   the gated delta rule over whole sequences ("fwd": outputs and final states; "train":
            these and every gradient)
  "step"    the same rule for a few new steps against states in a cache, advanced in place
  "norm"    layer norm over the last dimension ("fwd", or "train": outputs and gradients)
  "tables"  offsets, sequence ids and positions of a packed row, from the sequences' lengths

Where `own` is false everything is computed by elementary torch operations in 32 bits; where it is
true by this package's kernels.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}
_CHUNK = 64
_EPS = 1e-5


# ---- the cases ----------------------------------------------------------------------------

def _delta(name, mode, B, L, Hk, Hv, Dk, Dv, dtype, beta, seqs=0, states=True, fused=True):
    return {"name": name, "op": "delta", "mode": mode, "B": B, "L": L, "Hk": Hk, "Hv": Hv, "Dk": Dk, "Dv": Dv,
            "dtype": dtype, "beta": beta, "seqs": seqs, "states": states, "fused": fused}


def _step(name, B, T, slots, Hk, Hv, Dk, Dv, dtype, beta, idle):
    return {"name": name, "op": "step", "B": B, "T": T, "slots": slots, "Hk": Hk, "Hv": Hv, "Dk": Dk, "Dv": Dv,
            "dtype": dtype, "beta": beta, "idle": idle}


def _norm(name, mode, rows, heads, width, dtype, weight, pad=0):
    return {"name": name, "op": "norm", "mode": mode, "rows": rows, "heads": heads, "width": width, "dtype": dtype,
            "weight": weight, "pad": pad}


def _tables(name, count, total, fill):
    return {"name": name, "op": "tables", "count": count, "total": total, "fill": fill}


def listed():
    return [
        # a short prompt of one request in fp32, one head of the 64 channels of the small conv workload
        _delta("delta fwd f32 1x2048 h1 d64", "fwd", 1, 2048, 1, 1, 64, 64, "f32", "f32", states=False),
        # the bf16 conv workload's batch (4 x 4096, 2048 channels) as 16 heads of 128, prefill with carried states
        _delta("delta fwd bf16 4x4096 h16", "fwd", 4, 4096, 16, 16, 128, 128, "bf16", "bf16"),
        # serving prefill: the packed conv workload (65536 steps, 64 requests, 2560 channels), two value heads a key head
        _delta("delta fwd f16 packed 65536", "fwd", 1, 65536, 10, 20, 128, 128, "f16", "f32", seqs=64),
        # a training step of the same layer on 2 x 4096
        _delta("delta train bf16 2x4096 h16", "train", 2, 4096, 16, 16, 128, 128, "bf16", "bf16", states=False),
        # training in fp32 on a packed row of odd lengths, odd head widths and shared key heads
        _delta("delta train f32 packed 3011", "train", 1, 3011, 2, 6, 72, 96, "f32", "f32", seqs=7),
        # decoding: the update workload's 256 requests and 4096 channels, one step each
        _step("step bf16 B256 h32", 256, 1, 256, 32, 32, 128, 128, "bf16", "bf16", 0),
        # a few requests of a larger cache, some rows idle: what a single step costs at the least
        _step("step f16 B5 h20 of 64 slots", 5, 1, 64, 10, 20, 128, 128, "f16", "f32", 1),
        # the pre-norm of a decode step
        _norm("norm fwd bf16 256x4096", "fwd", 256, 1, 4096, "bf16", "bf16"),
        # the pre-norm of a training batch of 4 x 8192 tokens
        _norm("norm train bf16 32768x4096", "train", 32768, 1, 4096, "bf16", "f32"),
        # each head's output normalised: 65536 tokens of 20 heads, read out of a wider buffer
        _norm("norm train f16 65536x20x128", "train", 65536, 20, 128, "f16", "f32", pad=512),
        # a serving batch of 64 requests
        _tables("tables 64 of 65536", 64, 65536, 0.97),
        # a training row of a million steps packed with short samples
        _tables("tables 4001 of 1048576", 4001, 1048576, 1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["delta", "delta", "delta", "step", "norm", "tables"])
    if kind == "delta":
        mode = rng.choice(["fwd", "train"])
        Hk = rng.choice([1, 2, 3, 4, 8, 16])
        Hv = Hk * rng.choice([1, 1, 2, 3])
        Dk, Dv = rng.choice([(64, 64), (128, 128), (128, 128), (rng.randint(1, 128), rng.randint(1, 160)), (96, 64), (64, 128)])
        steps = min(32768 if mode == "fwd" else 8192, max(64, (1 << 17) // Hv))
        T = _log(rng, 1, steps)
        seqs = rng.choice([0, 0, rng.randint(1, 40)])
        B = 1 if seqs else max(1, min(8, T // 100))
        return _delta("", mode, B, max(1, T // B), Hk, Hv, Dk, Dv, rng.choice(["f32", "f16", "bf16"]),
                      rng.choice(["f32", "bf16"]), seqs, rng.random() < 0.6, rng.random() < 0.7) | {"draw": rng.randrange(1 << 20)}
    if kind == "step":
        B, Hk = _log(rng, 1, 256), rng.choice([1, 2, 4, 8, 16])
        Dk, Dv = rng.choice([(64, 64), (128, 128), (rng.randint(1, 128), rng.randint(1, 160))])
        return _step("", B, rng.choice([1, 1, 1, 2, 4]), B + rng.randint(0, 64), Hk, Hk * rng.choice([1, 2]), Dk, Dv,
                     rng.choice(["f32", "f16", "bf16"]), rng.choice(["f32", "bf16"]), rng.randint(0, min(B - 1, 3))) | {"draw": rng.randrange(1 << 20)}
    if kind == "norm":
        width = rng.choice([64, 128, 2048, 2560, 4096, _log(rng, 24, 20000)])
        rows = max(1, min(_log(rng, 1, 65536), (1 << 27) // width))
        heads = rng.choice([1, 4]) if width <= 256 else 1
        return _norm("", rng.choice(["fwd", "train"]), rows, heads, width, rng.choice(["f32", "f16", "bf16"]),
                     rng.choice(["f32", "bf16"]), rng.choice([0, 0, 8, 3])) | {"draw": rng.randrange(1 << 20)}
    count = _log(rng, 1, 4000)
    return _tables("", count, _log(rng, 1, 1 << 20), rng.choice([1.0, 0.9, 0.5])) | {"draw": rng.randrange(1 << 20)}


def _lengths(count, total, gen):
    """`count` lengths of sum `total`, some of them zero, as a list; the same for every seed's generator state."""
    if count <= 0:
        return []
    w = torch.empty(count, dtype=torch.float64).exponential_(generator=gen) + 0.1
    if count > 4:
        w[torch.randint(0, count, (max(1, count // 16),), generator=gen)] = 0.0
    edges = torch.floor(torch.cumsum(w / w.sum(), 0) * total + 1e-9).to(torch.int64)
    edges[-1] = total
    return torch.diff(edges, prepend=torch.zeros(1, dtype=torch.int64)).tolist()


# ---- inputs -------------------------------------------------------------------------------

def _unit(x):
    return x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()


def _silu(x):
    return x / (1 + torch.exp(-x))


def _softplus(x):
    return torch.log1p(torch.exp(x))


def _delta_inputs(case, seed, lead, gen):
    """Queries, keys and values as they leave the conv (SiLU), queries and keys of unit length; log decays
    -A softplus(a + dt) and write strengths sigmoid(b).  `lead` is (rows, steps)."""
    Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
    dt = _DT[case["dtype"]]
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    q, k = (_unit(_silu(rand(*lead, Hk, Dk))).to(dt) for _ in range(2))
    v = _silu(rand(*lead, Hv, Dv)).to(dt)
    if case.get("fused"):   # views of one buffer, as the projections leave the conv
        buf = torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], -1)
        a, b = Hk * Dk, 2 * Hk * Dk
        q, k, v = (t.unflatten(2, (h, -1)) for t, h in ((buf[..., :a], Hk), (buf[..., a:b], Hk), (buf[..., b:], Hv)))
    A = torch.rand(Hv, device="cuda", generator=gen) * 15 + 1
    step = torch.exp(torch.rand(Hv, device="cuda", generator=gen) * math.log(100.0) + math.log(1e-3))
    g = -A * _softplus(rand(*lead, Hv) * 0.5 + step + torch.log(-torch.expm1(-step)))
    beta = (1 / (1 + torch.exp(-rand(*lead, Hv)))).to(_DT[case["beta"]])
    return q, k, v, g, beta


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "delta":
        B, L, N = case["B"], case["L"], case["seqs"]
        s["q"], s["k"], s["v"], s["g"], s["beta"] = _delta_inputs(case, seed, (B, L), gen)
        rows = N or B
        s["lengths"] = _lengths(N, L, host) if N else None
        s["cu"] = torch.tensor([0] + torch.tensor(s["lengths"]).cumsum(0).tolist(), dtype=torch.int32, device="cuda") if N else None
        shape = (rows, case["Hv"], case["Dk"], case["Dv"])
        s["h0"] = torch.randn(shape, device="cuda", generator=gen) * 0.1 if case["states"] else None
        if case["mode"] == "train":
            s["dout"] = torch.randn(s["v"].shape, device="cuda", generator=gen).to(s["v"].dtype)
            s["dht"] = torch.randn(shape, device="cuda", generator=gen) * 0.1 if case["states"] else None
            for n in ("q", "k", "v", "g", "beta", "h0"):   # parameters' side of the step: gradients are wanted
                if s[n] is not None:
                    s[n] = s[n].detach().requires_grad_()
        if N:
            pad = max(max(s["lengths"]), 1)
            start = s["cu"][:-1].long()[:, None] + torch.arange(pad, device="cuda")[None]
            real = torch.arange(pad, device="cuda")[None] < torch.tensor(s["lengths"], device="cuda")[:, None]
            s["to"], s["real"] = torch.where(real, start, 0), real
    elif op == "step":
        s["q"], s["k"], s["v"], s["g"], s["beta"] = _delta_inputs(case, seed, (case["B"], case["T"]), gen)
        s["state"] = torch.randn(case["slots"], case["Hv"], case["Dk"], case["Dv"], device="cuda", generator=gen) * 0.3
        slots = torch.randperm(case["slots"], device="cuda", generator=gen)[: case["B"]].to(torch.int32)
        if case["idle"]:
            slots[torch.randperm(case["B"], device="cuda", generator=gen)[: case["idle"]]] = -1
        s["slots"] = slots
    elif op == "norm":
        shape = (case["rows"], case["heads"], case["width"] + case["pad"])
        x = torch.randn(shape, device="cuda", generator=gen) * 1.5 + 0.3
        s["x"] = x.to(_DT[case["dtype"]])[..., : case["width"]]
        wd = _DT[case["weight"]]
        s["w"] = (1 + 0.1 * torch.randn(case["width"], device="cuda", generator=gen)).to(wd)
        s["b"] = (0.1 * torch.randn(case["width"], device="cuda", generator=gen)).to(wd)
        if case["mode"] == "train":
            s["dout"] = torch.randn(s["x"].shape, device="cuda", generator=gen).to(s["x"].dtype)
            for n in ("x", "w", "b"):
                s[n] = s[n].detach().requires_grad_()
    else:
        n = int(case["total"] * case["fill"])
        s["lengths"] = torch.tensor(_lengths(case["count"], n, host), dtype=torch.int32, device="cuda")
    return s


# ---- plain forms --------------------------------------------------------------------------

def _gather(s, t):
    """[1, T, ...] packed -> [sequences, longest, ...], zeros past each sequence's end."""
    return t[0][s["to"]] * s["real"].view(*s["real"].shape, *[1] * (t.dim() - 2)).to(t.dtype)


def _heads(x, H):
    """[N, L, h, D] -> [N, H, chunks, 64, D], each of the h heads repeated for its group."""
    N, L, h, D = x.shape
    x = torch.cat([x, x.new_zeros(N, -L % _CHUNK, h, D)], 1) if L % _CHUNK else x
    x = x.transpose(1, 2).reshape(N, h, -1, _CHUNK, D)
    return x if h == H else x[:, torch.arange(H, device=x.device) // (H // h)]


def _plain_chunks(q, k, v, g, beta, scale, state):
    """The gated delta rule by chunks of 64 steps, all in 32 bits: [N, L, H, D] inputs, [N, H, Dk, Dv] state."""
    N, L, H = g.shape
    q, k, v = _heads(q, H), _heads(k, H), _heads(v, H)
    G = _heads(g[..., None], H)[..., 0].cumsum(-1)
    b = _heads(beta[..., None], H)
    low = torch.ones(_CHUNK, _CHUNK, device=q.device, dtype=torch.bool).tril()
    decay = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf))
    kt = k.transpose(-1, -2).contiguous()
    A = b * (decay * (k @ kt)).tril(-1)
    P = decay * (q @ kt)
    W = torch.eye(_CHUNK, device=q.device).expand_as(A)   # (1 + A)^-1, blocks of 1, 2, 4 ... joined in pairs
    i = torch.arange(_CHUNK, device=q.device)
    size = 1
    while size < _CHUNK:
        block, half = i // (2 * size), (i // size) % 2
        off = (block[:, None] == block[None]) & (half[:, None] == 1) & (half[None] == 0)
        W = W - W @ ((A * off) @ W)
        size *= 2
    gamma, rest, last = torch.exp(G)[..., None], torch.exp(G[..., -1:] - G)[..., None], torch.exp(G[..., -1])[..., None, None]
    out, bv, bk, gq, end = [], b * v, b * gamma * k, gamma * q, (rest * k).transpose(-1, -2).contiguous()
    for c in range(G.shape[2]):   # the state passes from chunk to chunk
        new = W[:, :, c] @ (bv[:, :, c] - bk[:, :, c] @ state)
        out.append(gq[:, :, c] @ state + P[:, :, c] @ new)
        state = last[:, :, c] * state + end[:, :, c] @ new
    o = scale * torch.stack(out, 2).flatten(2, 3).transpose(1, 2)[:, :L]
    return o, state


def _plain_delta(s, q, k, v, g, beta, h0):
    case = s["case"]
    args = [t.float() for t in (q, k, v, g, beta)]
    if case["seqs"]:
        args = [_gather(s, t) for t in args]
    if h0 is None:
        h0 = args[0].new_zeros(args[0].shape[0], case["Hv"], case["Dk"], case["Dv"])
    o, ht = _plain_chunks(*args, case["Dk"] ** -0.5, h0)
    if case["seqs"]:
        o = o[s["real"]][None]
    return o, ht


def _plain_step(s):
    case, state = s["case"], s["state"]
    live = s["slots"] >= 0
    slot = s["slots"][live].long()
    q, k, v, g, beta = (s[n][live].float() for n in ("q", "k", "v", "g", "beta"))
    head = torch.arange(case["Hv"], device=q.device) // (case["Hv"] // case["Hk"])
    S, out = state[slot], torch.zeros(s["v"].shape, device=q.device)
    rows = []
    for t in range(case["T"]):   # one step after the other
        kt, qt = k[:, t][:, head][..., None], q[:, t][:, head][..., None]
        S = torch.exp(g[:, t])[..., None, None] * S
        new = beta[:, t][..., None] * (v[:, t] - (S * kt).sum(-2))
        S = S + kt * new[..., None, :]
        rows.append((S * qt).sum(-2))
    out[live] = torch.stack(rows, 1) * case["Dk"] ** -0.5
    state[slot] = S
    return {"out": out.to(s["v"].dtype), "state": state}


def _plain_norm(x, w, b):
    x = x.float()
    d = x - x.mean(-1, keepdim=True)
    return d * torch.rsqrt(d.square().mean(-1, keepdim=True) + _EPS) * w.float() + b.float()


def _plain_norm_grads(x, w, dout):
    x, w, dy = x.float(), w.float(), dout.float()
    d = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(d.square().mean(-1, keepdim=True) + _EPS)
    n, a = d * r, dy * w
    dx = r * (a - a.mean(-1, keepdim=True) - n * (a * n).mean(-1, keepdim=True))
    return dx, (dy * n).sum((0, 1)), dy.sum((0, 1))


def _plain_tables(lengths, total):
    ends = lengths.cumsum(0, dtype=torch.int64)
    cu = torch.cat([ends.new_zeros(1), ends])
    t = torch.arange(total, device=lengths.device)
    seq = torch.zeros(total + 1, dtype=torch.int64, device=lengths.device).index_add(0, ends, torch.ones_like(ends)).cumsum(0)[:total]
    inside = t < cu[-1]
    seq = torch.where(inside, seq, -1)
    at = torch.where(inside, t - cu[seq], 0)
    return {"cu_seqlens": cu.int(), "seq_idx": seq.int()[None], "positions": at.int()[None]}


# ---- one pass -----------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _run_own(s, case, op)
    if op == "step":
        with torch.no_grad():
            return _plain_step(s)
    if op == "tables":
        return _plain_tables(s["lengths"], case["total"])
    if op == "norm":
        with torch.no_grad():
            out = {"out": _plain_norm(s["x"], s["w"], s["b"]).to(s["x"].dtype)}
            if case["mode"] == "train":
                for n, d in zip(("x", "w", "b"), _plain_norm_grads(s["x"], s["w"], s["dout"])):
                    out["d" + n] = d.to(s[n].dtype)
        return out
    names = [n for n in ("q", "k", "v", "g", "beta", "h0") if s[n] is not None]
    if case["mode"] == "fwd":
        with torch.no_grad():
            o, ht = _plain_delta(s, *(s[n] for n in ("q", "k", "v", "g", "beta", "h0")))
        return {"out": o.to(s["v"].dtype), "final_state": ht}
    o, ht = _plain_delta(s, *(s[n] for n in ("q", "k", "v", "g", "beta", "h0")))
    ends, seeds = ([o, ht], [s["dout"].float(), s["dht"]]) if case["states"] else ([o], [s["dout"].float()])
    grads = torch.autograd.grad(ends, [s[n] for n in names], seeds)
    return {"out": o.detach().to(s["v"].dtype), "final_state": ht.detach(), **{"d" + n: d for n, d in zip(names, grads)}}


def _run_own(s, case, op):
    import causal_depthwise_conv1d_amd as ccv
    if op == "step":
        out = ccv.gated_delta_rule_update(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], state_indices=s["slots"])
        return {"out": out, "state": s["state"]}
    if op == "tables":
        cu, seq, at = ccv.sequence_tables(s["lengths"], case["total"])
        return {"cu_seqlens": cu, "seq_idx": seq, "positions": at}
    if op == "norm":
        if case["mode"] == "fwd":
            return {"out": ccv.layer_norm_fwd(s["x"], s["w"], s["b"], eps=_EPS)}
        out = ccv.layer_norm_fn(s["x"], s["w"], s["b"], eps=_EPS)
        grads = torch.autograd.grad(out, [s["x"], s["w"], s["b"]], s["dout"])
        return {"out": out.detach(), **{"d" + n: d for n, d in zip(("x", "w", "b"), grads)}}
    if case["mode"] == "fwd":
        o, ht = ccv.gated_delta_rule_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], cu_seqlens=s["cu"],
                                         initial_state=s["h0"], return_final_state=True)
        return {"out": o, "final_state": ht}
    o, ht = ccv.gated_delta_rule_fn(s["q"], s["k"], s["v"], s["g"], s["beta"], cu_seqlens=s["cu"],
                                    initial_state=s["h0"], return_final_state=True)
    names = [n for n in ("q", "k", "v", "g", "beta", "h0") if s[n] is not None]
    ends, seeds = ([o, ht], [s["dout"], s["dht"]]) if case["states"] else ([o], [s["dout"]])
    grads = torch.autograd.grad(ends, [s[n] for n in names], seeds)
    return {"out": o.detach(), "final_state": ht.detach(), **{"d" + n: d for n, d in zip(names, grads)}}


# ---- from the definitions, in 64 bits -----------------------------------------------------

def _exact_delta(s):
    """Step by step: S <- e^g S, S <- S + k (beta (v - S^T k))^T, o = scale S^T q; gradients by the same steps backwards,
    states kept every 64 steps and made again from there."""
    case = s["case"]
    names = ("q", "k", "v", "g", "beta")
    pick = (lambda t: _gather(s, t)) if case["seqs"] else (lambda t: t)
    q, k, v, g, beta = (pick(s[n].detach()).double() for n in names)
    N, L, H = g.shape
    group = H // case["Hk"]
    qh, kh = (t.repeat_interleave(group, 2) for t in (q, k))
    scale = case["Dk"] ** -0.5
    S = s["h0"].detach().double() if s["h0"] is not None else g.new_zeros(N, H, case["Dk"], case["Dv"])
    alpha, out, kept = torch.exp(g), torch.empty_like(v), []

    def advance(S, t):
        D = alpha[:, t, :, None, None] * S
        e = v[:, t] - (kh[:, t, :, None] @ D)[:, :, 0]
        return D, e, D + kh[:, t, ..., None] * (beta[:, t, :, None] * e)[:, :, None]

    for t in range(L):
        if t % 64 == 0 and case["mode"] == "train":
            kept.append(S)
        S = advance(S, t)[2]
        out[:, t] = scale * (qh[:, t, :, None] @ S)[:, :, 0]
    back = (lambda t: t[s["real"]][None]) if case["seqs"] else (lambda t: t)
    ans = {"out": back(out), "final_state": S}
    if case["mode"] == "fwd":
        return ans
    do = pick(s["dout"]).double()
    dS = s["dht"].double() if s["dht"] is not None else torch.zeros_like(S)
    dq, dk, dv, dg, db = (torch.zeros_like(t) for t in (qh, kh, v, g, beta))
    for c in range(len(kept) - 1, -1, -1):
        ts = range(64 * c, min(L, 64 * c + 64))
        S, steps = kept[c], []
        for t in ts:
            D, e, S = advance(S, t)
            steps.append((D, e, S))
        for t in reversed(ts):
            D, e, S = steps.pop()
            kc, b = kh[:, t, ..., None], beta[:, t, :, None]
            dq[:, t] = scale * (S @ do[:, t, ..., None])[..., 0]
            dS = dS + scale * qh[:, t, ..., None] * do[:, t, :, None]
            du = (kh[:, t, :, None] @ dS)[:, :, 0]
            db[:, t] = (du * e).sum(-1)
            de = b * du
            dk[:, t] = (dS @ (b * e)[..., None] - D @ de[..., None])[..., 0]
            dv[:, t] = de
            dS = dS - kc * de[:, :, None]
            dg[:, t] = (dS * D).sum((-1, -2))
            dS = alpha[:, t, :, None, None] * dS
    dq, dk = (t.unflatten(2, (case["Hk"], group)).sum(3) for t in (dq, dk))
    ans.update(zip(("dq", "dk", "dv", "dg", "dbeta"), map(back, (dq, dk, dv, dg, db))))
    if s["h0"] is not None:
        ans["dh0"] = dS
    return ans


def exact(case, seed):
    if case["op"] == "tables":
        return None   # whole numbers
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"] == "delta":
            return _exact_delta(s)
        if case["op"] == "norm":
            x, w, b = (s[n].double() for n in ("x", "w", "b"))
            r = 1 / torch.sqrt(x.var(-1, keepdim=True, unbiased=False) + _EPS)
            n = (x - x.mean(-1, keepdim=True)) * r
            ans = {"out": n * w + b}
            if case["mode"] == "train":
                dy = s["dout"].double()
                a = dy * w
                along = (a * n).sum(-1, keepdim=True) / case["width"]
                ans["dx"] = (a - a.mean(-1, keepdim=True) - n * along) * r
                ans["dw"], ans["db"] = (dy * n).sum((0, 1)), dy.sum((0, 1))
            return ans
        state, out = s["state"].double(), torch.zeros(s["v"].shape, device="cuda", dtype=torch.float64)
        group = case["Hv"] // case["Hk"]
        for r, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            S = state[slot]
            for t in range(case["T"]):
                k, q = (s[n][r, t].double().repeat_interleave(group, 0) for n in ("k", "q"))
                S = torch.exp(s["g"][r, t].double())[:, None, None] * S
                e = s["beta"][r, t].double()[:, None] * (s["v"][r, t].double() - (k[:, None] @ S)[:, 0])
                S = S + k[..., None] * e[:, None]
                out[r, t] = case["Dk"] ** -0.5 * (q[:, None] @ S)[:, 0]
            state[slot] = S
        return {"out": out, "state": state}


# ---- what a pass cannot do without --------------------------------------------------------

def work(case):
    op = case["op"]
    es = _ES.get(case.get("dtype"), 4)
    if op == "delta":
        T, N = case["B"] * case["L"], case["seqs"] or case["B"]
        Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
        qk, v, gates, state = 2 * T * Hk * Dk * es, T * Hv * Dv * es, T * Hv * (4 + _ES[case["beta"]]), N * Hv * Dk * Dv * 4
        carried = state if case["states"] else 0
        nbytes = qk + 2 * v + gates + state + carried
        flops = 6 * T * Hv * Dk * Dv                      # S^T k, the write, S^T q
        if case["mode"] == "train":                       # dout in; the five gradients and the states' out
            nbytes += v + qk + v + gates + 2 * carried
            flops += 14 * T * Hv * Dk * Dv                # seven such products more
        return {"bytes": nbytes, "flops": flops}
    if op == "step":
        live, T = case["B"] - case["idle"], case["T"]
        Hk, Hv, Dk, Dv = case["Hk"], case["Hv"], case["Dk"], case["Dv"]
        per = 2 * Hv * Dk * Dv * 4 + T * ((2 * Hk * Dk + 2 * Hv * Dv) * es + Hv * (4 + _ES[case["beta"]]))
        return {"bytes": live * per, "flops": live * T * Hv * Dk * Dv * 7}
    if op == "norm":
        n = case["rows"] * case["heads"] * case["width"]
        if case["mode"] == "fwd":
            return {"bytes": 2 * n * es, "flops": 8 * n}
        return {"bytes": 4 * n * es, "flops": 24 * n}     # x, dout in; out, dx out
    return {"bytes": 8 * case["count"] + 8 * case["total"], "flops": 2 * case["total"]}
