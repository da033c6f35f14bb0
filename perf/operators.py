"""Cases of the recurrent-state operators: the gated linear recurrence (prefill,
training step, decode step) and beam search over recurrent states (selection,
reordering, decode steps that read the parents' states).

``run`` computes each in elementary torch operations, or, where ``own`` is set,
through the package's entry points.
"""
import math
import random

import torch

own = False

_F32 = torch.float32
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _kda():
    from gated_delta_rule_45_gb300 import kda
    return kda


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one short prompt of the smallest layer: launch latency
        dict(name="linrec_prefill_tiny", op="linrec_prefill", N=1, T=64, cut=0, H=2, d=32,
             dtype="fp32", gate="channel", complement=False, mu=3.0, s0=False),
        # one long document, the log gate of a trained layer in bf16
        dict(name="linrec_prefill_long", op="linrec_prefill", N=1, T=131072, cut=0, H=32, d=128,
             dtype="bf16", gate="log_bf16", complement=False, mu=5.0, s0=True),
        # a serving batch: 64 prompts of about 128 to 8300 tokens, continued from stored states
        dict(name="linrec_prefill_varlen", op="linrec_prefill", N=64, T=266240, cut=46, H=16,
             d=256, dtype="bf16", gate="channel", complement=False, mu=3.0, s0=True),
        # a training step of the standard shape: outputs, final states and every gradient
        dict(name="linrec_train", op="linrec_train", N=8, T=32768, cut=-1, H=32, d=128,
             dtype="bf16", gate="channel", complement=False, mu=3.0, s0=False),
        # odd widths, ragged lengths with empty sequences, one gate a head, leaky average
        dict(name="linrec_train_odd", op="linrec_train", N=13, T=5003, cut=7, H=5, d=67,
             dtype="fp32", gate="head", complement=True, mu=3.0, s0=True),
        # one token for each of 256 sequences (64 requests of 4 beams), states of the parents
        dict(name="linrec_decode", op="linrec_decode", B=64, K=4, H=32, d=128, dtype="bf16",
             gate="channel", complement=False),
        # one interactive request with 4 beams, a few of them finished
        dict(name="beam_select_one", op="beam_select", B=1, K=4, V=32000, n=8, dtype="fp32",
             masked=0.0),
        # a full batch, wide beams, 16-bit logits with a tenth of the vocabulary masked
        dict(name="beam_select_batch", op="beam_select", B=64, K=8, V=128000, n=16, dtype="bf16",
             masked=0.1),
        # one request: a small matrix state and a vector state move together
        dict(name="beam_reorder_one", op="beam_reorder", B=1, K=4, H=2, dv=32, dk=32),
        # 32 requests of 8 beams, one layer's matrix and vector states
        dict(name="beam_reorder_batch", op="beam_reorder", B=32, K=8, H=32, dv=128, dk=128),
        # the decode step of one request with 4 beams
        dict(name="kda_decode_parents_one", op="kda_decode_parents", B=1, K=4, H=16, dv=256,
             dk=128, dtype="bf16", gate="channel"),
        # the decode step of 32 requests of 8 beams
        dict(name="kda_decode_parents_batch", op="kda_decode_parents", B=32, K=8, H=32, dv=128,
             dk=128, dtype="bf16", gate="channel"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linrec_prefill", "linrec_prefill", "linrec_train", "linrec_decode",
                     "beam_select", "beam_select", "beam_reorder", "kda_decode_parents"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("linrec_prefill", "linrec_train"):
        H = _log_int(rng, 1, 48)
        d = rng.choice([32, 64, 64, 128, 128, 256, _log_int(rng, 1, 256)])
        most = (1 << 28) if op == "linrec_prefill" else (1 << 26)
        T = _log_int(rng, 1, min(200000, most // (H * d)))
        return dict(op=op, N=_log_int(rng, 1, 300), T=T, cut=rng.randrange(1, 10 ** 6), H=H, d=d,
                    dtype=dtype, gate=rng.choice(["channel", "channel", "log_bf16", "head"]),
                    complement=rng.random() < 0.4, mu=round(rng.uniform(2.0, 6.0), 2),
                    s0=rng.random() < 0.6)
    B, K = _log_int(rng, 1, 64), rng.choice([1, 2, 3, 4, 4, 5, 8, 8, 12, 16])
    if op == "beam_reorder":
        K = max(K, 2)
    if op == "linrec_decode":
        return dict(op=op, B=B, K=K, H=_log_int(rng, 1, 40),
                    d=rng.choice([64, 128, 128, 256, _log_int(rng, 1, 256)]), dtype=dtype,
                    gate=rng.choice(["channel", "log_bf16", "head"]),
                    complement=rng.random() < 0.4)
    if op == "beam_select":
        V = _log_int(rng, 40, 260000)
        B = min(B, max(1, 60_000_000 // (V * K)))
        return dict(op=op, B=B, K=K, V=V, n=min(rng.choice([K, 2 * K, 2 * K, K + 1]), K * V),
                    dtype=dtype, masked=rng.choice([0.0, 0.0, 0.1, 0.9]))
    H, dk = _log_int(rng, 1, 32), rng.choice([32, 64, 128, 128])
    dv = rng.choice([64, 128, 128, 256]) if op == "beam_reorder" else \
        rng.choice([64, 128, 128, 256, _log_int(rng, 1, 256)])
    B = min(B, max(1, 130_000_000 // (K * H * dv * dk)))
    case = dict(op=op, B=B, K=K, H=H, dv=dv, dk=dk)
    if op == "kda_decode_parents":
        case.update(dtype=dtype, gate=rng.choice(["channel", "log_bf16", "head"]))
    return case


def _lengths(case):
    """Sequence lengths that add up to T: cut < 0 equal ones, else cut points drawn
    from the number (empty sequences among them)."""
    N, T, cut = case["N"], case["T"], case["cut"]
    if N == 1:
        return [T]
    if cut < 0:
        base = [T // N] * N
        base[-1] += T - sum(base)
        return base
    r = random.Random(cut)
    if T >= 128 * N:
        # each at least 128 and the rest shared out by uniform weights
        w = [r.random() for _ in range(N)]
        spare = T - 128 * N
        lens = [128 + int(spare * x / sum(w)) for x in w]
        lens[-1] += T - sum(lens)
        if N >= 8 and cut % 2:
            lens[1] += lens[3]
            lens[3] = 0
        return lens
    points = sorted(r.randint(0, T) for _ in range(N - 1))
    return [b - a for a, b in zip([0] + points, points + [T])]


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _gate(g, lead, H, d, layout, mu):
    if layout == "head":
        return torch.sigmoid(_randn(g, *lead, H) + mu)
    z = _randn(g, *lead, H, d).add_(mu)
    if layout == "log_bf16":
        return torch.nn.functional.logsigmoid(z).to(torch.bfloat16)
    return z.sigmoid_()


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _parents(g, B, K):
    """int32 [B K]: for each beam the row of its parent, among its own request's rows."""
    p = torch.randint(0, K, (B, K), device="cuda", generator=g)
    return (p + torch.arange(B, device="cuda")[:, None] * K).to(torch.int32).reshape(-1)


def prepare(case, seed):
    g, op, s = _gen(seed), case["op"], dict(case)
    if op in ("linrec_prefill", "linrec_train"):
        T, H, d, N = case["T"], case["H"], case["d"], case["N"]
        dt = _DT[case["dtype"]]
        s["x"] = _randn(g, T, H, d).to(dt)
        s["a"] = _gate(g, (T,), H, d, case["gate"], case["mu"])
        s["S0"] = _randn(g, N, H, d) * 0.1 if case["s0"] else None
        lens = _lengths(case)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["longest"] = max(lens)
        # first and last token of the sequences that have any, and which sequences those are
        full = [n for n in range(N) if lens[n] > 0]
        s["seq"] = torch.tensor(full, dtype=torch.int64, device="cuda")
        s["first"] = torch.tensor([cu[n] for n in full], dtype=torch.int64, device="cuda")
        s["last"] = torch.tensor([cu[n + 1] - 1 for n in full], dtype=torch.int64, device="cuda")
        if op == "linrec_train":
            s["dy"] = _randn(g, T, H, d).to(dt)
            s["dS_T"] = _randn(g, N, H, d)
        return s
    B, K = case["B"], case["K"]
    R = B * K
    if op == "beam_select":
        V = case["V"]
        x = _randn(g, R, V).mul_(3.0)
        if case["masked"] > 0:
            x.masked_fill_(torch.rand(R, V, device="cuda", generator=g) < case["masked"],
                           -math.inf)
        s["logits"] = x.to(_DT[case["dtype"]])
        s["scores"] = (-8.0 * torch.rand(B, K, device="cuda", generator=g) - 20.0)
        s["finished"] = (torch.rand(B, K, device="cuda", generator=g) < 0.15).to(torch.uint8)
        s["eos"] = 2
        return s
    H = case["H"]
    s["parents"] = _parents(g, B, K)
    if op == "linrec_decode":
        d = case["d"]
        s["x"] = _randn(g, R, H, d).to(_DT[case["dtype"]])
        s["a"] = _gate(g, (R,), H, d, case["gate"], 4.0)
        s["S"] = _randn(g, R, H, d) * 0.1
        s["S_out"] = torch.empty_like(s["S"])
        return s
    dv, dk = case["dv"], case["dk"]
    if op == "beam_reorder":
        s["states"] = [_randn(g, R, H, dv, dk), _randn(g, R, H, dv)]
        return s
    dt = _DT[case["dtype"]]
    s["q"] = _unit(_randn(g, R, H, dk)).to(dt)
    s["k"] = _unit(_randn(g, R, H, dk)).to(dt)
    s["v"] = _randn(g, R, H, dv).to(dt)
    s["alpha"] = _gate(g, (R,), H, dv, case["gate"], 4.0)
    s["beta"] = torch.sigmoid(_randn(g, R, H))
    s["S"] = _randn(g, R, H, dv, dk) * 0.1
    s["S_out"] = torch.empty_like(s["S"])
    return s


# ---------------------------------------------------------------- plain forms

def _gate32(a, layout):
    """The gate and one minus the gate in 32 bits, broadcastable over [.., H, d]."""
    if layout == "log_bf16":
        la = a.to(_F32)
        return torch.exp(la), -torch.expm1(la)
    a = a.unsqueeze(-1) if layout == "head" else a
    return a, 1.0 - a


def _scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling; a is 0 where nothing is
    carried in, and nothing is carried over more than `longest` rows."""
    off = 1
    while off < longest:
        b = torch.cat([b[:off], torch.addcmul(b[off:], a[off:], b[:-off])])
        a = torch.cat([a[:off], a[off:] * a[:-off]])
        off *= 2
    return b


def _linrec_forward(s):
    x = s["x"].to(_F32)
    a, na = _gate32(s["a"], s["gate"])
    u = na * x if s["complement"] else x.clone()
    a = a.expand(x.shape).clone()
    if s["S0"] is not None:
        u[s["first"]] += a[s["first"]] * s["S0"][s["seq"]]
    a[s["first"]] = 0.0
    h = _scan(a, u, s["longest"])
    N = s["cu"].numel() - 1
    S_T = torch.zeros((N,) + x.shape[1:], dtype=_F32, device="cuda") if s["S0"] is None \
        else s["S0"].clone()
    S_T[s["seq"]] = h[s["last"]]
    return h, S_T


def _linrec_backward(s, h):
    x = s["x"].to(_F32)
    a, na = _gate32(s["a"], s["gate"])
    a = a.expand(x.shape)
    # g_t = dy_t + a_{t+1} g_{t+1}, a sequence's last token starting from dS_T
    c = torch.zeros_like(x)
    c[:-1] = a[1:]
    c[s["last"]] = 0.0
    b = s["dy"].to(_F32)
    b = b.clone() if b is s["dy"] else b
    b[s["last"]] += s["dS_T"][s["seq"]]
    g = _scan(c.flip(0), b.flip(0), s["longest"]).flip(0)
    prev = torch.zeros_like(h)
    prev[1:] = h[:-1]
    prev[s["first"]] = s["S0"][s["seq"]] if s["S0"] is not None else 0.0
    da = g * (prev - x) if s["complement"] else g * prev
    if s["gate"] == "log_bf16":
        da = a * da
    elif s["gate"] == "head":
        da = da.sum(-1)
    dS0 = s["dS_T"].clone()
    dS0[s["seq"]] = a[s["first"]] * g[s["first"]]
    return {"dx": na * g if s["complement"] else g, "dgate": da, "dS0": dS0}


def _ordered(x):
    """A whole number that sorts as the 32-bit float does."""
    i = x.view(torch.int32).to(torch.int64)
    return torch.where(i >= 0, i, -(i & 0x7fffffff) - 1)


def _beam_select(s):
    B, K, V, n = s["B"], s["K"], s["V"], s["n"]
    x = s["logits"].to(_F32).reshape(B, K, V)
    x = torch.where(torch.isnan(x), -math.inf, x)
    fin = s["finished"].reshape(B, K).bool()
    token = torch.arange(V, device="cuda")
    only = torch.where(token == s["eos"], 0.0, -math.inf)
    x = torch.where(fin[..., None], only, x)
    top = x.amax(-1, keepdim=True).double()
    top = torch.where(torch.isinf(top), 0.0, top)
    # 64 bits from here on: candidates of different beams lie close together
    lse = top + torch.log(torch.exp(x.double() - top).sum(-1, keepdim=True))
    # each beam's n best, equal logits by the lowest token
    m = min(n, V)
    code = _ordered(x) * (1 << 31) + (V - 1 - token)
    at = code.topk(m, dim=-1).indices
    key = s["scores"].double()[..., None] + (x.gather(-1, at).double() - lse)
    key = torch.where(torch.isnan(key), -math.inf, key).reshape(B, K * m)
    best, pick = torch.sort(key, dim=-1, descending=True, stable=True)
    pick = pick[:, :n]
    beam = pick // m
    rows = beam + torch.arange(B, device="cuda")[:, None] * K
    return {"scores": best[:, :n].to(_F32), "parents": rows.to(torch.int32),
            "tokens": at.reshape(B, K * m).gather(1, pick).to(torch.int32)}


def _kda_decode(s):
    q, k, v = (s[n].to(_F32) for n in ("q", "k", "v"))
    al, _ = _gate32(s["alpha"], s["gate"])
    S = s["S"][s["parents"].long()] * al.unsqueeze(-1)
    err = s["beta"].unsqueeze(-1) * (v - (S * k.unsqueeze(-2)).sum(-1))
    S += err.unsqueeze(-1) * k.unsqueeze(-2)
    s["S_out"].copy_(S)
    return {"o": (S * q.unsqueeze(-2)).sum(-1).to(s["q"].dtype), "S": s["S_out"]}


def run(s):
    op = s["op"]
    if own:
        return _run_own(s)
    if op == "linrec_prefill":
        h, S_T = _linrec_forward(s)
        return {"y": h.to(s["x"].dtype), "S_T": S_T}
    if op == "linrec_train":
        h, S_T = _linrec_forward(s)
        return {"y": h.to(s["x"].dtype), "S_T": S_T, **_linrec_backward(s, h)}
    if op == "linrec_decode":
        x = s["x"].to(_F32)
        a, na = _gate32(s["a"], s["gate"])
        S = a * s["S"][s["parents"].long()] + (na * x if s["complement"] else x)
        s["S_out"].copy_(S)
        return {"y": S.to(s["x"].dtype), "S": s["S_out"]}
    if op == "beam_select":
        return _beam_select(s)
    if op == "beam_reorder":
        p = s["parents"].long()
        return [t.copy_(t[p]) for t in s["states"]]
    return _kda_decode(s)


def _run_own(s):
    kda, op = _kda(), s["op"]
    if op == "linrec_prefill":
        y, S_T = kda.linrec_prefill(s["x"], s["a"], s["S0"], s["cu"], gate=s["gate"],
                                    complement=s["complement"])
        return {"y": y, "S_T": S_T}
    if op == "linrec_train":
        y, S_T, states = kda.linrec_prefill(s["x"], s["a"], s["S0"], s["cu"], gate=s["gate"],
                                            complement=s["complement"], save_states=True)
        grads = kda.linrec_backward(s["x"], s["a"], s["S0"], s["cu"], s["dy"], s["dS_T"],
                                    states=states, gate=s["gate"], complement=s["complement"])
        return {"y": y, "S_T": S_T, "dx": grads["dx"], "dgate": grads["dgate"],
                "dS0": grads["dS0"]}
    if op == "linrec_decode":
        y = kda.linrec_decode_step(s["x"], s["a"], s["S"], parents=s["parents"],
                                   S_out=s["S_out"], gate=s["gate"], complement=s["complement"])
        return {"y": y, "S": s["S_out"]}
    if op == "beam_select":
        scores, parents, tokens = kda.beam_select(s["logits"], s["scores"], s["n"],
                                                  finished=s["finished"], eos=s["eos"])
        return {"scores": scores, "parents": parents, "tokens": tokens}
    if op == "beam_reorder":
        kda.beam_reorder(s["states"], s["parents"], s["K"])
        return s["states"]
    o = kda.decode_step_parents(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["S"],
                                s["parents"], s["S_out"], gate=s["gate"])
    return {"o": o, "S": s["S_out"]}


# ---------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("linrec_prefill", "linrec_train"):
        T, H, d, N = case["T"], case["H"], case["d"], case["N"]
        e, D = _DT[case["dtype"]].itemsize, H * d
        gate = {"channel": 4 * D, "log_bf16": 2 * D, "head": 4 * H}[case["gate"]]
        state = 4 * N * D
        total = T * (2 * e * D + gate) + state * (2 if case["s0"] else 1)
        flops = 2 * T * D
        if op == "linrec_train":
            # x, gate and dy in, dx and the gate's gradient out, in 32 bits
            dgate = 4 * H if case["gate"] == "head" else 4 * D
            total += T * (2 * e * D + gate + 4 * D + dgate) + 2 * state
            flops += 6 * T * D
        return {"bytes": total, "flops": flops}
    B, K = case["B"], case["K"]
    R = B * K
    if op == "beam_select":
        e = _DT[case["dtype"]].itemsize
        return {"bytes": R * case["V"] * e + R * 5 + B * case["n"] * 12,
                "flops": 3 * R * case["V"]}
    # rows of a request that some beam descends from, parents drawn uniformly
    parents = K * (1.0 - (1.0 - 1.0 / K) ** K)
    H = case["H"]
    if op == "linrec_decode":
        D, e = H * case["d"], _DT[case["dtype"]].itemsize
        gate = {"channel": 4 * D, "log_bf16": 2 * D, "head": 4 * H}[case["gate"]]
        return {"bytes": R * (2 * e * D + gate + 4 * D + 4) + B * parents * 4 * D,
                "flops": 2 * R * D}
    dv, dk = case["dv"], case["dk"]
    if op == "beam_reorder":
        row = 4 * H * dv * (dk + 1)
        moved = K - 1.0                                       # rows whose parent is another row
        read = K * (1.0 - (1.0 - 1.0 / K) ** (K - 1))         # rows that another row descends from
        return {"bytes": B * (moved + read) * row + 4 * R, "flops": 0}
    e, row = _DT[case["dtype"]].itemsize, 4 * H * dv * dk
    gate = {"channel": 4 * H * dv, "log_bf16": 2 * H * dv, "head": 4 * H}[case["gate"]]
    return {"bytes": R * row + B * parents * row + R * (2 * e * H * (dk + dv) + gate + 4 * H + 4),
            "flops": 7 * R * H * dv * dk}


# ---------------------------------------------------------------- 64 bits

def _exact_gate(s, a):
    a = a.double()
    if s["gate"] == "log_bf16":
        a = a.exp()
    return a.unsqueeze(-1) if s["gate"] == "head" else a


def _exact_linrec(s):
    """Token by token, all sequences that are still running at once."""
    cu = s["cu"].tolist()
    order = sorted(range(len(cu) - 1), key=lambda n: cu[n] - cu[n + 1])   # longest first
    lens = [cu[n + 1] - cu[n] for n in order]
    start = torch.tensor([cu[n] for n in order], device="cuda")
    at = torch.tensor(order, device="cuda")
    T, H, d = s["x"].shape
    S = torch.zeros(len(order), H, d, dtype=torch.float64, device="cuda") if s["S0"] is None \
        else s["S0"].double()[at]
    h = torch.zeros(T, H, d, dtype=torch.float64, device="cuda")
    live = len(order)
    for t in range(lens[0]):
        while live and lens[live - 1] <= t:
            live -= 1
        tok = start[:live] + t
        a = _exact_gate(s, s["a"][tok])
        x = s["x"][tok].double()
        S[:live] = a * S[:live] + ((1.0 - a) * x if s["complement"] else x)
        h[tok] = S[:live]
    S_T = torch.empty_like(S)
    S_T[at] = S
    out = {"y": h, "S_T": S_T}
    if s["op"] == "linrec_prefill":
        return out
    # G: the gradient that reaches the state from behind
    G = s["dS_T"].double()[at]
    S0 = torch.zeros_like(S) if s["S0"] is None else s["S0"].double()[at]
    dx = torch.zeros_like(h)
    da = torch.zeros(s["a"].shape, dtype=torch.float64, device="cuda")
    live = 0
    for t in range(lens[0] - 1, -1, -1):
        while live < len(order) and lens[live] > t:
            live += 1
        tok = start[:live] + t
        a = _exact_gate(s, s["a"][tok])
        x = s["x"][tok].double()
        g = G[:live] + s["dy"][tok].double()
        before = S0[:live] if t == 0 else h[tok - 1]
        if s["complement"]:
            dx[tok], w = (1.0 - a) * g, g * (before - x)
        else:
            dx[tok], w = g, g * before
        da[tok] = w.sum(-1) if s["gate"] == "head" else a * w if s["gate"] == "log_bf16" else w
        G[:live] = a * g
    dS0 = torch.empty_like(G)
    dS0[at] = G
    return {**out, "dx": dx, "dgate": da, "dS0": dS0}


def _exact_beam_select(s):
    B, K, V, n = s["B"], s["K"], s["V"], s["n"]
    best = []
    for b in range(B):
        x = s["logits"][b * K:(b + 1) * K].double()
        c = s["scores"][b].double()[:, None] + torch.log_softmax(x, dim=-1)
        for k in range(K):
            if s["finished"][b, k]:
                c[k] = -math.inf
                c[k, s["eos"]] = s["scores"][b, k].double()
        c = c.reshape(-1)
        c = torch.where(torch.isnan(c), -math.inf, c)
        best.append(torch.topk(c, n).values)
    return {"scores": torch.stack(best), "parents": None, "tokens": None}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("linrec_prefill", "linrec_train"):
        return _exact_linrec(s)
    if op == "beam_select":
        return _exact_beam_select(s)
    rows = s["parents"].tolist()
    if op == "beam_reorder":
        return [torch.stack([t[p] for p in rows]).double() for t in s["states"]]
    if op == "linrec_decode":
        a, x = _exact_gate(s, s["a"]), s["x"].double()
        u = (1.0 - a) * x if case["complement"] else x
        S = a * torch.stack([s["S"][p] for p in rows]).double() + u
        return {"y": S, "S": S}
    o, S_new = [], []
    for i, p in enumerate(rows):
        q, k, v = (s[n][i].double() for n in ("q", "k", "v"))
        al = _exact_gate(s, s["alpha"][i])
        S = al.unsqueeze(-1) * s["S"][p].double()
        guess = torch.einsum("hvk,hk->hv", S, k)
        S = S + torch.einsum("hv,hk->hvk", s["beta"][i].double()[:, None] * (v - guess), k)
        o.append(torch.einsum("hvk,hk->hv", S, q))
        S_new.append(S.float() if S.numel() * len(rows) > 1 << 26 else S)
    return {"o": torch.stack(o), "S": torch.stack(S_new).double()}
