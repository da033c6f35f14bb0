"""Cases of the operators around the recurrences of a layer: the short causal convolution
before them, the selective state space scan (a recurrence whose step sizes and projections
come with each token) and the gated group norm of the heads behind them: prefill, training
step and decode step.

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
        dict(name="conv_prefill_tiny", op="conv_prefill", N=1, T=64, cut=0, H=2, d=32, W=4,
             dtype="fp32", silu=True, bias=True, s0=False),
        # a serving batch: 64 prompts of about 128 to 8300 tokens, continued from stored states
        dict(name="conv_prefill_varlen", op="conv_prefill", N=64, T=266240, cut=46, H=16, d=256,
             W=4, dtype="bf16", silu=True, bias=True, s0=True),
        # a training step of the standard shape: outputs, final states and every gradient
        dict(name="conv_train", op="conv_train", N=8, T=32768, cut=-1, H=32, d=128, W=4,
             dtype="bf16", silu=True, bias=True, s0=False),
        # one token for each of 256 sequences (64 requests of 4 beams), states of the parents
        dict(name="conv_decode", op="conv_decode", B=64, K=4, H=32, d=128, W=4, dtype="bf16",
             silu=True, bias=True),
        # one short prompt of the smallest layer
        dict(name="scan_prefill_tiny", op="scan_prefill", N=1, T=64, cut=0, H=1, d=64, n=16,
             dtype="fp32", z=True, bias=True, skip=True, s0=False),
        # one long document: few channels for the whole GPU, many tokens
        dict(name="scan_prefill_long", op="scan_prefill", N=1, T=131072, cut=0, H=1, d=4096, n=16,
             dtype="bf16", z=True, bias=True, skip=True, s0=True),
        # the serving batch of ragged prompts
        dict(name="scan_prefill_varlen", op="scan_prefill", N=64, T=266240, cut=46, H=1, d=2048,
             n=16, dtype="bf16", z=True, bias=True, skip=True, s0=True),
        # a training step of the standard shape: outputs, final states and every gradient
        dict(name="scan_train", op="scan_train", N=8, T=32768, cut=-1, H=1, d=4096, n=16,
             dtype="bf16", z=True, bias=True, skip=True, s0=False),
        # odd widths, ragged lengths with empty sequences, three groups of channels, no gate
        dict(name="scan_train_odd", op="scan_train", N=13, T=5003, cut=7, H=3, d=67, n=12,
             dtype="fp32", z=False, bias=False, skip=True, s0=True),
        # one token for each of 256 sequences, states of the parents
        dict(name="scan_decode", op="scan_decode", B=64, K=4, H=1, d=4096, n=16, dtype="bf16",
             z=True, bias=True, skip=True),
        # the outputs of 256 sequences' decode step, gated
        dict(name="norm_decode", op="norm_forward", T=256, H=32, d=128, dtype="bf16", z=True,
             act="sigmoid", center=False, affine="shared"),
        # a training step of the standard shape: output and every gradient
        dict(name="norm_train", op="norm_train", T=32768, H=32, d=128, dtype="bf16", z=True,
             act="silu", center=True, affine="head"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_prefill", "conv_train", "conv_decode", "scan_prefill", "scan_prefill",
                     "scan_train", "scan_train", "scan_decode", "norm_forward", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op.startswith("norm"):
        H = _log_int(rng, 1, 64)
        d = rng.choice([64, 128, 128, 256, 512, _log_int(rng, 1, 256), _log_int(rng, 256, 8192)])
        T = _log_int(rng, 1, max(2, min(100000, (1 << 27) // (H * d))))
        return dict(op=op, T=T, H=H, d=d, dtype=dtype, z=rng.random() < 0.7,
                    act=rng.choice(["silu", "silu", "sigmoid", "none"]),
                    center=rng.random() < 0.5,
                    affine=rng.choice(["shared", "shared", "head", "none"]))
    if op.startswith("conv"):
        case = dict(op=op, W=rng.choice([2, 3, 4, 4, 4]), dtype=dtype, silu=rng.random() < 0.8,
                    bias=rng.random() < 0.6)
    else:
        case = dict(op=op, n=rng.choice([8, 16, 16, 16, 16, 32, 64, _log_int(rng, 1, 64)]),
                    dtype=dtype, z=rng.random() < 0.6, bias=rng.random() < 0.7,
                    skip=rng.random() < 0.8)
    H = rng.choice([1, 1, 2, 4, _log_int(rng, 1, 32)])
    wide = _log_int(rng, 1, 8192 // H)
    d = rng.choice([64, 128, wide, wide, max(1, wide // 64) * 64])
    states = case.get("n", 1)
    if op.endswith("decode"):
        B, K = _log_int(rng, 1, 256), rng.choice([1, 1, 2, 4, 4, 5, 8])
        B = min(B, max(1, (1 << 25) // (K * H * d * states)))
        return dict(case, B=B, K=K, H=H, d=d)
    most = (1 << 31) if op == "scan_prefill" else (1 << 30) if op == "scan_train" else (1 << 27)
    T = _log_int(rng, 1, min(200000, max(2, most // (H * d * states))))
    return dict(case, N=_log_int(rng, 1, 200), T=T, cut=rng.randrange(1, 10 ** 6), H=H, d=d,
                s0=rng.random() < 0.6)


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


def _rand(g, *shape):
    return torch.rand(*shape, device="cuda", generator=g)


def _parents(g, B, K):
    """int32 [B K]: for each beam the row of its parent, among its own request's rows."""
    p = torch.randint(0, K, (B, K), device="cuda", generator=g)
    return (p + torch.arange(B, device="cuda")[:, None] * K).to(torch.int32).reshape(-1)


def _packed(s, case):
    N = case["N"]
    lens = _lengths(case)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    dev = dict(dtype=torch.int64, device="cuda")
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["longest"] = max(lens)
    # first and last token of the sequences that have any, and which sequences those are
    full = [n for n in range(N) if lens[n] > 0]
    s["seq"] = torch.tensor(full, **dev)
    s["first"] = torch.tensor([cu[n] for n in full], **dev)
    s["last"] = torch.tensor([cu[n + 1] - 1 for n in full], **dev)
    # each token's sequence
    s["of"] = torch.repeat_interleave(torch.arange(N, device="cuda"),
                                      torch.tensor(lens, **dev))


def _scan_inputs(s, g, rows, case):
    """Inputs of the scan as a trained layer has them: steps of 0.001 to 0.1, decays of
    1 to n, projections of unit size."""
    H, d, n, dt = case["H"], case["d"], case["n"], _DT[case["dtype"]]
    s["x"] = _randn(g, rows, H, d).to(dt)
    step = torch.exp(_rand(g, H, d) * math.log(100.0) + math.log(1e-3))
    raw = step + torch.log(-torch.expm1(-step))      # softplus(raw) = step
    s["dt_bias"] = raw if case["bias"] else None
    s["dt"] = (_randn(g, rows, H, d) * 0.7 + (0.0 if case["bias"] else raw)).to(dt)
    s["A"] = -torch.exp(torch.log(torch.arange(1, n + 1, device="cuda").float())
                        + 0.1 * _randn(g, H, d, n))
    s["B"] = _randn(g, rows, H, n).to(dt)
    s["C"] = _randn(g, rows, H, n).to(dt)
    s["D"] = 1.0 + 0.1 * _randn(g, H, d) if case["skip"] else None
    s["z"] = _randn(g, rows, H, d).to(dt) if case["z"] else None


def prepare(case, seed):
    g, op, s = _gen(seed), case["op"], dict(case)
    H, d, dt = case["H"], case["d"], _DT[case["dtype"]]
    if op.startswith("norm"):
        T = case["T"]
        s["x"] = (_randn(g, T, H, d) * torch.exp(_randn(g, T, H, 1)) + 0.3).to(dt)
        s["z"] = _randn(g, T, H, d).to(dt) if case["z"] else None
        shape = {"shared": (d,), "head": (H, d), "none": None}[case["affine"]]
        s["w"] = 1.0 + 0.2 * _randn(g, *shape) if shape else None
        s["b"] = 0.2 * _randn(g, *shape) if shape and case["center"] else None
        if op == "norm_train":
            s["dy"] = _randn(g, T, H, d).to(dt)
        return s
    rows = case["B"] * case["K"] if op.endswith("decode") else case["T"]
    if op.startswith("conv"):
        W = case["W"]
        s["x"] = _randn(g, rows, H, d).to(dt)
        s["w"] = (2.0 * _rand(g, H, d, W) - 1.0) / math.sqrt(W)
        s["b"] = 0.1 * _randn(g, H, d) if case["bias"] else None
        state = lambda N: _randn(g, N, W - 1, H, d)
    else:
        _scan_inputs(s, g, rows, case)
        state = lambda N: _randn(g, N, H, d, case["n"]) * 0.1
    if op.endswith("decode"):
        s["parents"] = _parents(g, case["B"], case["K"])
        s["S"] = state(rows)
        if op == "conv_decode":
            s["S"] = s["S"].to(dt)
        s["S_out"] = torch.empty_like(s["S"])
        return s
    s["S0"] = state(case["N"]) if case["s0"] else None
    if op.startswith("conv") and case["s0"]:
        s["S0"] = s["S0"].to(dt)
    _packed(s, case)
    if op.endswith("train"):
        s["dy"] = _randn(g, rows, H, d).to(dt)
        s["dS_T"] = state(case["N"])
    return s


# ---------------------------------------------------------------- plain forms

def _silu_grad(v):
    g = torch.sigmoid(v)
    return g * (1.0 + v * (1.0 - g))


def _conv_window(s):
    """The inputs that reach each token, [W, T, H, d]: rows before a sequence's first come
    from its state; and the final states."""
    W, N = s["W"], s["cu"].numel() - 1
    x, cu = s["x"].to(_F32), s["cu"].long()
    S0 = torch.zeros((N, W - 1) + x.shape[1:], device="cuda") if s["S0"] is None \
        else s["S0"].to(_F32)
    t = torch.arange(x.shape[0], device="cuda")
    at = t - cu[s["of"]]                        # position in the sequence
    # every sequence's state and tokens in one column: row (W - 1)(n + 1) + t holds token t
    col = torch.empty((x.shape[0] + N * (W - 1),) + x.shape[1:], device="cuda")
    col[t + (W - 1) * (s["of"] + 1)] = x
    lead = cu[:-1, None] + (W - 1) * torch.arange(N, device="cuda")[:, None] \
        + torch.arange(W - 1, device="cuda")
    col[lead] = S0
    own_row = cu[s["of"]] + (W - 1) * (s["of"] + 1) + at
    tail = cu[1:, None] + (W - 1) * torch.arange(N, device="cuda")[:, None] \
        + torch.arange(W - 1, device="cuda")
    return torch.stack([col[own_row - (W - 1) + j] for j in range(W)]), col[tail], own_row, lead, \
        tail, col.shape[0]


def _conv_forward(s):
    win, S_T, *where = _conv_window(s)
    pre = (win * s["w"].permute(2, 0, 1)[:, None]).sum(0)
    if s["b"] is not None:
        pre = pre + s["b"]
    y = pre * torch.sigmoid(pre) if s["silu"] else pre
    return y.to(s["x"].dtype), S_T.to(s["x"].dtype), win, pre, where


def _conv_train(s):
    y, S_T, win, pre, (own_row, lead, tail, rows) = _conv_forward(s)
    W = s["W"]
    dpre = s["dy"].to(_F32) * _silu_grad(pre) if s["silu"] else s["dy"].to(_F32)
    dcol = torch.zeros((rows,) + dpre.shape[1:], device="cuda")
    for j in range(W):
        dcol[own_row - (W - 1) + j] += s["w"][..., j] * dpre
    dcol[tail] += s["dS_T"]
    return {"y": y, "S_T": S_T, "dx": dcol[own_row], "dS0": dcol[lead],
            "dw": torch.stack([(win[j] * dpre).sum(0) for j in range(W)], dim=-1),
            **({"db": dpre.sum(0)} if s["b"] is not None else {})}


def _conv_decode(s):
    win = torch.cat([s["S"][s["parents"].long()], s["x"][:, None]], dim=1)
    pre = (win.to(_F32) * s["w"].permute(2, 0, 1)).sum(1)
    if s["b"] is not None:
        pre = pre + s["b"]
    y = pre * torch.sigmoid(pre) if s["silu"] else pre
    s["S_out"].copy_(win[:, 1:])
    return {"y": y.to(s["x"].dtype), "S": s["S_out"]}


def _scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling; a is 0 where nothing is
    carried in, and nothing is carried over more than `longest` rows.  Overwrites a."""
    off = 1
    while off < longest:
        nb = torch.empty_like(b)
        nb[:off] = b[:off]
        torch.addcmul(b[off:], a[off:], b[:-off], out=nb[off:])
        b = nb
        if 2 * off < longest:
            na = torch.empty_like(a)
            na[:off] = a[:off]
            torch.mul(a[off:], a[:-off], out=na[off:])
            a = na
        off *= 2
    return b


_SLICE = 1 << 27      # state values of one slice of channels


def _scan_step_size(s):
    v = s["dt"].to(_F32)
    if s["dt_bias"] is not None:
        v = v + s["dt_bias"]
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-v.abs())), torch.sigmoid(v)


def _scan_slices(s, train):
    """Prefill, and with `train` every gradient, channels of one group at a time in slices
    that fit the memory."""
    x, H, d, n = s["x"], s["H"], s["d"], s["n"]
    T, N = x.shape[0], s["cu"].numel() - 1
    first, last, seq = s["first"], s["last"], s["seq"]
    new = lambda *shape: torch.zeros(*shape, device="cuda")
    out = {"y": torch.empty_like(x), "S_T": new(N, H, d, n) if s["S0"] is None else s["S0"].clone()}
    if train:
        out.update(dx=new(T, H, d), ddt=new(T, H, d), dA=new(H, d, n), dB=new(T, H, n),
                   dC=new(T, H, n), dS0=s["dS_T"].clone())
        if s["D"] is not None:
            out["dD"] = new(H, d)
        if s["z"] is not None:
            out["dz"] = new(T, H, d)
        if s["dt_bias"] is not None:
            out["ddt_bias"] = new(H, d)
    step, slope = _scan_step_size(s)
    wide = max(1, _SLICE // (T * n))
    for h in range(H):
        Bm, Cm = s["B"][:, h].to(_F32)[:, None], s["C"][:, h].to(_F32)[:, None]
        for c in range(0, d, wide):
            k = (slice(None), h, slice(c, min(d, c + wide)))
            A, dl, u = s["A"][k[1:]], step[k], x[k].to(_F32)
            a = torch.exp(dl[..., None] * A)
            b = (dl * u)[..., None] * Bm
            if s["S0"] is not None:
                b[first] += a[first] * s["S0"][seq][k]
            g = a.clone() if train else a
            g[first] = 0.0
            hs = _scan(g, b, s["longest"])
            out["S_T"][:, h, k[2]] = out["S_T"][k].index_copy(0, seq, hs[last])
            raw = (hs * Cm).sum(-1)
            if s["D"] is not None:
                raw = raw + s["D"][k[1:]] * u
            z = s["z"][k].to(_F32) if s["z"] is not None else None
            out["y"][k] = (raw if z is None else raw * (z * torch.sigmoid(z))).to(x.dtype)
            if not train:
                continue
            dr = s["dy"][k].to(_F32)
            if z is not None:
                out["dz"][k] = dr * raw * _silu_grad(z)
                dr = dr * (z * torch.sigmoid(z))
            # g_t: the gradient of h_t, = C_t dr_t + a_{t+1} g_{t+1}
            carry = torch.zeros_like(a)
            carry[:-1] = a[1:]
            carry[last] = 0.0
            g = dr[..., None] * Cm
            g[last] += s["dS_T"][seq][k]
            g = _scan(carry.flip(0), g.flip(0), s["longest"]).flip(0)
            out["dS0"][:, h, k[2]] = out["dS0"][k].index_copy(0, seq, a[first] * g[first])
            out["dC"][:, h] += (hs * dr[..., None]).sum(1)
            out["dB"][:, h] += (g * (dl * u)[..., None]).sum(1)
            gb = (g * Bm).sum(-1)
            # what came in from the step before, times its gate
            w = hs - (dl * u)[..., None] * Bm
            w *= g
            out["dA"][k[1:]] = (w * dl[..., None]).sum(0)
            ddl = (w * A).sum(-1) + gb * u
            du = gb * dl
            if s["D"] is not None:
                du = du + s["D"][k[1:]] * dr
                out["dD"][k[1:]] = (dr * u).sum(0)
            out["dx"][k] = du
            out["ddt"][k] = ddl * slope[k]
            if s["dt_bias"] is not None:
                out["ddt_bias"][k[1:]] = out["ddt"][k].sum(0)
    return out


def _scan_decode(s):
    step, _ = _scan_step_size(s)
    x = s["x"].to(_F32)
    S = torch.exp(step[..., None] * s["A"]) * s["S"][s["parents"].long()]
    S += (step * x)[..., None] * s["B"].to(_F32)[:, :, None]
    y = (S * s["C"].to(_F32)[:, :, None]).sum(-1)
    if s["D"] is not None:
        y = y + s["D"] * x
    if s["z"] is not None:
        z = s["z"].to(_F32)
        y = y * (z * torch.sigmoid(z))
    s["S_out"].copy_(S)
    return {"y": y.to(s["x"].dtype), "S": s["S_out"]}


_EPS = 1e-5


def _act(v, act):
    """act(v) and its slope."""
    g = torch.sigmoid(v)
    if act == "silu":
        return v * g, g * (1.0 + v * (1.0 - g))
    if act == "sigmoid":
        return g, g * (1.0 - g)
    return v, torch.ones_like(v)


def _norm(s):
    x, d = s["x"].to(_F32), s["d"]
    xc = x - x.mean(-1, keepdim=True) if s["center"] else x
    r = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + _EPS)
    xh = xc * r
    v = xh * s["w"] if s["w"] is not None else xh
    if s["b"] is not None:
        v = v + s["b"]
    if s["z"] is not None:
        z = s["z"].to(_F32)
        act, slope = _act(z, s["act"])
        y = v * act
    else:
        y, slope = _act(v, s["act"])
    out = {"y": y.to(s["x"].dtype)}
    if s["op"] == "norm_forward":
        return out
    dy = s["dy"].to(_F32)
    if s["z"] is not None:
        out["dz"] = dy * v * slope
        dv = dy * act
    else:
        dv = dy * slope
    if s["w"] is not None:
        over = (0, 1) if s["w"].dim() == 1 else (0,)
        out["dw"] = (dv * xh).sum(over)
        if s["b"] is not None:
            out["db"] = dv.sum(over)
        dv = dv * s["w"]
    dx = dv - xh * (dv * xh).mean(-1, keepdim=True)
    if s["center"]:
        dx = dx - dv.mean(-1, keepdim=True)
    out["dx"] = dx * r
    return out


def run(s):
    op = s["op"]
    if own:
        return _run_own(s)
    if op == "conv_prefill":
        y, S_T, *_ = _conv_forward(s)
        return {"y": y, "S_T": S_T}
    if op == "conv_train":
        return _conv_train(s)
    if op == "conv_decode":
        return _conv_decode(s)
    if op in ("scan_prefill", "scan_train"):
        return _scan_slices(s, op == "scan_train")
    if op == "scan_decode":
        return _scan_decode(s)
    return _norm(s)


def _run_own(s):
    kda, op = _kda(), s["op"]
    if op == "conv_prefill":
        y, S_T = kda.causalconv_prefill(s["x"], s["w"], s["b"], s["S0"], s["cu"], silu=s["silu"])
        return {"y": y, "S_T": S_T}
    if op == "conv_train":
        y, S_T = kda.causalconv_prefill(s["x"], s["w"], s["b"], s["S0"], s["cu"], silu=s["silu"])
        grads = kda.causalconv_backward(s["x"], s["w"], s["b"], s["S0"], s["cu"], s["dy"],
                                        s["dS_T"], silu=s["silu"])
        return {"y": y, "S_T": S_T, **grads}
    if op == "conv_decode":
        y = kda.causalconv_decode_step(s["x"], s["w"], s["b"], s["S"], parents=s["parents"],
                                       S_out=s["S_out"], silu=s["silu"])
        return {"y": y, "S": s["S_out"]}
    if op.startswith("scan"):
        more = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
        ins = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    if op == "scan_prefill":
        y, S_T = kda.selscan_prefill(*ins, s["S0"], s["cu"], **more)
        return {"y": y, "S_T": S_T}
    if op == "scan_train":
        y, S_T, states = kda.selscan_prefill(*ins, s["S0"], s["cu"], save_states=True, **more)
        grads = kda.selscan_backward(*ins, s["S0"], s["cu"], s["dy"], s["dS_T"], states=states,
                                     **more)
        return {"y": y, "S_T": S_T, **grads}
    if op == "scan_decode":
        y = kda.selscan_decode_step(*ins, s["S"], parents=s["parents"], S_out=s["S_out"], **more)
        return {"y": y, "S": s["S_out"]}
    kw = dict(z=s["z"], act=s["act"], center=s["center"], eps=_EPS)
    y = kda.groupnorm_forward(s["x"], s["w"], s["b"], **kw)
    if op == "norm_forward":
        return {"y": y}
    return {"y": y, **kda.groupnorm_backward(s["x"], s["w"], s["b"], s["dy"], **kw)}


# ---------------------------------------------------------------- work

def work(case):
    op, H, d = case["op"], case["H"], case["d"]
    D, e = H * d, _DT[case["dtype"]].itemsize
    if op.startswith("norm"):
        T = case["T"]
        par = {"shared": d, "head": D, "none": 0}[case["affine"]] * (2 if case["center"] else 1)
        total, flops = T * D * e * (3 if case["z"] else 2) + 4 * par, 8 * T * D
        if op == "norm_train":
            # x, gate and dy in, their gradients out in 32 bits
            total += T * D * (e * (3 if case["z"] else 2) + (8 if case["z"] else 4)) + 8 * par
            flops += 20 * T * D
        return {"bytes": total, "flops": flops}
    train = op.endswith("train")
    if op.startswith("conv"):
        W = case["W"]
        par = 4 * D * (W + (1 if case["bias"] else 0))
        if op == "conv_decode":
            R, K = case["B"] * case["K"], case["K"]
            parents = K * (1.0 - (1.0 - 1.0 / K) ** K)
            return {"bytes": R * (2 * e * D + (W - 1) * e * D + 4) +
                    case["B"] * parents * (W - 1) * e * D + par, "flops": 2 * W * R * D}
        T, N = case["T"], case["N"]
        state = N * (W - 1) * D
        total, flops = T * D * 2 * e + state * e * (2 if case["s0"] else 1) + par, 2 * W * T * D
        if train:
            total += T * D * (2 * e + 4) + state * (8 + (e if case["s0"] else 0)) + 2 * par
            flops += 6 * W * T * D
        return {"bytes": total, "flops": flops}
    n = case["n"]
    par = 4 * D * (n + (1 if case["bias"] else 0) + (1 if case["skip"] else 0))
    rows = 2 * D + 2 * H * n + (D if case["z"] else 0)      # x, dt, B, C and the gate
    if op == "scan_decode":
        R, K = case["B"] * case["K"], case["K"]
        parents = K * (1.0 - (1.0 - 1.0 / K) ** K)
        return {"bytes": R * (e * (rows + D) + 4 * D * n + 4) + case["B"] * parents * 4 * D * n +
                par, "flops": 7 * R * D * n}
    T, N = case["T"], case["N"]
    state = 4 * N * D * n
    total, flops = T * e * (rows + D) + state * (2 if case["s0"] else 1) + par, 7 * T * D * n
    if train:
        total += T * (e * (rows + D) + 4 * rows) + state * (3 if case["s0"] else 2) + 2 * par
        flops += 20 * T * D * n
    return {"bytes": total, "flops": flops}


# ---------------------------------------------------------------- 64 bits

def _f64(t):
    return None if t is None else t.double()


def _d_silu(v):
    e = torch.exp(-v)
    return (1.0 + e + v * e) / (1.0 + e) ** 2


def _exact_conv(s):
    """One sequence after another."""
    cu, W = s["cu"].tolist(), s["W"]
    w, b, N = s["w"].double(), _f64(s["b"]), s["cu"].numel() - 1
    S0 = torch.zeros((N, W - 1) + s["x"].shape[1:], dtype=torch.float64, device="cuda") \
        if s["S0"] is None else s["S0"].double()
    out = {k: [] for k in ("y", "S_T", "dx", "dS0")}
    dw, db = torch.zeros_like(w), torch.zeros_like(w[..., 0])
    train = s["op"] == "conv_train"
    for i in range(N):
        L = cu[i + 1] - cu[i]
        full = torch.cat([S0[i], s["x"][cu[i]:cu[i + 1]].double()])
        v = sum(full[j:j + L] * w[..., j] for j in range(W))
        v = v if b is None else v + b
        out["y"].append(v / (1.0 + torch.exp(-v)) if s["silu"] else v)
        out["S_T"].append(full[L:])
        if train:
            g = s["dy"][cu[i]:cu[i + 1]].double()
            g = g * _d_silu(v) if s["silu"] else g
            back = torch.zeros_like(full)
            for j in range(W):
                back[j:j + L] += g * w[..., j]
                dw[..., j] += (g * full[j:j + L]).sum(0)
            db += g.sum(0)
            back[L:] += s["dS_T"][i].double()
            out["dx"].append(back[W - 1:])
            out["dS0"].append(back[:W - 1])
    res = {"y": torch.cat(out["y"]), "S_T": torch.stack(out["S_T"])}
    if train:
        res.update(dx=torch.cat(out["dx"]), dS0=torch.stack(out["dS0"]), dw=dw)
        if b is not None:
            res["db"] = db
    return res


def _softplus64(s, rows):
    v = s["dt"][rows].double()
    if s["dt_bias"] is not None:
        v = v + s["dt_bias"].double()
    return torch.logaddexp(v, torch.zeros_like(v)), 1.0 / (1.0 + torch.exp(-v))


def _exact_scan(s):
    """Token by token, all sequences that are still running at once."""
    cu, train = s["cu"].tolist(), s["op"] == "scan_train"
    order = sorted(range(len(cu) - 1), key=lambda n: cu[n] - cu[n + 1])   # longest first
    lens = [cu[n + 1] - cu[n] for n in order]
    start = torch.tensor([cu[n] for n in order], device="cuda")
    at = torch.tensor(order, device="cuda")
    T, H, d = s["x"].shape
    A, skip, n = s["A"].double(), _f64(s["D"]), s["n"]
    f64 = dict(dtype=torch.float64, device="cuda")
    S0 = torch.zeros(len(order), H, d, n, **f64) if s["S0"] is None else s["S0"].double()[at]
    S, raw = S0.clone(), torch.zeros(T, H, d, **f64)
    kept = torch.zeros(T, H, d, n, **f64) if train else None      # the state before each token
    live = len(order)
    for t in range(lens[0]):
        while live and lens[live - 1] <= t:
            live -= 1
        tok = start[:live] + t
        dl, _ = _softplus64(s, tok)
        if train:
            kept[tok] = S[:live]
        S[:live] *= torch.exp(dl[..., None] * A)
        S[:live] += (dl * s["x"][tok].double())[..., None] * s["B"][tok].double()[:, :, None]
        raw[tok] = torch.einsum("bhdn,bhn->bhd", S[:live], s["C"][tok].double())
    if skip is not None:
        raw += skip * s["x"].double()
    z = _f64(s["z"])
    S_T = torch.empty_like(S)
    S_T[at] = S
    out = {"y": raw if z is None else raw * z / (1.0 + torch.exp(-z)), "S_T": S_T}
    if not train:
        return out
    dr = s["dy"].double()
    if z is not None:
        out["dz"] = dr * raw * _d_silu(z)
        dr = dr * z / (1.0 + torch.exp(-z))
    zeros = lambda *shape: torch.zeros(*shape, **f64)
    out.update(dx=zeros(T, H, d), ddt=zeros(T, H, d), dA=zeros(H, d, n), dB=zeros(T, H, n),
               dC=zeros(T, H, n))
    G = s["dS_T"].double()[at]      # the gradient that reaches the state from behind
    live = 0
    for t in range(lens[0] - 1, -1, -1):
        while live < len(order) and lens[live] > t:
            live += 1
        tok = start[:live] + t
        dl, slope = _softplus64(s, tok)
        x, Bm, Cm = (s[k][tok].double() for k in ("x", "B", "C"))
        a = torch.exp(dl[..., None] * A)
        ah = a * kept[tok]
        g = G[:live] + dr[tok][..., None] * Cm[:, :, None]
        out["dC"][tok] = torch.einsum("bhd,bhdn->bhn", dr[tok],
                                      ah + (dl * x)[..., None] * Bm[:, :, None])
        out["dB"][tok] = torch.einsum("bhdn,bhd->bhn", g, dl * x)
        gb = torch.einsum("bhdn,bhn->bhd", g, Bm)
        out["dA"] += torch.einsum("bhdn,bhd->hdn", g * ah, dl)
        out["dx"][tok] = gb * dl
        out["ddt"][tok] = (gb * x + (g * ah * A).sum(-1)) * slope
        G[:live] = a * g
    if skip is not None:
        out["dx"] += skip * dr
        out["dD"] = (dr * s["x"].double()).sum(0)
    if s["dt_bias"] is not None:
        out["ddt_bias"] = out["ddt"].sum(0)
    out["dS0"] = torch.empty_like(G)
    out["dS0"][at] = G
    return out


def _exact_norm(s):
    """Gradients from the derivative of each normalised value by each input."""
    x, d = s["x"].double(), s["d"]
    w = torch.ones(d, dtype=torch.float64, device="cuda") if s["w"] is None else s["w"].double()
    mean = x.sum(-1, keepdim=True) / d if s["center"] else torch.zeros_like(x[..., :1])
    sd = torch.sqrt(((x - mean) ** 2).sum(-1, keepdim=True) / d + _EPS)
    unit = (x - mean) / sd
    lin = unit * w + (0.0 if s["b"] is None else s["b"].double())
    arg = lin if s["z"] is None else s["z"].double()
    sig = 1.0 / (1.0 + torch.exp(-arg))
    f, df = {"silu": (arg * sig, _d_silu(arg)), "sigmoid": (sig, sig / (1.0 + torch.exp(arg))),
             "none": (arg, torch.ones_like(arg))}[s["act"]]
    out = {"y": f if s["z"] is None else lin * f}
    if s["op"] == "norm_forward":
        return out
    dy = s["dy"].double()
    if s["z"] is not None:
        out["dz"] = dy * lin * df
    dlin = dy * (df if s["z"] is None else f)
    du = dlin * w
    dsd = -(du * (x - mean)).sum(-1, keepdim=True) / sd ** 2
    dx = du / sd + dsd * (x - mean) / (d * sd)
    if s["center"]:
        # through the mean; the sum of x - mean is zero
        dx = dx - (du.sum(-1, keepdim=True) / sd) / d
    out["dx"] = dx
    if s["w"] is not None:
        over = [0] if s["w"].dim() == 2 else [0, 1]
        out["dw"] = (dlin * unit).sum(over)
        if s["b"] is not None:
            out["db"] = dlin.sum(over)
    return out


def exact(case, seed):
    op = case["op"]
    if op == "scan_train" and case["T"] * case["H"] * case["d"] * case["n"] > 1 << 32:
        return None      # the states of every token in 64 bits
    s = prepare(case, seed)
    if op in ("conv_prefill", "conv_train"):
        return _exact_conv(s)
    if op in ("scan_prefill", "scan_train"):
        return _exact_scan(s)
    if op.startswith("norm"):
        return _exact_norm(s)
    rows = s["parents"].tolist()
    S, x = torch.stack([s["S"][p] for p in rows]).double(), s["x"].double()
    if op == "conv_decode":
        w, W = s["w"].double(), s["W"]
        v = x * w[..., W - 1]
        for j in range(W - 1):
            v = v + S[:, j] * w[..., j]
        v = v if s["b"] is None else v + s["b"].double()
        return {"y": v / (1.0 + torch.exp(-v)) if s["silu"] else v,
                "S": torch.cat([S[:, 1:], x[:, None]], dim=1)}
    dl, _ = _softplus64(s, slice(None))
    S = torch.exp(torch.einsum("bhd,hdn->bhdn", dl, s["A"].double())) * S
    S = S + torch.einsum("bhd,bhn->bhdn", dl * x, s["B"].double())
    y = torch.einsum("bhdn,bhn->bhd", S, s["C"].double())
    if s["D"] is not None:
        y = y + s["D"].double() * x
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z / (1.0 + torch.exp(-z))
    return {"y": y, "S": S}
