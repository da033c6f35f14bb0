"""The operators around a recurrence together, as a layer uses them: convolution, projections,
scan and gated norm (a state space layer), and convolution, matrix-state recurrence and gated
norm (a linear attention layer); prompts and single tokens, and every gradient."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

from gated_delta_rule_45_gb300 import kda
from layer_checks import offsets

pytestmark = pytest.mark.gpu
EPS = 1e-5


def _layer(D, n, H, seed=0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    p = dict(w=rn(D, 4) * 0.4, b=0.1 * rn(D), P=rn(D, D + 2 * n) / D ** 0.5,
             A=-torch.exp(rn(1, D, n) * 0.5), Dk=rn(1, D), bias=rn(1, D) - 2.0,
             nw=1 + 0.2 * rn(D // H), nb=0.1 * rn(D // H))
    return {k: v.cuda() for k, v in p.items()}


def _split(proj, D, n):
    """dt, B and C as slices of one projection: strided rows."""
    T = proj.shape[0]
    return (proj[:, :D].unflatten(1, (1, D)), proj[:, D:D + n].unflatten(1, (1, n)),
            proj[:, D + n:].unflatten(1, (1, n)))


def _forward(p, xz, D, n, H, cu, S=None, save=False):
    """xz [T, 2 D]: input and gate, slices of one projection too."""
    T = xz.shape[0]
    conv0, scan0 = S if S is not None else (None, None)
    c, conv1 = kda.causalconv_prefill(xz[:, :D], p["w"], p["b"], conv0, cu)
    dt, B, C = _split(c @ p["P"], D, n)
    z = xz[:, D:]
    out = kda.selscan_prefill(c.view(T, 1, D), dt, p["A"], B, C, scan0, cu, D=p["Dk"],
                              dt_bias=p["bias"], save_states=save)
    y = kda.groupnorm_forward(out[0].view(T, H, D // H), p["nw"], p["nb"],
                              z=z.unflatten(1, (H, D // H)), center=True, eps=EPS)
    return y.view(T, D), (conv1, out[1]), (c, out[0], out[2] if save else None)


def _step(p, xz, D, n, H, S):
    R = xz.shape[0]
    c = kda.causalconv_decode_step(xz[:, :D], p["w"], p["b"], S[0])
    dt, B, C = _split(c @ p["P"], D, n)
    y = kda.selscan_decode_step(c.view(R, 1, D), dt, p["A"], B, C, S[1], D=p["Dk"],
                                dt_bias=p["bias"])
    return kda.groupnorm_forward(y.view(R, H, D // H), p["nw"], p["nb"],
                                 z=xz[:, D:].unflatten(1, (H, D // H)), center=True,
                                 eps=EPS).view(R, D)


@pytest.mark.parametrize("D,n,H", [(64, 16, 2), (96, 5, 4)])
def test_prompts_then_single_tokens(D, n, H):
    """A prompt and then steps give what the whole sequence gives.  Both sides keep some 200
    roundings of 2^-24 a value on the way (a state of up to 40 tokens, sums over n and over a
    head); the norm's row is of size 1."""
    p, lens, steps = _layer(D, n, H), [33, 7, 20], 6
    N = len(lens)
    g = torch.Generator().manual_seed(3)
    xz = torch.randn(N, max(lens) + steps, 2 * D, generator=g).cuda()
    whole = torch.cat([xz[i, :L + steps] for i, L in enumerate(lens)])
    cu_all, cu_t = offsets([L + steps for L in lens])
    want, (conv_w, scan_w), _ = _forward(p, whole, D, n, H, cu_t.cuda())
    prompt = torch.cat([xz[i, :L] for i, L in enumerate(lens)])
    cu, cut = offsets(lens)
    got, S, _ = _forward(p, prompt, D, n, H, cut.cuda())
    tol = 400 * 2.0 ** -24
    for i, L in enumerate(lens):
        torch.testing.assert_close(got[cu[i]:cu[i + 1]], want[cu_all[i]:cu_all[i] + L], rtol=tol,
                                   atol=4 * tol)
    S = (S[0].clone(), S[1].clone())
    for t in range(steps):
        y = _step(p, torch.stack([xz[i, L + t] for i, L in enumerate(lens)]), D, n, H, S)
        torch.testing.assert_close(y, torch.stack([want[cu_all[i] + L + t]
                                                   for i, L in enumerate(lens)]), rtol=tol,
                                   atol=4 * tol)
    torch.testing.assert_close(S[0], conv_w, rtol=0, atol=0)
    torch.testing.assert_close(S[1], scan_w, rtol=tol, atol=4 * tol)


def _plain(q, xz, D, n, H, cu):
    """The layer in 64 bits, token by token, for autograd."""
    outs = []
    for a, e in zip(cu, cu[1:]):
        x, z = xz[a:e, :D], xz[a:e, D:]
        L = e - a
        pad = torch.cat([x.new_zeros(3, D), x])
        c = F.silu(sum(pad[j:j + L] * q["w"][:, j] for j in range(4)) + q["b"])
        proj = c @ q["P"]
        step = F.softplus(proj[:, :D] + q["bias"][0])
        h = x.new_zeros(D, n)
        ys = []
        for t in range(L):
            h = torch.exp(step[t][:, None] * q["A"][0]) * h + \
                (step[t] * c[t])[:, None] * proj[t, D:D + n]
            ys.append(h @ proj[t, D + n:] + q["Dk"][0] * c[t])
        y = torch.stack(ys) if L else x
        v = F.group_norm(y, H, q["nw"].repeat(H), q["nb"].repeat(H), EPS)
        outs.append(v * F.silu(z))
    return torch.cat(outs)


@pytest.mark.parametrize("lens,D,n,H", [([17, 0, 30], 32, 8, 2), ([300], 16, 4, 1),
                                        ([5, 1, 40], 24, 16, 3)])
def test_gradients_of_the_layer(lens, D, n, H):
    """The chain of the three backward passes against autograd of the plain layer in 64 bits.
    Every operator and product leaves some 100 roundings of 2^-24 of the terms it adds up; five
    of them in a row, with sums that cancel to a fourth: 2000 of the largest gradient."""
    cu, cut = offsets(lens)
    T = cu[-1]
    p, g = _layer(D, n, H, seed=1), torch.Generator().manual_seed(4)
    xz, dy = torch.randn(T, 2 * D, generator=g).cuda(), torch.randn(T, D, generator=g).cuda()
    cut = cut.cuda()
    y, _, (c, ys, states) = _forward(p, xz, D, n, H, cut, save=True)

    shaped = lambda t: t.reshape(T, H, D // H)
    gn = kda.groupnorm_backward(shaped(ys), p["nw"], p["nb"], shaped(dy), z=shaped(xz[:, D:]),
                                center=True, eps=EPS)
    dt, B, C = _split(c @ p["P"], D, n)
    gs = kda.selscan_backward(c.view(T, 1, D), dt, p["A"], B, C, None, cut,
                              gn["dx"].view(T, 1, D), D=p["Dk"], dt_bias=p["bias"], states=states)
    dproj = torch.cat([gs["ddt"][:, 0], gs["dB"][:, 0], gs["dC"][:, 0]], 1)
    dc = gs["dx"][:, 0] + dproj @ p["P"].T
    gc = kda.causalconv_backward(xz[:, :D], p["w"], p["b"], None, cut, dc)
    got = dict(xz=torch.cat([gc["dx"], gn["dz"].view(T, D)], 1), w=gc["dw"], b=gc["db"],
               P=c.T @ dproj, A=gs["dA"], Dk=gs["dD"], bias=gs["ddt_bias"], nw=gn["dw"],
               nb=gn["db"])

    q = {k: v.double().requires_grad_() for k, v in p.items()}
    x64 = xz.double().requires_grad_()
    out = _plain(q, x64, D, n, H, cu)
    torch.testing.assert_close(y.double(), out.detach(), rtol=2000 * 2.0 ** -24,
                               atol=2000 * 2.0 ** -24)
    (out * dy.double()).sum().backward()
    for k, v in got.items():
        want = x64.grad if k == "xz" else q[k].grad
        off = (v.double() - want.view_as(v)).abs().max()
        assert off <= 2000 * 2.0 ** -24 * max(1.0, float(want.abs().max())), (k, float(off))


def test_linear_attention_layer():
    """Convolutions of q, k and v (slices of one projection), the matrix-state recurrence, the
    norm of its heads with a sigmoid gate: prompt and steps against the whole."""
    H, d, T, steps = 2, 128, 70, 5
    g = torch.Generator().manual_seed(2)
    rn = lambda *s: torch.randn(*s, generator=g)
    bf = lambda t: t.to(torch.bfloat16).cuda()
    proj, z = bf(rn(T + steps, 3 * H * d)), bf(rn(T + steps, H, d))
    w = (rn(3, H, d, 4) * 0.4).cuda()
    alpha = torch.sigmoid(rn(T + steps, H, d) + 4).cuda()
    beta = torch.sigmoid(rn(T + steps, H)).cuda()
    nw = (1 + 0.2 * rn(d)).cuda()
    cut = lambda L: torch.tensor([0, L], dtype=torch.int32, device="cuda")
    part = lambda t, i: t[:, i * H * d:(i + 1) * H * d].unflatten(1, (H, d))
    unit = lambda t: (t.float() / t.float().norm(dim=-1, keepdim=True)).to(torch.bfloat16)

    def prefill(L):
        conv = [kda.causalconv_prefill(part(proj[:L], i), w[i], None, None, cut(L))
                for i in range(3)]
        q, k, v = (c[0] for c in conv)
        o, S = kda.prefill(unit(q), unit(k), v, alpha[:L].contiguous(), beta[:L].contiguous(),
                           None, cut(L))
        return kda.groupnorm_forward(o, nw, z=z[:L], act="sigmoid"), [c[1] for c in conv], S

    want, _, S_want = prefill(T + steps)
    got, conv, S = prefill(T)
    # one bf16 step of o either way, through a norm that keeps relative errors, and y's own
    tol = 4 * torch.finfo(torch.bfloat16).eps
    torch.testing.assert_close(got.float(), want[:T].float(), rtol=tol, atol=tol)
    for t in range(T, T + steps):
        q, k, v = (kda.causalconv_decode_step(part(proj[t:t + 1], i), w[i], None, conv[i])
                   for i in range(3))
        o = kda.decode_step(unit(q), unit(k), v, alpha[t:t + 1].clone(), beta[t:t + 1].clone(), S)
        y = kda.groupnorm_forward(o, nw, z=z[t:t + 1], act="sigmoid")
        torch.testing.assert_close(y.float(), want[t:t + 1].float(), rtol=tol, atol=tol)
    assert float((S - S_want).norm() / S_want.norm()) < 2e-3


def test_beams_of_a_layer():
    """Steps that read the parents' states are the steps after the states were moved."""
    D, n, H, K = 64, 16, 2, 4
    p, g = _layer(D, n, H, seed=5), torch.Generator().manual_seed(6)
    R = 3 * K
    conv, scan = torch.randn(R, 3, D, generator=g).cuda(), torch.randn(R, 1, D, n, generator=g).cuda()
    xz = torch.randn(R, 2 * D, generator=g).cuda()
    par = (torch.randint(0, K, (3, K), generator=g) + torch.arange(3)[:, None] * K)
    par = par.reshape(-1).to(torch.int32).cuda()
    c2, s2 = torch.empty_like(conv), torch.empty_like(scan)
    c = kda.causalconv_decode_step(xz[:, :D], p["w"], p["b"], conv, parents=par, S_out=c2)
    dt, B, C = _split(c @ p["P"], D, n)
    y = kda.selscan_decode_step(c.view(R, 1, D), dt, p["A"], B, C, scan, D=p["Dk"],
                                dt_bias=p["bias"], parents=par, S_out=s2)
    moved = [conv.clone(), scan.clone()]
    kda.beam_reorder(moved, par, K)
    c1 = kda.causalconv_decode_step(xz[:, :D], p["w"], p["b"], moved[0])
    y1 = kda.selscan_decode_step(c.view(R, 1, D), dt, p["A"], B, C, moved[1], D=p["Dk"],
                                 dt_bias=p["bias"])
    assert torch.equal(c, c1) and torch.equal(y, y1)
    assert torch.equal(c2, moved[0]) and torch.equal(s2, moved[1])


def test_a_captured_step():
    D, n, H, R = 64, 16, 2, 4
    p = _layer(D, n, H, seed=7)
    g = torch.Generator().manual_seed(8)
    xz = torch.randn(R, 2 * D, generator=g).cuda()
    S0 = (torch.randn(R, 3, D, generator=g).cuda(), torch.randn(R, 1, D, n, generator=g).cuda())
    eager = tuple(s.clone() for s in S0)
    ys = [_step(p, xz, D, n, H, eager) for _ in range(3)]
    S, side, graph = tuple(s.clone() for s in S0), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):      # the library of the products sets itself up once
        _step(p, xz, D, n, H, tuple(s.clone() for s in S0))
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        y = _step(p, xz, D, n, H, S)
    for want in ys:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert all(torch.equal(a, b) for a, b in zip(S, eager))
