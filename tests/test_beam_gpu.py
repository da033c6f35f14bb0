"""Beam search on the GPU against its fp64 oracle: the selection, the moves of the states
and the decode steps that read the parents' states, and a search that runs them together.

Parents and tokens have to be the oracle's exactly; where that needs the candidates to lie
apart, the test checks on the oracle's values that they do.  A value is off by at most one
rounding to fp32 (2^-24 of it) and the error of a 32-bit sum of exponentials: a piece of the
row adds at most 64 terms a thread, each off by 2^-22 and one argument rounding
(40 x 2^-23 for arguments above -40; smaller terms do not show), so its logarithm by at most
(64 + 4 + 80) 2^-24 < 1e-5."""
import numpy as np
import pytest
import torch

from gated_delta_rule_45_gb300 import kda
from oracle import beam as ref
from oracle import linrec as linrec_ref
import oracle

pytestmark = pytest.mark.gpu

SUM_ERR = 148 * 2.0 ** -24
F32_HALF = 2.0 ** -24


def _np(t):
    return t.detach().double().cpu().numpy()


def _check_select(logits, scores, n, finished=None, eos=0, view=None, exact_order=True):
    """logits on the CPU [B K, V]; view: the CUDA tensor to pass (default: a copy)."""
    fin = None if finished is None else finished.numpy()
    vals, par, tok = ref.select(_np(logits), _np(scores), n, fin, eos)
    B, K = scores.shape
    if exact_order:   # neighbours are equal (then ordered by index) or further apart than errors
        every, _, _ = ref.select(_np(logits), _np(scores), min(n + 1, K * logits.shape[1]), fin,
                                 eos)
        with np.errstate(invalid="ignore"):
            gaps = every[:, :-1] - every[:, 1:]
        gaps = gaps[np.isfinite(gaps)]
        assert ((gaps == 0) | (gaps > 2 * SUM_ERR)).all(), "the test's inputs lie too close"
    dev = view if view is not None else logits.cuda()
    s, p, t = kda.beam_select(dev, scores.cuda(), n,
                              finished=None if finished is None else finished.cuda(), eos=eos)
    torch.cuda.synchronize()
    s = _np(s)
    assert np.array_equal(np.isneginf(s), np.isneginf(vals))
    ok = np.isfinite(vals)
    assert (np.abs(s[ok] - vals[ok]) <= SUM_ERR + F32_HALF * np.abs(vals[ok])).all()
    np.testing.assert_array_equal(p.cpu().numpy(), par)
    np.testing.assert_array_equal(t.cpu().numpy(), tok)


def _spread(rows, V, seed, step=1.0 / 64):
    """Logits on a grid: equal ones tie exactly, others lie apart."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, V, generator=g) * 3 / step).round() * step


def _scores(B, K, seed):
    """Odd multiples of 1/200 apart from the grid, so that beams never tie by chance."""
    g = torch.Generator().manual_seed(seed)
    return -20 * torch.rand(B, K, generator=g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,K,V,n", [
    (1, 1, 1, 1), (1, 1, 7, 7), (2, 3, 5, 15), (1, 4, 40, 8), (3, 4, 1000, 8), (2, 8, 4097, 16),
    (5, 2, 33333, 3), (1, 32, 515, 64), (2, 5, 131072, 10), (1, 1, 1 << 20, 64), (64, 4, 63, 5),
])
def test_select(B, K, V, n, dtype):
    logits = torch.randn(B * K, V, generator=torch.Generator().manual_seed(V + n)).to(dtype) * 3
    _check_select(logits, _scores(B, K, V), n)


@pytest.mark.parametrize("K,n", [(4, 8), (8, 16), (32, 64), (1, 64)])
def test_equal_logits_go_to_the_lowest_index(K, n):
    B, V = 2, 70001
    z = torch.zeros(B * K, V)
    same = torch.full((B, K), -3.0)
    _check_select(z, same, n)                       # every candidate equal
    z[:, 1::2] = 1.0
    _check_select(z.bfloat16(), same, n)            # two values only
    _check_select(_spread(B * K, V, K, step=0.5), _scores(B, K, K), n)


def test_descending_rows():
    """The best tokens of a row in one place, at its start, middle and end."""
    V = 50000
    for at in (0, 20011, V - 100):
        z = torch.zeros(4, V)
        z[:, at:at + 100] = torch.arange(100, 0, -1) / 16
        _check_select(z, _scores(1, 4, at), 64)
        z[:, at:at + 100] = torch.arange(1, 101) / 16
        _check_select(z.bfloat16(), _scores(1, 4, at), 64)


def test_masked_and_missing():
    V, K = 9000, 4
    z = torch.full((2 * K, V), -float("inf"))
    z[0, 17], z[0, 8999], z[1, 5] = 1.0, 0.25, 3.0   # three tokens of request 0
    z[5, 100] = 2.0
    sc = torch.tensor([[-1.0, -2.0, -3.0, -4.0], [-1.0, -0.5, -float("inf"), -2.0]])
    _check_select(z, sc, 8)
    _check_select(z.bfloat16(), sc, 8)
    _check_select(torch.full((K, V), -float("inf")), sc[:1], 16)           # nothing is left
    first = torch.tensor([[0.0] + [-float("inf")] * 3])                    # a search's first step
    _check_select(_spread(K, V, 1).repeat(1, 1), first, 8)
    _check_select(_spread(K, 3, 1), first, 12)                             # fewer than asked for


def test_values_that_are_not_finite():
    V, K = 3001, 3
    z = _spread(K, V, 2)
    z[0, ::3] = float("nan")
    z[1, 77] = float("inf")
    z[2] = float("nan")
    sc = torch.tensor([[-1.0, -2.0, float("nan")]])
    for dtype in (torch.float32, torch.bfloat16):
        # a +inf logit takes all of its row: the others of the row are far below
        _check_select(z.to(dtype), sc, 5, exact_order=False)


def test_finished_beams():
    for seed in range(3):
        B, K, V = 6, 4, 5000
        g = torch.Generator().manual_seed(seed)
        fin = (torch.rand(B, K, generator=g) < 0.5).to(torch.uint8)
        fin[0] = 1
        z = torch.randn(B * K, V, generator=g) * 3
        z[fin.reshape(-1).bool()] = float("nan")     # not read
        _check_select(z, _scores(B, K, seed) / 4, 8, finished=fin, eos=4999)
    _check_select(z.bfloat16(), _scores(B, K, seed), 8, finished=fin, eos=0)


def test_padded_vocabulary():
    """Rows wider than the vocabulary: the columns behind it are not read."""
    wide = torch.full((8, 1024), 1e9)
    wide[:, :1001] = _spread(8, 1001, 3)
    for dtype in (torch.float32, torch.bfloat16):
        z = wide.to(dtype)
        _check_select(z[:, :1001].contiguous(), _scores(2, 4, 1), 8, view=z.cuda()[:, :1001])


def test_select_on_another_stream_and_captured():
    z, sc = _spread(8, 32000, 4), _scores(2, 4, 4)
    zd, sd = z.cuda(), sc.cuda()
    want = kda.beam_select(zd, sd, 8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [kda.beam_select(zd, sd, 8, stream=s) for _ in range(4)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = kda.beam_select(zd, sd, 8)
    graph.replay()
    torch.cuda.synchronize()
    for o in (*outs, cap):
        for u, v in zip(o, want):
            assert torch.equal(u, v)


# ---------------------------------------------------------------- reordering

def _parents(B, K, seed, kind="any"):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, K, (B, K), generator=g)
    if kind == "same":
        p = torch.arange(K).repeat(B, 1)
    elif kind == "first":
        p = torch.zeros(B, K, dtype=torch.int64)
    elif kind == "reversed":
        p = torch.arange(K - 1, -1, -1).repeat(B, 1)
    return (p + torch.arange(B)[:, None] * K).to(torch.int32).reshape(-1)


@pytest.mark.parametrize("kind", ["any", "same", "first", "reversed"])
@pytest.mark.parametrize("B,K", [(1, 1), (3, 2), (2, 4), (5, 7), (2, 16), (3, 32)])
def test_reorder(B, K, kind):
    g = torch.Generator().manual_seed(B * K)
    p = _parents(B, K, B + K, kind)
    shapes = [((2, 16, 32), torch.float32), ((5, 67), torch.float32), ((3,), torch.bfloat16),
              ((7,), torch.uint8), ((4, 8, 128), torch.float32), ((1001,), torch.float32),
              ((), torch.int64)]
    states = [(torch.randn(B * K, *s, generator=g) * 100).to(t) for s, t in shapes]
    dev = [t.cuda() for t in states]
    kda.beam_reorder(dev, p.cuda(), K)
    torch.cuda.synchronize()
    for t, d in zip(states, dev):
        want = ref.reorder(t.float().numpy(), p.tolist(), K)
        np.testing.assert_array_equal(d.cpu().float().numpy(), want)


def test_reorder_leaves_rows_with_foreign_parents():
    p = torch.tensor([1, 4, -1, 2, 5, 99, 3, 2 ** 31 - 1], dtype=torch.int32)
    t = torch.arange(8 * 40, dtype=torch.float32).reshape(8, 40)
    d = t.cuda()
    kda.beam_reorder([d], p.cuda(), 4)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(d.cpu().numpy(), ref.reorder(t.numpy(), p.tolist(), 4))


def test_reorder_many_tensors_and_requests():
    g = torch.Generator().manual_seed(1)
    p = _parents(70000, 1, 1)
    t = torch.randn(70000, 3, generator=g)
    d = t.cuda()
    kda.beam_reorder([d], p.cuda(), 1)
    assert torch.equal(d.cpu(), t)
    p = _parents(70000, 2, 2)
    t = torch.randn(140000, 4, generator=g)
    d = t.cuda()
    kda.beam_reorder([d], p.cuda(), 2)
    assert torch.equal(d.cpu(), t[p.long()])
    p = _parents(3, 4, 3)
    many = [torch.randn(12, 5 + i, generator=g) for i in range(150)]
    dev = [t.cuda() for t in many]
    kda.beam_reorder(dev, p.cuda(), 4)
    for t, d in zip(many, dev):
        assert torch.equal(d.cpu(), t[p.long()])


def test_reorder_offsets_beyond_32_bits():
    """8 rows of 0.8 GB: the last rows start past 2^32 bytes."""
    cols = 200_000_003
    t = torch.empty(8, cols, dtype=torch.float32, device="cuda")
    for i in range(8):
        t[i] = i
    t[:, -1] += 100
    kda.beam_reorder([t], _parents(2, 4, 0, "reversed").cuda(), 4)
    torch.cuda.synchronize()
    for i, want in enumerate([3, 2, 1, 0, 7, 6, 5, 4]):
        assert (t[i, :-1] == want).all() and t[i, -1] == want + 100


# ---------------------------------------------------------------- decode from parents

@pytest.mark.parametrize("gate", ["channel", "head", "log_bf16"])
@pytest.mark.parametrize("dtype,dk,dv", [(torch.bfloat16, 128, 128), (torch.float32, 64, 33),
                                         (torch.bfloat16, 256, 70), (torch.float32, 16, 1)])
def test_decode_step_parents(dtype, dk, dv, gate):
    """The same bits as decode_step_gates on the gathered states."""
    B, H, rows = 7, 3, 5
    g = torch.Generator().manual_seed(dk)
    rn = lambda *s: torch.randn(*s, generator=g)
    q, k, v = rn(B, H, dk).to(dtype), rn(B, H, dk).to(dtype) / 8, rn(B, H, dv).to(dtype)
    al = torch.sigmoid(rn(B, H) if gate == "head" else rn(B, H, dv))
    if gate == "log_bf16":
        al = al.log().bfloat16()
    be = torch.sigmoid(rn(B, H))
    table = rn(rows, H, dv, dk)
    p = torch.tensor([0, 4, 4, -1, 2, rows, 4], dtype=torch.int32)
    ok = (p >= 0) & (p < rows)
    S = torch.zeros(B, H, dv, dk)
    S[ok] = table[p[ok].long()]
    dev = [t.cuda() for t in (q, k, v, al, be)]
    S_ref, tab = S.cuda(), table.cuda()
    o_ref = kda.decode_step_gates(*dev, S_ref, gate=gate)
    S_out = torch.full((B, H, dv, dk), float("nan"), device="cuda")
    o = kda.decode_step_parents(*dev, tab, p.cuda(), S_out, gate=gate)
    torch.cuda.synchronize()
    assert torch.equal(o, o_ref) and torch.equal(S_out, S_ref)
    assert torch.equal(tab.cpu(), table)


def test_a_search_over_states():
    """A prompt through a KDA layer and a linear recurrence, then six steps of beam search:
    decode from the parents' states, logits, selection; a third state tensor is moved by
    beam_reorder.  Every step is held to the oracles, which follow the GPU's choices."""
    B, K, H, dk, dv, V, T = 2, 4, 2, 128, 128, 601, 150
    g = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=g)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    emb = {n: rn(V, H, d) for n, d in (("q", dk), ("k", dk), ("v", dv), ("x", dv))}
    emb["q"], emb["k"] = unit(emb["q"]), unit(emb["k"])
    emb["al"], emb["a"] = torch.sigmoid(rn(V, H, dv) + 3), torch.sigmoid(rn(V, H, dv) + 3)
    emb["be"] = torch.sigmoid(rn(V, H))
    head = rn(2 * H * dv, V) * 0.1
    dev = {n: t.cuda() for n, t in emb.items()}
    headd = head.cuda()
    prompt = torch.randint(0, V, (B * T,), generator=g).cuda()
    cu = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda")
    row = lambda n, tok: dev[n][tok].contiguous()
    _, S = kda.prefill(*(row(n, prompt) for n in ("q", "k", "v", "al", "be")), None, cu, chunk=16)
    _, s = kda.linrec_prefill(row("x", prompt), row("a", prompt), None, cu)
    first = torch.arange(B).repeat_interleave(K).to(torch.int32).cuda()
    tokens = torch.randint(0, V, (B * K,), generator=g).cuda()
    scores = torch.zeros(B, K, device="cuda")
    history = torch.zeros(B * K, 9, dtype=torch.int32, device="cuda")
    finished = torch.zeros(B, K, dtype=torch.uint8, device="cuda")
    parents, n_rows = first, B
    for step in range(6):
        S_in, s_in = _np(S), _np(s)
        S2 = torch.empty(B * K, H, dv, dk, device="cuda")
        s2 = torch.empty(B * K, H, dv, device="cuda")
        args = [row(n, tokens) for n in ("q", "k", "v", "al", "be")]
        o = kda.decode_step_parents(*args, S, parents, S2)
        y = kda.linrec_decode_step(row("x", tokens), row("a", tokens), s, parents=parents,
                                   S_out=s2)
        logits = (torch.cat([o, y], -1).reshape(B * K, -1) @ headd).contiguous()
        # oracles, from the states the GPU had
        pl = parents.cpu().numpy()
        f = lambda n: _np(row(n, tokens)).astype(np.float32)
        o_ref, S_ref = oracle.decode_step(f("q"), f("k"), f("v"), f("al"), f("be"), S_in[pl])
        assert np.linalg.norm(_np(o) - o_ref) <= 1e-5 * np.linalg.norm(o_ref)
        assert np.linalg.norm(_np(S2) - S_ref) <= 1e-5 * np.linalg.norm(S_ref)
        one = list(range(B * K + 1))
        a, x = _np(row("a", tokens)), _np(row("x", tokens))
        h, _ = linrec_ref.forward(x, a, s_in[pl], one)
        _, e, _ = linrec_ref.forward_bound(x, a, s_in[pl], one, False, 2)
        assert (np.abs(_np(s2) - h) <= e).all()
        vals, par, tok = ref.select(_np(logits), _np(scores), K, finished.cpu().numpy(), eos=1)
        scores, parents2, tok2 = kda.beam_select(logits, scores, K, finished=finished, eos=1)
        np.testing.assert_array_equal(parents2.cpu().numpy(), par)
        np.testing.assert_array_equal(tok2.cpu().numpy(), tok)
        assert (np.abs(_np(scores) - vals) <= SUM_ERR + F32_HALF * np.abs(vals)).all()
        # the beams' histories and finished marks move in place
        before = history.cpu().numpy().copy()
        fin_before = finished.cpu().numpy().reshape(-1).copy()
        fin = finished.reshape(-1, 1).contiguous()
        parents, tokens = parents2.reshape(-1), tok2.reshape(-1).long()
        kda.beam_reorder([history, fin], parents, K)
        np.testing.assert_array_equal(history.cpu().numpy(),
                                      ref.reorder(before, parents.tolist(), K))
        np.testing.assert_array_equal(fin.cpu().numpy()[:, 0],
                                      ref.reorder(fin_before, parents.tolist(), K))
        history[:, step] = tokens.to(torch.int32)
        finished = (fin.reshape(B, K) | (tokens.reshape(B, K) == 1)).to(torch.uint8)
        S, s = S2, s2
    assert torch.isfinite(scores).all()
