"""The state operators where offsets pass 32 bits: the last sequence and the last requests of
a batch of more than 2^32 elements come out as they do alone."""
import pytest
import torch

from gated_delta_rule_45_gb300 import kda

pytestmark = pytest.mark.gpu


def test_linrec_beyond_32_bits():
    """Its first token lies on a tile's border, so that the same bits are expected."""
    H, d, last = 32, 128, 5120
    first = (1 << 32) // (H * d) + 256 * 11
    T = first + last
    assert first % 256 == 0 and T * H * d > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(T, H, d, device="cuda", dtype=torch.bfloat16, generator=g)
    la = torch.randn(T, H, d, device="cuda", dtype=torch.bfloat16, generator=g).abs_().mul_(-0.05)
    S0 = torch.randn(2, H, d, device="cuda", generator=g)
    cu = torch.tensor([0, first, T], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, last], dtype=torch.int32, device="cuda")
    y, S_T, st = kda.linrec_prefill(x, la, S0, cu, gate="log_bf16", save_states=True,
                                    check_device_status=True)
    tail = [t[first:].contiguous() for t in (x, la)]
    y1, S1, st1 = kda.linrec_prefill(*tail, S0[1:].contiguous(), one, gate="log_bf16",
                                     save_states=True)
    assert torch.equal(y[first:], y1) and torch.equal(S_T[1:], S1)
    assert torch.equal(st[first // kda.LINREC_CHUNK:], st1)
    # gradients, x standing in for dy
    gr = kda.linrec_backward(x, la, S0, cu, x, S0, states=st, gate="log_bf16",
                             check_device_status=True)
    g1 = kda.linrec_backward(*tail, S0[1:].contiguous(), one, tail[0], S0[1:].contiguous(),
                             states=st1, gate="log_bf16")
    for k in ("dx", "dgate"):
        assert torch.equal(gr[k][first:], g1[k])
    assert torch.equal(gr["dS0"][1:], g1["dS0"])


def test_linrec_decode_beyond_32_bits():
    B, H, d = 40000, 64, 2048
    assert B * H * d > 1 << 32
    S = torch.zeros(B, H, d, device="cuda")
    x = torch.ones(B, H, d, device="cuda", dtype=torch.bfloat16)
    a = torch.full((B, H), 0.5, device="cuda")
    S[-1], x[-1], a[-1] = 2.0, 3.0, 0.25
    y = kda.linrec_decode_step(x, a, S, gate="head")
    assert (S[:-1] == 1).all() and (y[:-1] == 1).all()
    assert (S[-1] == 3.5).all() and (y[-1] == 3.5).all()


def test_selection_beyond_32_bits():
    K, V, B = 8, 128000, 4300
    assert B * K * V > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(0)
    z = torch.randn(B * K, V, device="cuda", dtype=torch.bfloat16, generator=g).mul_(3)
    sc = -torch.rand(B, K, device="cuda", generator=g)
    s, p, t = kda.beam_select(z, sc, 8)
    for b in (0, 2095, B - 1):
        s1, p1, t1 = kda.beam_select(z[b * K:(b + 1) * K].contiguous(), sc[b:b + 1].contiguous(), 8)
        # another number of pieces: the sums are rounded otherwise (1e-6 at most each)
        torch.testing.assert_close(s[b:b + 1], s1, rtol=0, atol=4e-6)
        assert torch.equal(p[b:b + 1], p1 + b * K) and torch.equal(t[b:b + 1], t1)
