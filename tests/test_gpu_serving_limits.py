"""Paged attention and the gated delta rule at the stated limits: very many sequences, tokens and cached tokens."""
import numpy as np
import pytest

import chunked_weight_sequence_amd as ttt
from helpers import host_f64, requires_gpu
from test_gpu_attention import _i32

pytestmark = [pytest.mark.gpu, requires_gpu]


def test_paged_as_many_sequences_as_there_may_be():
    """A query with one key gets that key's value, bit for bit; without a key zeros."""
    import torch
    print("case: 2^20 sequences of one new token", flush=True)
    S, Hq, dh, page = 1 << 20, 4, 64, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    pages = 1 << 14
    K, V = (torch.randn((pages * page, 1, dh), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((S, Hq, dh), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randint(0, pages, (S, 1), generator=g, device="cuda").to(torch.int32)
    lens = torch.randint(0, 2, (S,), generator=g, device="cuda").to(torch.int32)
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    O, L = ttt.attention_paged(q, K, V, cu, table, lens, page, with_lse=True)
    want = torch.where(lens[:, None, None] > 0, V[table[:, 0].long() * page], torch.zeros_like(V[:1]))
    assert torch.equal(O, want.expand(S, Hq, dh).contiguous())
    assert torch.equal(torch.isneginf(L), (lens <= 0)[:, None].expand(S, Hq))


def test_paged_very_many_new_tokens():
    """2^23 new tokens of 2^17 sequences of unlike lengths, in pages of their own: equal keys, so a query's result is
    the mean of the values it sees, here of ones and of its sequence's number."""
    import torch
    print("case: 2^23 new tokens", flush=True)
    S, N, dh, page = 1 << 17, 1 << 23, 64, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    new = torch.randint(0, 129, (S,), generator=g, device="cuda")
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)]).clamp(max=N).to(torch.int32)
    new = (cu[1:] - cu[:-1]).long()
    end = int(cu[-1])
    table = (torch.arange(S, device="cuda")[:, None] % 251).expand(S, 8).to(torch.int32).contiguous()
    K = torch.zeros((251 * page, 1, dh), dtype=torch.bfloat16, device="cuda")
    V = torch.ones_like(K)
    V[:, 0, 1] = (torch.arange(251 * page, device="cuda") // page).to(torch.bfloat16)  # whole numbers that bf16 holds
    q = torch.ones((N, 1, dh), dtype=torch.bfloat16, device="cuda")
    O = torch.full_like(q, 7.0)
    _, L = ttt.attention_paged(q, K, V, cu, table, new.to(torch.int32), page, O=O, with_lse=True)
    owner = torch.repeat_interleave(torch.arange(S, device="cuda"), new)
    want = V[(owner % 251) * page]
    assert torch.equal(O[:end], want) and (O[end:] == 7).all()
    seen = torch.arange(end, device="cuda") - cu[:-1].long()[owner] + 1
    assert float((L[:end, 0].double() - seen.double().log()).abs().max()) <= 2.0 ** -18


@pytest.mark.parametrize("Nq,window", [(1, 0), (5, 0), (3, (1 << 29) + 77)])
def test_paged_as_many_tokens_as_a_table_may_hold(Nq, window):
    """2^30 tokens: 16384 pages of 65536, two of them over and over, the last one once. Equal logits: the values'
    mean, and the logarithm of their number; a lane's sums of ones are whole numbers below 2^24."""
    import torch
    print(f"case: 2^30 tokens of one sequence, {Nq} new, window {window}", flush=True)
    page, pages, dh, n = 65536, 1 << 14, 64, 1 << 30
    K = torch.zeros((4 * page, 1, dh), dtype=torch.bfloat16, device="cuda")
    V = torch.ones_like(K)
    V[3 * page:, 0, 2] = 2.0 ** 14
    V[-1, 0, 3] = 2.0 ** 40  # the last token, which the last query alone sees
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None] % 2
    table[0, -1] = 3
    q = torch.ones((Nq, 3, dh), dtype=torch.bfloat16, device="cuda")
    O, L = ttt.attention_paged(q, K, V, _i32([0, Nq]), table.contiguous(), _i32([n]), page, window=window, with_lse=True)
    got = host_f64(O)
    last = n - Nq + np.arange(Nq)
    seen = np.minimum(last + 1, window) if window else last + 1
    assert np.abs(host_f64(L) - np.log(seen)[:, None]).max() <= 2.0 ** -18
    assert np.abs(got[..., 0] - 1).max() <= 2.0 ** -8
    marked = last - (n - page) + 1  # of the last page, all in a window
    want = (seen + marked * (2.0 ** 14 - 1)) / seen
    assert (np.abs(got[..., 2] - want[:, None]) <= 2.0 ** -8 * want[:, None] + 2.0 ** -18).all()
    high = (2.0 ** 40 + seen[-1] - 1) / seen[-1]
    assert (got[:-1, :, 3] == 1).all() and np.abs(got[-1, :, 3] - high).max() <= 1.01 * 2.0 ** -8 * high


def test_delta_as_many_sequences_as_there_may_be():
    """2^20 sequences of one token that start at zero: u = beta v, the state k u^T, o = scale (q . k) u. Both calls.
    Sums of 64 products in fp32, a rounding of u, k u, and of o (twice in the packed call, whose weight of a token
    for itself is in bf16)."""
    import torch
    S, dk, dv = 1 << 20, 64, 64
    g = torch.Generator(device="cuda").manual_seed(7)
    q, k, v = (torch.randn((S, 1, 64), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    beta = torch.rand((S, 1), generator=g, device="cuda")
    gate = -torch.rand((S, 1), generator=g, device="cuda")
    u = beta.double() * v[:, 0].double()
    qk = (q.double() * k.double()).sum(-1)
    size = 0.5 * (q.double() * k.double()).abs().sum(-1) * u.abs()
    out = torch.empty((S, 1, dk, dv), device="cuda")
    cu = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    for packed in (False, True):
        print(f"case: 2^20 sequences of the gated delta rule, packed {packed}", flush=True)
        out.fill_(7.0)
        if packed:
            O, st = ttt.gated_delta_packed(q, k, v, gate, beta, cu, state_out=out, scale=0.5, normalize=False)
        else:
            O, st = ttt.gated_delta_decode(q, k, v, gate, beta, None, state_out=out, scale=0.5, normalize=False)
        want = 0.5 * qk * u
        half = 1.01 * 2.0 ** -8 * (2 if packed else 1)
        assert st is out
        assert ((O[:, 0].double() - want).abs() <= half * want.abs() + 80 * 2.0 ** -24 * size + 1e-37).all()
        for s in range(0, S, 1 << 17):
            part = slice(s, s + (1 << 17))
            w = k[part, 0].float()[:, :, None] * u[part].float()[:, None, :]
            # u rounded twice here and, from three bf16 planes, by at most 2^-24 there; the product's rounding on both sides
            assert ((st[part, 0] - w).abs() <= 8 * 2.0 ** -24 * w.abs() + 1e-37).all()
