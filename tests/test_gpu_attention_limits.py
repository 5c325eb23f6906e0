"""Norm and rotation, packed and one-token attention at the stated limits: sizes of heads whose squares
leave fp32, very many sequences and tokens."""
import numpy as np
import pytest

import chunked_weight_sequence_amd as ttt
import gen
import oracle.attention as oa
from helpers import dev, host_f64, requires_gpu
from test_gpu_attention import _check, _cu, _draw, _f, _i32, _logit_size, _packed

pytestmark = [pytest.mark.gpu, requires_gpu]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,by,eps", [(128, 1e25, 1e-6), (128, 2.0 ** 127, 1e-6), (80, 1e19, 0.0), (64, 1e-25, 0.0),
                                       (256, 1e-36, 0.0), (64, 1e-22, 1e-40), (64, 1e-25, 1e-6)])
def test_norms_of_very_large_and_small_heads(dtype, dh, by, eps):
    """x / sqrt(mean(x^2) + eps) is of ordinary size wherever x lies in its type's range. Bound: the sum's
    dh / 2 half steps and 16 more for the root, the products and a scaling, then the output's rounding."""
    import torch
    print(f"case: norm of heads of size {by} {dtype} dh={dh} eps={eps}", flush=True)
    rng = np.random.default_rng(dh)
    x = (by * rng.uniform(-1, 1, (5, 3, dh))).astype(np.float32)
    x[1, 1] /= 1e12 if by > 1 else 1  # an ordinary head among them, in the same waves
    x[2, 0] = 1.5
    if dtype == "bf16":
        x = gen.f32_to_bf16_bits(x)
    w = rng.uniform(0.5, 1.5, dh).astype(np.float32)
    X = _f(x) if dtype == "bf16" else x.astype(np.float64)
    e = float(np.float32(eps))
    Q, _ = ttt.qk_norm_rope(dev(x, dtype), dev(x, dtype), _i32([0] * 5),
                            torch.zeros(0, dtype=torch.float64, device="cuda"), q_weight=dev(w, "f32"),
                            eps=eps)
    torch.cuda.synchronize()
    want = oa.norm_rope(X, w, e, [0] * 5, np.zeros(0), "half", 1.0)
    bound = ((dh / 2 + 16) * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)) * np.abs(want) + 2e-38
    off = np.abs(host_f64(Q) - want) / bound
    print(f"  {off.max():.3f} of the bound", flush=True)
    assert np.isfinite(host_f64(Q)).all() and off.max() <= 1.0


@pytest.mark.parametrize("n", [64, 4097, 5000])
def test_packed_thousands_of_sequences(n):
    print(f"case: {n} sequences", flush=True)
    rng = np.random.default_rng(n)
    lq = rng.integers(0, 4, n)
    more = rng.integers(-1, 5, n)
    lk = np.maximum(lq + more, 0)
    cu_q, cu_k = _cu(lq), _cu(lk)
    Q = _draw(rng, max(cu_q[-1], 1), 2, 64)
    K, V = _draw(rng, max(cu_k[-1], 1), 1, 64), _draw(rng, max(cu_k[-1], 1), 1, 64)
    O, L = _packed(Q, K, V, cu_q, cu_k, 0.2, 0)
    _check(O, L, oa.packed(_f(Q), _f(K), _f(V), cu_q, cu_k, 0.2), _logit_size(_f(Q), _f(K), 0.2), 64, "many")


@pytest.mark.parametrize("n,dh", [(300001, 64), (1 << 20, 64), (70000, 128)])
def test_packed_sequences_of_one_token_return_their_values(n, dh):
    """Up to 2^20 sequences, the most there may be: a query with one key gets that key's value, bit for bit,
    and its logit."""
    import torch
    print(f"case: {n} sequences of one token, dh {dh}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    q, k, v = (torch.randn((n, 1, dh), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    O, L = ttt.attention_packed(q, k, v, cu, scale=0.5, with_lse=True)
    assert torch.equal(O, v)
    x = 0.5 * (q.double() * k.double()).sum(-1)
    X = 0.5 * (q.double() * k.double()).abs().sum(-1)
    assert ((L - x).abs() <= (dh + 8) * 2.0 ** -24 * X + 2.0 ** -20).all()


def test_packed_as_many_tokens_as_there_may_be():
    """2^26 tokens in 2^20 sequences of unlike lengths, in which every key of a sequence is the same: a query's
    result is the mean of the values it sees, here of ones and of its sequence's number."""
    import torch
    print("case: 2^26 tokens", flush=True)
    n, N, dh = 1 << 20, 1 << 26, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    cuts = torch.randint(0, N + 1, (n - 1,), generator=g, device="cuda").sort().values
    cu = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), N)]).to(torch.int32)
    owner = torch.bucketize(torch.arange(N, device="cuda"), cu[1:].long(), right=True)
    q = torch.ones((N, 1, dh), dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros_like(q), torch.ones_like(q)
    v[:, 0, 1] = (owner % 251).to(torch.bfloat16)  # whole numbers that bf16 holds
    O, L = ttt.attention_packed(q, k, v, cu, with_lse=True)
    assert torch.equal(O, v)
    seen = torch.arange(N, device="cuda") - cu[:-1].long()[owner] + 1
    assert float((L[:, 0].double() - seen.double().log()).abs().max()) <= 2.0 ** -18


def test_decode_as_many_sequences_as_there_may_be():
    import torch
    print("case: 2^20 sequences of one token", flush=True)
    S, Hq, dh, page = 1 << 20, 8, 64, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    pages = 1 << 14
    K, V = (torch.randn((pages * page, 1, dh), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((S, Hq, dh), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randint(0, pages, (S, 1), generator=g, device="cuda").to(torch.int32)
    lens = torch.randint(0, 2, (S,), generator=g, device="cuda").to(torch.int32)
    O, L = ttt.attention_decode(q, K, V, table, lens, page, with_lse=True)
    want = torch.where(lens[:, None, None] > 0, V[table[:, 0].long() * page], torch.zeros_like(V[:1]))
    assert torch.equal(O, want.expand(S, Hq, dh).contiguous())
    assert torch.equal(torch.isneginf(L), (lens <= 0)[:, None].expand(S, Hq))


def test_rotation_of_as_many_tokens_as_there_may_be():
    """2^25 tokens: a quarter turn more each, so the pair (1, 0) goes through four places."""
    import torch
    print("case: 2^25 tokens of norm and rotation", flush=True)
    N, dh = 1 << 25, 16
    x = torch.zeros((N, 1, dh), dtype=torch.bfloat16, device="cuda")
    x[:, 0, :8] = 1
    freq = torch.full((8,), np.pi / 2, dtype=torch.float64, device="cuda")
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    Q, K = ttt.qk_norm_rope(x, x, pos, freq)
    turn = torch.tensor([[1, 0], [0, 1], [-1, 0], [0, -1]], dtype=torch.float32, device="cuda")[pos % 4]
    for y in (Q, K):
        got = y[:, 0].float()
        assert float((got[:, 0] - turn[:, 0]).abs().max()) <= 2.0 ** -20
        assert float((got[:, 8] - turn[:, 1]).abs().max()) <= 2.0 ** -20
        assert torch.equal(got[:, :1].expand(N, 8), got[:, :8]) and torch.equal(got[:, 8:9].expand(N, 8), got[:, 8:])


@pytest.mark.parametrize("Nq,window", [(1, 0), (130, 0), (3, (1 << 26) - 77)])
def test_packed_as_many_keys_as_there_may_be(Nq, window):
    """2^26 keys of one logit: the values' mean, and the logarithm of their number. Each piece's sums are exact
    (weights of 1), the halves of channel 1 cancel."""
    import torch
    print(f"case: {Nq} queries, 2^26 keys, window {window}", flush=True)
    Nk, dh = 1 << 26, 64
    q = torch.ones((Nq, 2, dh), dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros((Nk, 1, dh), dtype=torch.bfloat16, device="cuda"), torch.ones(
        (Nk, 1, dh), dtype=torch.bfloat16, device="cuda")
    v[: Nk // 2, 0, 1] = -1
    v[-1, 0, 2] = 2.0 ** 26  # the last key's value is seen by the last query alone
    O, L = ttt.attention_packed(q, k, v, _i32([0, Nq]), _i32([0, Nk]), window=window, with_lse=True)
    last = Nk - Nq + np.arange(Nq)
    seen = np.minimum(last + 1, window) if window else last + 1
    assert np.abs(host_f64(L) - np.log(seen)[:, None]).max() <= 2.0 ** -18
    got = host_f64(O)
    first = last + 1 - seen
    one = (seen - 2 * np.maximum(Nk // 2 - first, 0)) / seen
    assert np.abs(got[..., 0] - 1).max() <= 2.0 ** -8
    assert np.abs(got[..., 1] - one[:, None]).max() <= 2.0 ** -8 * np.abs(one).max() + 2.0 ** -20
    assert (got[:-1, :, 2] == 1).all() and np.abs(got[-1, :, 2] - 2).max() <= 2.0 ** -6


def test_decode_as_many_tokens_as_a_table_may_hold():
    """2^30 tokens: 16384 pages of 65536, three of them over and over, the last one once. Equal logits; each
    wave's sums of ones are whole numbers below 2^24."""
    import torch
    print("case: 2^30 tokens of one sequence", flush=True)
    page, pages, dh = 65536, 1 << 14, 64
    K = torch.zeros((4 * page, 1, dh), dtype=torch.bfloat16, device="cuda")
    V = torch.ones_like(K)
    V[page:2 * page, 0, 1] = -1
    V[3 * page:, 0, 2] = 2.0 ** 14
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None] % 2
    table[0, -1] = 3
    q = torch.ones((1, 3, dh), dtype=torch.bfloat16, device="cuda")
    O, L = ttt.attention_decode(q, K, V, table.contiguous(), _i32([1 << 30]), page, with_lse=True)
    got = host_f64(O)[0]
    assert np.abs(host_f64(L) - np.log(2.0 ** 30)).max() <= 2.0 ** -18
    assert np.abs(got[:, 0] - 1).max() <= 2.0 ** -8 and np.abs(got[:, 1] - 2.0 ** -13).max() <= 2.0 ** -20
    assert np.abs(got[:, 2] - (2.0 - 2.0 ** -14)).max() <= 2.0 ** -6
