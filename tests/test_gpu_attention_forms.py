"""Each form of the packed and one-token kernels and of the joining of pieces against the fp64 oracle, at
sizes that are held to take it (test_attention_plan.py). Tolerances as in test_gpu_attention.py. O and lse
begin as 7 everywhere, so that a row that is not written shows."""
import numpy as np
import pytest

import chunked_weight_sequence_amd as ttt
import gen
import oracle.attention as oa
from attention_forms import DECODE, PACKED
from helpers import dev, host_f64, requires_gpu
from test_gpu_attention import _check, _cu, _draw, _f, _i32, _logit_size, _packed, _some_rows

pytestmark = [pytest.mark.gpu, requires_gpu]


def _sevens(*shape):
    import torch
    return (torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda"),
            torch.full(shape[:2], 7.0, device="cuda"))


@pytest.mark.parametrize("hidden", [False, True], ids=["", "hidden"])
@pytest.mark.parametrize("case,form", PACKED, ids=[str(i) for i in range(len(PACKED))])
def test_packed_form(case, form, hidden):
    """With `hidden`, a key in the middle of the first sequence's own part has an infinite value in two
    channels: rows that see it get that infinity there, the others what they get without."""
    lq, more, Hq, Hkv, dh, window = case
    print(f"case: packed form {form} lq={lq} more={more} {Hq}/{Hkv}x{dh} window={window} "
          f"hidden={hidden}", flush=True)
    rng = np.random.default_rng(sum(lq) + dh + window)
    # three rows before the first sequence and two behind the last, which stay; the sizes of the call grow
    # by so little that the form is the same (test_attention_plan.py)
    front, back = 3, 2
    cu_q, cu_k = _cu(lq, front), _cu(np.array(lq) + np.array(more))
    Nq = int(cu_q[-1]) + back
    Q = _draw(rng, Nq, Hq, dh)
    K, V = _draw(rng, cu_k[-1], Hkv, dh), _draw(rng, cu_k[-1], Hkv, dh)
    scale = 1.1 * dh ** -0.5
    at = int(cu_k[1]) - lq[0] // 2 - 1
    v, V1 = _f(V), V.copy()
    if hidden:
        V1[at, 0, [5, dh - 1]] = gen.f32_to_bf16_bits(np.float32([-np.inf]))[0]
    O, L = _sevens(Nq, Hq, dh)
    _packed(Q, K, V1, cu_q, cu_k, scale, window, O=O, lse=L)
    for x in (O[:front], O[-back:], L[:front], L[-back:]):
        assert (x == 7).all()
    near = [front + x for x in range(min(lq[0], 40))] + [front + lq[0] - 1, front + lq[0] // 2]
    tokens = sorted({*near, Nq - back - 1, *rng.integers(front, Nq - back, 20).tolist()})
    heads = sorted({0, Hq // Hkv - 1, Hq - 1, *rng.integers(0, Hq, 2).tolist()})
    q, k = _f(Q), _f(K)
    o, lse, a = _some_rows(q, k, v, cu_q, cu_k, scale, window, tokens, heads)
    got = O[tokens][:, heads].clone()
    if hidden:
        for i, t in enumerate(tokens):
            last = t - front + more[0]
            if t >= front + lq[0] or not (last - window < at if window else True) or at > last:
                continue
            for j, h in enumerate(heads):
                if h < Hq // Hkv:
                    assert np.isneginf(host_f64(got[i, j, [5, dh - 1]])).all(), (t, h)
                    got[i, j, [5, dh - 1]], o[i, j, [5, dh - 1]] = 0, 0
    _check(got, L[tokens][:, heads], (o, lse, a), _logit_size(q[tokens], k, scale)[:, heads], dh, "form")
    # every row of a sequence: written, and within the convex hull of V where the values are finite
    all_ = host_f64(O[front:-back])
    if hidden:
        assert not np.isnan(all_).any()
        all_ = np.where(np.isneginf(all_), 0, all_)
    assert np.abs(all_).max() <= np.abs(v).max() * (1 + 2.0 ** -6)
    assert not (all_ == 7).all(-1).any() and not (L[front:-back] == 7).any()


@pytest.mark.parametrize("case,form", DECODE, ids=[str(i) for i in range(len(DECODE))])
def test_decode_form(case, form):
    """Sequences share the pages of one cache; what no sequence sees is NaN."""
    import torch
    lens, pages, page, Hq, Hkv, dh, window = case
    print(f"case: decode form {form} lens={lens[:6]} page={page} {Hq}/{Hkv}x{dh} window={window}",
          flush=True)
    rng = np.random.default_rng(sum(lens) + dh + window)
    S, G, scale, longest = len(lens), Hq // Hkv, 1.1 * dh ** -0.5, max(lens)
    held = -(-longest // page)
    order = rng.permutation(held + 2)
    Kc = np.full(((held + 2) * page, Hkv, dh), 0x7FC0, np.uint16)
    Vc = np.full_like(Kc, 0x7FC0)
    table = np.full((S, pages), -1, np.int32)
    firsts = [max(0, n - window) if window else 0 for n in lens]
    rows = np.array([order[j // page] * page + j % page for j in range(longest)])
    seen = sorted({j for f, n in zip(firsts, lens) for j in (f, n - 1) if n} | set(range(
        min([f for f, n in zip(firsts, lens) if n]), longest)))
    Kc[rows[seen]], Vc[rows[seen]] = _draw(rng, len(seen), Hkv, dh), _draw(rng, len(seen), Hkv, dh)
    for s, n in enumerate(lens):
        table[s, :-(-n // page)] = order[:-(-n // page)]
    Q = _draw(rng, S, Hq, dh)
    O, L = _sevens(S, Hq, dh)
    ttt.attention_decode(dev(Q, "bf16"), dev(Kc, "bf16"), dev(Vc, "bf16"), _i32(table), _i32(lens), page,
                         scale=scale, window=window, O=O, lse=L)
    torch.cuda.synchronize()
    some = sorted({*range(min(S, 6)), S - 1, *rng.integers(0, S, 4).tolist()})
    heads = sorted({0, G - 1, Hq - 1, Hq // 2, *rng.integers(0, Hq, 4).tolist()})
    k, v, q = _f(Kc[rows]), _f(Vc[rows]), _f(Q)
    res = [oa.attend(q[s, h], k[firsts[s]:lens[s], h // G], v[firsts[s]:lens[s], h // G], scale)
           for s in some for h in heads]
    want = [np.array([x[i] for x in res]).reshape(len(some), len(heads), *np.shape(res[0][i]))
            for i in range(3)]
    X = scale * np.abs(q[some][:, heads]).sum(-1) * np.nanmax(np.abs(k))
    _check(O[some][:, heads], L[some][:, heads], want, X, dh, "form")
    all_ = host_f64(O)
    assert np.isfinite(all_).all() and np.abs(all_).max() <= np.nanmax(np.abs(v)) * (1 + 2.0 ** -6)
    assert not (all_ == 7).all(-1).any() and not (L == 7).any()
