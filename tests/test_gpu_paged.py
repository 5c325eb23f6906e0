"""GPU parity of ttt_attention_paged against the fp64 oracle; tolerances as in test_gpu_attention.py."""
import numpy as np
import pytest

import chunked_weight_sequence_amd as ttt
import oracle.serving as osv
from helpers import dev, host_bits, host_f64, requires_gpu
from test_gpu_attention import _check, _draw, _f, _i32, _logit_size

pytestmark = [pytest.mark.gpu, requires_gpu]

NAN = 0x7FC0


def _pool(rng, lens, page, Hkv, dh, spare=2, most=None):
    """A cache whose pages lie in any order: bits of K and V, and the page table. Whatever no sequence holds
    is NaN, entries of the table behind a sequence's last page are no pages."""
    held = [-(-max(n, 0) // page) for n in lens]
    n_pages = sum(held) + spare
    most = max(1, max(held)) if most is None else most
    order = rng.permutation(n_pages).astype(np.int32)
    table = rng.choice([-1, n_pages, 1 << 30, -(1 << 31)], (len(lens), most)).astype(np.int32)
    K, V = (np.full((n_pages * page, Hkv, dh), NAN, np.uint16) for _ in range(2))
    at = 0
    for s, n in enumerate(lens):
        table[s, :held[s]] = order[at:at + held[s]]
        at += held[s]
        for j0 in range(0, max(n, 0), page):
            r, m = int(table[s, j0 // page]) * page, min(page, n - j0)
            K[r:r + m], V[r:r + m] = _draw(rng, m, Hkv, dh), _draw(rng, m, Hkv, dh)
    return K, V, table


def _run(rng, new, lens, page, Hq, Hkv, dh, window=0, some=None, first=0, behind=0, scale=None, kv=None):
    """Calls the operator on len(new) sequences and checks every row, or `some` of them."""
    import torch
    K, V, table = kv or _pool(rng, lens, page, Hkv, dh)
    cu = np.concatenate([[first], first + np.cumsum(new)]).astype(np.int32)
    N = int(cu[-1]) + behind
    Q = _draw(rng, N, Hq, dh)
    O = torch.full((N, Hq, dh), 7.0, dtype=torch.bfloat16, device="cuda")
    L = torch.full((N, Hq), 7.0, device="cuda")
    ttt.attention_paged(dev(Q, "bf16"), dev(K, "bf16"), dev(V, "bf16"), _i32(cu), _i32(table), _i32(lens), page,
                        window=window, scale=scale, O=O, lse=L)
    torch.cuda.synchronize()
    mine = np.arange(int(cu[0]), int(cu[-1]))
    rest = np.setdiff1d(np.arange(N), mine)
    assert (host_f64(O)[rest] == 7).all() and (host_f64(L)[rest] == 7).all()
    if some is not None:
        mine = np.unique(np.concatenate([rng.choice(mine, min(some, len(mine)), replace=False), mine[:2], mine[-2:]]))
    if not len(mine):
        return O, L
    sc = dh ** -0.5 if scale is None else scale
    o, lse, a = osv.paged(_f(Q), _f(K), _f(V), cu, table, lens, page, sc, window, set(mine.tolist()))
    X = _logit_size(_f(Q)[mine], np.nan_to_num(_f(K)), sc)
    _check(O[mine], L[mine], (o[mine], lse[mine], a[mine]), X, dh, f"{len(mine)} rows")
    return O, L


@pytest.mark.parametrize("Hq,Hkv,dh", [(8, 2, 128), (4, 4, 64), (6, 1, 64), (7, 1, 128), (40, 1, 64), (160, 1, 128), (2, 2, 128)])
@pytest.mark.parametrize("page", [16, 32, 64, 256])
def test_sizes(Hq, Hkv, dh, page):
    """Several sequences: a piece after others, a whole prompt, single tokens, nothing new, nothing at all, more
    queries than tokens, lengths at and beside the pages' and tiles' ends."""
    print(f"case: paged {Hq}/{Hkv}x{dh} page {page}", flush=True)
    rng = np.random.default_rng(Hq + dh + page)
    new = [5, 33, 1, 0, 0, 4, 1, 20, 3]
    lens = [77, 33, 64, 50, 0, 0, 1, 16, 129]
    _run(rng, new, lens, page, Hq, Hkv, dh, first=2, behind=3)


@pytest.mark.parametrize("window", [1, 16, 60, 64, 100, 1 << 30])
@pytest.mark.parametrize("Hq,Hkv,dh", [(8, 2, 128), (4, 4, 64)])
def test_windows(Hq, Hkv, dh, window):
    print(f"case: paged {Hq}/{Hkv}x{dh} window {window}", flush=True)
    rng = np.random.default_rng(window % 1000 + dh)
    _run(rng, [70, 1, 130, 9], [300, 200, 131, 9], 32, Hq, Hkv, dh, window=window)


@pytest.mark.parametrize("new,lens,page,Hq,Hkv,dh,window", [
    ([1], [1], 16, 1, 1, 64, 0), ([1], [4000], 16, 8, 1, 128, 0), ([3], [5000], 64, 16, 4, 64, 0),
    ([64], [6000], 32, 8, 2, 128, 0), ([512], [9000], 64, 32, 8, 128, 0), ([700, 1], [3000, 2500], 16, 16, 4, 64, 0),
    ([1100], [5000], 256, 32, 8, 128, 0), ([600], [5000], 64, 16, 16, 64, 700), ([2100], [2100], 64, 32, 8, 128, 0),
    ([300] + [1] * 20, [4000] + [100 * i + 1 for i in range(20)], 16, 16, 4, 128, 0),
    ([5] * 16, [500 * i + 5 for i in range(16)], 16, 16, 4, 64, 0), ([2, 1] * 50, [40, 30] * 50, 16, 8, 2, 128, 0),
    ([1] * 70, [20] * 70, 16, 4, 4, 64, 0), ([0, 0], [100, 50], 16, 8, 2, 128, 0),
    ([400, 139, 500, 300, 200], [2560, 1000, 500, 2300, 2559], 16, 32, 8, 128, 0), ([1] * 15, [97 * i for i in range(15)], 32, 32, 8, 128, 0)])
def test_long_and_many(new, lens, page, Hq, Hkv, dh, window):
    """The forms of the kernels: rows by 128 and by 256, keys split over workgroups, many sequences."""
    print(f"case: paged long {new[:4]} {lens[:4]} {Hq}/{Hkv}x{dh} page {page}", flush=True)
    rng = np.random.default_rng(sum(new) + sum(lens))
    _run(rng, new, lens, page, Hq, Hkv, dh, window=window, some=40, behind=1 if not sum(new) else 0)


@pytest.mark.parametrize("new,lens,Hq,Hkv", [
    ([200, 9, 200], [4256, 900, 4100], 32, 4), ([1000, 224], [6560, 224], 8, 2), ([260, 260], [8000, 3900], 32, 8),
    ([512] + [1] * 13, [6000] + [431 * i for i in range(13)], 32, 8)])
def test_several_sequences_in_pieces(new, lens, Hq, Hkv):
    """Rows by 256, then by 128, of several sequences whose keys are split over workgroups (test_paged_plan.py has which
    sizes take which), the last one with the sequences in the order of their lengths."""
    print(f"case: paged, several in pieces, {new[:3]} {lens[:3]} {Hq}/{Hkv}", flush=True)
    rng = np.random.default_rng(sum(new) + sum(lens))
    _run(rng, new, lens, 16, Hq, Hkv, 128, some=60, first=1, behind=2)


@pytest.mark.parametrize("new,n,room,Hq,Hkv", [(1, 33000, 33000, 32, 8), (5, 50000, 50000, 16, 4), (32, 700, 131072, 32, 8), (40, 1, 70000, 8, 2), (33, 33000, 33000, 16, 4)])
def test_one_sequence_on_a_long_table(new, n, room, Hq, Hkv):
    """A few tokens on many keys, and on few keys of a table that has room for many."""
    print(f"case: paged, {new} tokens on {n} of {room}, {Hq}/{Hkv}", flush=True)
    rng = np.random.default_rng(new + n)
    kv = _pool(rng, [n], 64, Hkv, 128, most=-(-room // 64))
    _run(rng, [new], [n], 64, Hq, Hkv, 128, kv=kv, some=8)


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("n", [100, 3000])
def test_pages_that_are_not_there(n, dh):
    """Tokens of a page outside the cache are left out, wherever they lie; a row that sees only such tokens sees
    nothing; lengths past the table are cut, negative ones hold nothing. What the first page holds is NaN."""
    print(f"case: paged, missing pages, {n} {dh}", flush=True)
    rng = np.random.default_rng(n + dh)
    page, Hkv = 16, 2
    lens = [n, 48, n]
    K, V, table = _pool(rng, lens, page, Hkv, dh, spare=3)
    order = rng.permutation(len(K) // page)
    away = np.argmax(order)  # the first page to the last place, so that no sequence has it
    swap = {0: int(order[away]), int(order[away]): 0}
    K0, V0, t0 = K.copy(), V.copy(), table.copy()
    for p, q in swap.items():
        K[q * page:(q + 1) * page], V[q * page:(q + 1) * page] = (x[p * page:(p + 1) * page] for x in (K0, V0))
        table[t0 == p] = q
    for s, holes in ((0, [1, 2, n // 32, (n - 1) // page]), (1, [0, 1, 2]), (2, [0, 1, 3])):
        table[s, holes] = rng.choice([-1, len(K) // page, 1 << 29], len(holes))
    K[:page], V[:page] = NAN, NAN
    table[(table == 0)] = -1
    _run(rng, [40, 5, 7], lens, page, 8, Hkv, dh, kv=(K, V, table), some=30)
    long = [table.shape[1] * page + 1000, -5, 1 << 30]
    full = [table.shape[1] * page, 0, table.shape[1] * page]
    Q = _draw(rng, 12, 8, dh)
    a = [dev(Q, "bf16"), dev(K, "bf16"), dev(V, "bf16"), _i32([0, 4, 8, 12]), _i32(table)]
    got = ttt.attention_paged(*a, _i32(long), page, with_lse=True)
    cut = ttt.attention_paged(*a, _i32(full), page, with_lse=True)
    np.testing.assert_array_equal(host_bits(got[0]), host_bits(cut[0]))
    np.testing.assert_array_equal(host_bits(got[1]), host_bits(cut[1]))
    assert np.isneginf(host_f64(got[1])[4:8]).all() and (host_f64(got[0])[4:8] == 0).all()


@pytest.mark.parametrize("dh", [64, 128])
def test_infinities_and_nan_that_are_not_seen(dh):
    """Values of later tokens and before the window, in pages that the rows do see others of; and a value that
    is seen."""
    import torch
    print(f"case: paged, values not seen, {dh}", flush=True)
    rng = np.random.default_rng(dh)
    page, Hkv, Hq, n, new, window = 32, 2, 4, 400, 50, 100
    K, V, table = _pool(rng, [n], page, Hkv, dh)
    row = lambda j: int(table[0, j // page]) * page + j % page  # noqa: E731
    V[row(390), 0, 5], V[row(395), 1, 40], K[row(398), 0, 3] = 0x7F80, NAN, NAN
    V[row(240), 0, 60], K[row(230), 1] = 0xFF80, NAN
    Q = _draw(rng, new, Hq, dh)
    cu = [0, new]
    O, L = ttt.attention_paged(dev(Q, "bf16"), dev(K, "bf16"), dev(V, "bf16"), _i32(cu), _i32(table), _i32([n]), page,
                               window=window, with_lse=True)
    torch.cuda.synchronize()
    o, lse, a = osv.paged(_f(Q), _f(K), _f(V), cu, table, [n], page, dh ** -0.5, window)
    seen = np.isfinite(a) & np.isfinite(lse)[..., None]
    assert seen.mean() > 0.9 and not seen.all()
    got = host_f64(O)
    assert np.isfinite(got[seen]).all()
    X = _logit_size(_f(Q), np.nan_to_num(_f(K)), dh ** -0.5)
    d = (dh + 4) * 2.0 ** -24 * X[..., None]
    bound = 1.01 * (2.0 ** -8 * (np.abs(o) + a) + (4 * d + 2.0 ** -19) * a) + 1e-38
    assert (np.abs(got - o)[seen] <= bound[seen]).all()
    assert not np.isfinite(got[40:, 0, 5]).any() and np.isnan(got[45:, 2, 40]).all()


def test_one_token_and_whole_prompts_agree_with_the_other_calls():
    """Single tokens: attention_decode's result; a prompt in pages that lie in order: attention_packed's."""
    import torch
    print("case: paged against the other calls", flush=True)
    rng = np.random.default_rng(9)
    page, Hq, Hkv, dh = 64, 8, 2, 128
    lens = [200, 1, 64, 77]
    K, V, table = _pool(rng, lens, page, Hkv, dh)
    Q = dev(_draw(rng, 4, Hq, dh), "bf16")
    a = [dev(K, "bf16"), dev(V, "bf16")]
    one = ttt.attention_paged(Q, *a, _i32(range(5)), _i32(table), _i32(lens), page)
    two = ttt.attention_decode(Q, *a, _i32(table), _i32(lens), page)
    assert float((one.float() - two.float()).abs().max()) <= 2 * 2.0 ** -7 * float(two.float().abs().max())
    n = 300
    K, V = dev(_draw(rng, 320, Hkv, dh), "bf16"), dev(_draw(rng, 320, Hkv, dh), "bf16")
    Q = dev(_draw(rng, n, Hq, dh), "bf16")
    one = ttt.attention_paged(Q, K, V, _i32([0, n]), _i32([range(5)]), _i32([n]), page, with_lse=True)
    two = ttt.attention_packed(Q, K[:n], V[:n], _i32([0, n]), with_lse=True)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])  # the same tiles, the same order


def test_refusals():
    import torch
    print("case: paged refusals", flush=True)
    rng = np.random.default_rng(0)
    K, V, table = _pool(rng, [40, 20], 16, 2, 64)
    base = dict(Q=dev(_draw(rng, 6, 4, 64), "bf16"), K_cache=dev(K, "bf16"), V_cache=dev(V, "bf16"),
                cu_q=_i32([0, 4, 6]), page_table=_i32(table), lengths=_i32([40, 20]), page_size=16)
    ttt.attention_paged(**base)
    for kw, err in [
            (dict(Q=base["Q"].float()), TypeError), (dict(Q=base["Q"][0]), ValueError), (dict(Q=base["Q"].cpu()), ValueError),
            (dict(Q=base["Q"][..., :32]), ValueError), (dict(K_cache=base["K_cache"][0]), ValueError),
            (dict(V_cache=base["V_cache"][:16]), ValueError), (dict(cu_q=_i32([0, 6])), ValueError),
            (dict(cu_q=base["cu_q"].long()), TypeError), (dict(cu_q=_i32([[0, 4, 6]])), ValueError),
            (dict(page_table=base["page_table"][0]), ValueError), (dict(lengths=_i32([40])), ValueError),
            (dict(page_size=24), ttt.TTTError), (dict(page_size=8), ttt.TTTError), (dict(page_size=0), ValueError),
            (dict(page_size=256), ttt.TTTError),  # no whole page
            (dict(window=-1), ValueError), (dict(scale=0.0), ttt.TTTError), (dict(O=base["Q"]), ttt.TTTError),
            (dict(lse=torch.zeros(6, 3, device="cuda")), ValueError),
            (dict(Q=dev(_draw(rng, 6, 3, 64), "bf16")), ttt.TTTError)]:
        with pytest.raises(err):
            ttt.attention_paged(**{**base, **kw})
