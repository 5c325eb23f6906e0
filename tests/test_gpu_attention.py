"""GPU parity of ttt_attention_packed and ttt_attention_decode against the fp64 oracle.

Tolerance, element by element. A weight w_j = exp(x_j - m) / n enters the value product as bf16:
off by at most half a step, 2^-8 of itself (the sum n is of the unrounded ones), so o is off by
2^-8 sum_j w_j |v_j| plus its own rounding, 2^-8 |o|. The logits are fp32 sums of dh exact
products: with X the largest sum_c scale |q_c k_c| of the row, off by at most
d = (dh + 4) 2^-24 X, the exponential's argument is rounded on the scale of X too, and the
exponential by a few steps: a weight is off by 2 d + 2^-20 more, and so is n. lse is off by
d + 2^-20 + 4 half steps of its size and of X."""
import numpy as np
import pytest

import chunked_weight_sequence_amd as ttt
import gen
import oracle.attention as oa
from helpers import dev, host_bits, host_f64, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


def _draw(rng, *shape, by=1.0):
    return gen.f32_to_bf16_bits((by * rng.standard_normal(shape)).astype(np.float32))


def _f(x):
    return gen.bf16_bits_to_f32(x).astype(np.float64)


def _i32(x):
    import torch
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def _logit_size(Q, K, scale):
    """[Nq, Hq]: an upper bound of sum_c scale |q_c k_c| over all keys of the head."""
    G = Q.shape[1] // K.shape[1]
    top = np.abs(K).max(axis=0)  # [Hkv, dh]
    return scale * (np.abs(Q) * np.repeat(top, G, axis=0)[None]).sum(-1)


def _check(O, L, want, X, dh, what):
    o, lse, a = want
    got, gl = host_f64(O), host_f64(L)
    d = (dh + 4) * 2.0 ** -24 * X
    bound = 1.01 * (2.0 ** -8 * (np.abs(o) + a) + (4 * d[..., None] + 2.0 ** -19) * a) + 1e-38
    worst = float((np.abs(got - o) / bound).max())
    gone = np.isneginf(lse)
    assert (np.isneginf(gl) == gone).all(), f"{what}: lse of the empty rows"
    assert (got[gone] == 0).all(), f"{what}: empty rows"
    lb = d + 2.0 ** -20 + 4 * 2.0 ** -24 * (np.abs(np.where(gone, 0, lse)) + X)
    lworst = float((np.abs(np.where(gone, 0, gl) - np.where(gone, 0, lse)) / lb).max())
    print(f"  {what}: o {worst:.3f}, lse {lworst:.3f} of their bounds", flush=True)
    assert np.isfinite(got).all() and worst <= 1.0 and lworst <= 1.0, what


def _cu(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)


def _packed(Q, K, V, cu_q, cu_k, scale, window, **kw):
    import torch
    O, L = ttt.attention_packed(dev(Q, "bf16"), dev(K, "bf16"), dev(V, "bf16"), _i32(cu_q),
                                _i32(cu_k), scale=scale, window=window, with_lse=True, **kw)
    torch.cuda.synchronize()
    return O, L


PACKED = [
    # lq of each sequence, lk - lq, Hq, Hkv, dh, window
    ([1], [0], 1, 1, 64, 0),
    ([1], [0], 32, 8, 128, 0),
    ([77], [0], 4, 4, 64, 0),
    ([64, 64], [0, 0], 4, 2, 128, 0),
    ([63, 1, 65], [0, 0, 0], 3, 1, 64, 0),
    ([0, 5, 0, 0, 130, 0], [0, 3, 9, 0, 0, 0], 8, 2, 128, 0),
    ([257], [0], 7, 1, 128, 0),                       # 7 heads to a key head
    ([300, 20], [0, 0], 6, 2, 64, 40),                # a window shorter than a tile
    ([200], [0], 4, 2, 128, 1),                       # only the own key
    ([500], [0], 2, 2, 64, 64),
    ([130], [0], 4, 4, 128, 1 << 30),
    ([17], [1000], 4, 1, 128, 0),                     # the last piece of a prompt
    ([1], [700], 8, 8, 64, 0),
    ([33], [900], 4, 2, 64, 100),
    ([100, 8], [-40, 5], 4, 2, 128, 0),               # 40 queries see nothing
    ([100, 8], [-40, 5], 4, 2, 64, 16),
    ([9, 12], [-9, 0], 2, 1, 64, 0),                  # a sequence without keys
    ([1] * 70, [3] * 70, 2, 1, 64, 0),                # more sequences than a wave has lanes
    ([700], [0], 8, 2, 128, 0),
    ([3, 2, 1, 600, 2], [0] * 5, 2, 1, 128, 0),
    ([40], [3000], 2, 1, 128, 0),                     # few rows, many keys
    ([5, 3], [2, 0], 200, 1, 64, 0),                  # the heads of one query fill more than a row tile
    ([2, 3], [3000, 2000], 300, 2, 128, 700),
    ([64, 1, 0, 33], [1900, 2500, 1000, 0], 4, 2, 64, 0),   # split, of unlike lengths
]


@pytest.mark.parametrize("lq,more,Hq,Hkv,dh,window", PACKED)
def test_packed(lq, more, Hq, Hkv, dh, window):
    print(f"case: packed lq={lq[:8]} more={more[:8]} {Hq}/{Hkv}x{dh} window={window}", flush=True)
    rng = np.random.default_rng(sum(lq) + dh + window % 97)
    cu_q, cu_k = _cu(lq), _cu(np.array(lq) + np.array(more))
    Q = _draw(rng, cu_q[-1], Hq, dh)
    K, V = _draw(rng, max(cu_k[-1], 1), Hkv, dh), _draw(rng, max(cu_k[-1], 1), Hkv, dh)
    scale = 1.3 * dh ** -0.5
    O, L = _packed(Q, K, V, cu_q, cu_k, scale, window)
    _check(O, L, oa.packed(_f(Q), _f(K), _f(V), cu_q, cu_k, scale, window),
           _logit_size(_f(Q), _f(K), scale), dh, "packed")


@pytest.mark.parametrize("by", [4.0, 0.01])
def test_packed_sharp_and_flat_softmax(by):
    print(f"case: packed logits of size {by}", flush=True)
    rng = np.random.default_rng(3)
    Q, K, V = _draw(rng, 300, 4, 128, by=by), _draw(rng, 300, 2, 128, by=by), _draw(rng, 300, 2, 128)
    # rising logits: the running maximum moves in every tile
    K = gen.f32_to_bf16_bits((_f(K) * np.linspace(0.2, 2, 300)[:, None, None]).astype(np.float32))
    O, L = _packed(Q, K, V, [0, 300], [0, 300], 0.5, 0)
    _check(O, L, oa.packed(_f(Q), _f(K), _f(V), [0, 300], [0, 300], 0.5),
           _logit_size(_f(Q), _f(K), 0.5), 128, "packed")


def test_packed_strides_and_rows_of_no_sequence():
    """Slices of one fused buffer in, every second row block out; rows before the first sequence
    and behind the last are left as they were."""
    import torch
    print("case: packed slices, unowned rows", flush=True)
    rng = np.random.default_rng(8)
    N, Hq, Hkv, dh = 150, 4, 2, 64
    row = _draw(rng, N, (Hq + 2 * Hkv) * dh)
    R = dev(row, "bf16")
    q = R[:, :Hq * dh].view(N, Hq, dh)
    k = R[:, Hq * dh:(Hq + Hkv) * dh].view(N, Hkv, dh)
    v = R[:, (Hq + Hkv) * dh:].view(N, Hkv, dh)
    cu = np.array([7, 40, 40, 139], np.int32)
    buf = torch.full((N, 2 * Hq * dh), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, Hq * dh:].view(N, Hq, dh)
    lse = torch.full((N, Hq), 7.0, device="cuda")
    ttt.attention_packed(q, k, v, _i32(cu), scale=0.2, O=out, lse=lse)
    torch.cuda.synchronize()
    f = _f(row)
    qf, kf, vf = (f[:, a * dh:b * dh].reshape(N, -1, dh) for a, b in
                  ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    want = oa.packed(qf, kf, vf, cu, cu, 0.2)
    on = slice(7, 139)
    _check(out[on], lse[on], [x[on] for x in want], _logit_size(qf, kf, 0.2)[on], dh, "slices")
    for part in (buf[:7], buf[139:], buf[:, :Hq * dh], lse[:7], lse[139:]):
        assert (part == 7).all()


def test_packed_neighbours_do_not_leak():
    """NaN in the rows of other sequences, and in rows of none, reaches nothing; a NaN of the own
    sequence reaches the queries that see it and no other."""
    print("case: packed NaN", flush=True)
    rng = np.random.default_rng(9)
    N, dh = 200, 128
    Q, K, V = _draw(rng, N, 4, dh), _draw(rng, N, 2, dh), _draw(rng, N, 2, dh)
    cu = np.array([10, 75, 140, 190], np.int32)
    ref, lref = (host_bits(x) for x in _packed(Q, K, V, cu, cu, 0.1, 0))
    K1, V1 = K.copy(), V.copy()
    for s in (slice(0, 75), slice(140, N)):
        K1[s], V1[s] = 0x7FC0, 0x7F80
    got, lgot = (host_bits(x) for x in _packed(Q, K1, V1, cu, cu, 0.1, 0))
    np.testing.assert_array_equal(got[75:140], ref[75:140])
    np.testing.assert_array_equal(lgot[75:140], lref[75:140])
    K1 = K.copy()
    K1[100, 0] = 0x7FC0
    got = host_f64(_packed(Q, K1, V, cu, cu, 0.1, 0)[0])
    np.testing.assert_array_equal(got[75:100], gen.bf16_bits_to_f32(ref[75:100]))
    assert np.isnan(got[100:140, :2]).all()
    np.testing.assert_array_equal(got[:, 2:][75:140], gen.bf16_bits_to_f32(ref[75:140, 2:]))


def _some_rows(Q, K, V, cu_q, cu_k, scale, window, tokens, heads):
    """The oracle at chosen tokens and heads: (o, lse, sums of weight * |v|) [tokens, heads, ..]."""
    G = Q.shape[1] // K.shape[1]
    out = []
    for t in tokens:
        s = int(np.searchsorted(cu_q, t, side="right")) - 1
        last = t - cu_q[s] + (cu_k[s + 1] - cu_k[s]) - (cu_q[s + 1] - cu_q[s])
        first = max(0, last - window + 1) if window else 0
        ks = slice(cu_k[s] + first, cu_k[s] + max(first, last + 1))
        out += [oa.attend(Q[t, h], K[ks, h // G], V[ks, h // G], scale) for h in heads]
    shape = (len(tokens), len(heads))
    return [np.array([x[i] for x in out]).reshape(*shape, *np.shape(out[0][i])) for i in range(3)]


# long rows whose workgroups of 256 rows fill the compute units evenly: (lq, lk - lq, Hq, Hkv, window)
WIDE = [([4200], [0], 15, 15, 0), ([4200], [0], 30, 15, 0), ([1000], [3000], 32, 32, 2500),
        ([2100, 2050], [2000, 2100], 32, 8, 0), ([300], [2500], 28, 28, 0), ([4200], [0], 45, 45, 0),
        ([2100, 2050], [2000, 2100], 60, 15, 0), ([256], [4200], 64, 8, 0), ([256], [16000], 32, 8, 0)]


@pytest.mark.parametrize("lq,more,Hq,Hkv,window", WIDE)
def test_packed_long_rows(lq, more, Hq, Hkv, window):
    print(f"case: packed long rows lq={lq} more={more} {Hq}/{Hkv} window={window}", flush=True)
    dh, rng = 128, np.random.default_rng(sum(lq) + Hq)
    cu_q, cu_k = _cu(lq), _cu(np.array(lq) + np.array(more))
    Q = _draw(rng, cu_q[-1], Hq, dh)
    K, V = _draw(rng, cu_k[-1], Hkv, dh), _draw(rng, cu_k[-1], Hkv, dh)
    scale = 1.3 * dh ** -0.5
    O, L = _packed(Q, K, V, cu_q, cu_k, scale, window)
    tokens = sorted({0, 1, 63, 64, 127, 128, 255, int(cu_q[-1]) - 1, int(cu_q[1]) - 1,
                     *rng.integers(0, cu_q[-1], 12).tolist()})
    heads = sorted({0, Hq - 1, *rng.integers(0, Hq, 3).tolist()})
    q, k, v = _f(Q), _f(K), _f(V)
    X = _logit_size(q[tokens], k, scale)[:, heads]
    _check(O[tokens][:, heads], L[tokens][:, heads],
           _some_rows(q, k, v, cu_q, cu_k, scale, window, tokens, heads), X, dh, "long rows")
    got = host_f64(O)  # every row was written, none with what lies outside the convex hull of V
    assert np.isfinite(got).all() and np.abs(got).max() <= np.abs(v).max() * (1 + 2.0 ** -6)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("lq,more,Hq,Hkv,dh,window", [
    ([150], [0], 4, 2, 128, 0), ([150], [0], 4, 2, 64, 0), ([90, 130], [30, 0], 3, 1, 64, 50),
    ([40], [3000], 2, 1, 128, 0),                       # the keys are split
    ([40], [3000], 2, 1, 128, 1000), ([300], [2500], 28, 28, 128, 0), ([256], [4200], 64, 8, 128, 0)])
def test_packed_hidden_values_reach_nothing(lq, more, Hq, Hkv, dh, window, bad):
    """Infinities and NaN among the own sequence's keys and values reach the rows that see them, and
    no other row, although the same tiles are multiplied."""
    print(f"case: packed hidden {bad} lq={lq} more={more} {Hq}/{Hkv}x{dh} window={window}", flush=True)
    rng = np.random.default_rng(sum(lq) + dh)
    cu_q, cu_k = _cu(lq), _cu(np.array(lq) + np.array(more))
    Q = _draw(rng, cu_q[-1], Hq, dh)
    K, V = _draw(rng, cu_k[-1], Hkv, dh), _draw(rng, cu_k[-1], Hkv, dh)
    scale = dh ** -0.5
    # key head 0: one value channel of a key in the middle of the first sequence's own part, another of
    # a key near its start; a key vector 10 behind the middle
    mid, near, key = int(cu_k[1]) - lq[0] // 2, 3, int(cu_k[1]) - lq[0] // 2 + 10
    x, q, k, v = gen.f32_to_bf16_bits(np.float32([bad]))[0], _f(Q), _f(K), _f(V)
    V1 = V.copy()
    V1[mid, 0, 5], V1[near, 0, dh - 1] = x, x
    K1 = K.copy()
    K1[key, 0] = 0x7FC0
    O, L = _packed(Q, K1, V1, cu_q, cu_k, scale, window)
    G = Hq // Hkv
    tokens = sorted({*range(min(lq[0], 150)), *rng.integers(0, cu_q[-1], 10).tolist()})
    heads = sorted({0, G - 1, Hq - 1})
    o, lse, a = _some_rows(q, k, v, cu_q, cu_k, scale, window, tokens, heads)
    got, gl = O[tokens][:, heads].clone(), L[tokens][:, heads].clone()
    for i, t in enumerate(tokens):
        last = t + more[0] if t < lq[0] else -1
        first = max(0, last - window + 1) if window else 0
        for j, h in enumerate(heads):
            if h >= G:
                continue
            if first <= key <= last:  # a logit is NaN: the row is
                assert np.isnan(host_f64(got[i, j])).all() and np.isnan(host_f64(gl[i, j]))
                got[i, j], gl[i, j], o[i, j], a[i, j], lse[i, j] = 0, 0, 0, 0, 0
            for at, c in ((mid, 5), (near, dh - 1)):
                if first <= at <= last and not first <= key <= last:
                    np.testing.assert_equal(host_f64(got[i, j, c]), bad)
                    got[i, j, c], o[i, j, c], a[i, j, c] = 0, 0, 0
    k[key, 0] = 0
    _check(got, gl, (o, lse, a), _logit_size(q[tokens], k, scale)[:, heads], dh, "hidden values")


def test_packed_bad_offsets_stay_in_bounds():
    """Offsets outside the tensors or decreasing: nothing outside is read or written. The buffers are
    slices of larger ones, whose other rows would show a write."""
    import torch
    print("case: packed bad offsets", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    big = torch.randn((300, 2, 64), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full((300, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    x = big[100:200]
    for cq, ck in (([0, 500], [0, 500]), ([-9, 50, 100], [-(1 << 31), 50, (1 << 31) - 1]),
                   ([90, 20, 100], [0, 50, 100]), ([0, 100], [60, 30])):
        ttt.attention_packed(x, x, x, _i32(cq), _i32(ck), O=out[100:200])
        torch.cuda.synchronize()
        assert (out[:100] == 7).all() and (out[200:] == 7).all()


DECODE = [
    # lengths, page, Hq, Hkv, dh, window
    ([1], 16, 1, 1, 64, 0),
    ([17], 16, 8, 2, 128, 0),
    ([0, 1, 31, 32, 33, 64, 300], 16, 4, 4, 64, 0),
    ([500, 0, 129, 1000], 64, 14, 2, 128, 0),
    ([300, 40, 7], 32, 32, 1, 64, 0),
    ([90, 200], 128, 66, 1, 128, 0),                  # more heads to a key head than a block of 32
    ([300, 40, 7, 999], 16, 4, 2, 128, 40),
    ([300, 40, 7, 0], 64, 4, 2, 64, 1),
    ([2000], 256, 8, 8, 128, 0),
    ([800] * 40, 16, 16, 16, 64, 0),                  # enough workgroups without splitting far
]


def _cache(rng, lens, page, Hkv, dh, extra=2):
    """Paged caches whose unused rows are NaN: (Kc, Vc, table)."""
    held = [-(-n // page) for n in lens]
    n_pages = sum(held) + extra
    order = rng.permutation(n_pages)
    most = max(max(held), 1) + 1
    table = np.full((len(lens), most), -1, np.int32)
    Kc = np.full((n_pages * page, Hkv, dh), 0x7FC0, np.uint16)
    Vc = np.full((n_pages * page, Hkv, dh), 0x7F80, np.uint16)
    at = 0
    for s, n in enumerate(lens):
        table[s, :held[s]] = order[at:at + held[s]]
        at += held[s]
        rows = [table[s, j // page] * page + j % page for j in range(n)]
        Kc[rows], Vc[rows] = _draw(rng, n, Hkv, dh), _draw(rng, n, Hkv, dh)
    return Kc, Vc, table


def _seen(Kc, table, lens, page):
    return max([float(np.abs(_f(Kc[table[s, j // page] * page + j % page])).max())
                for s, n in enumerate(lens) for j in range(n)] + [1.0])


@pytest.mark.parametrize("lens,page,Hq,Hkv,dh,window", DECODE)
def test_decode(lens, page, Hq, Hkv, dh, window):
    import torch
    print(f"case: decode lens={lens[:8]} page={page} {Hq}/{Hkv}x{dh} window={window}", flush=True)
    rng = np.random.default_rng(sum(lens) + dh)
    S, scale = len(lens), 1.2 * dh ** -0.5
    Kc, Vc, table = _cache(rng, lens, page, Hkv, dh)
    Q = _draw(rng, S, Hq, dh)
    O, L = ttt.attention_decode(dev(Q, "bf16"), dev(Kc, "bf16"), dev(Vc, "bf16"), _i32(table),
                                _i32(lens), page, scale=scale, window=window, with_lse=True)
    torch.cuda.synchronize()
    X = scale * np.abs(_f(Q)).sum(-1) * _seen(Kc, table, lens, page)
    _check(O, L, oa.decode(_f(Q), _f(Kc), _f(Vc), table, lens, page, scale, window), X, dh, "decode")


def test_decode_stale_window_rows_bad_pages_and_lengths():
    """Rows and pages before a window may hold NaN or be gone; pages outside the cache are left out;
    lengths below zero and past the table are cut."""
    import torch
    print("case: decode stale rows, bad pages", flush=True)
    rng = np.random.default_rng(4)
    lens, page, H, dh = [200, 150, 64], 16, 2, 64
    Kc, Vc, table = _cache(rng, lens, page, H, dh)
    Q = _draw(rng, 3, H, dh)
    K1, V1, t1 = Kc.copy(), Vc.copy(), table.copy()
    for s, n in enumerate(lens):  # what a window of 20 no longer sees
        for j in range(n - 20):
            K1[table[s, j // page] * page + j % page] = 0x7FC0
            V1[table[s, j // page] * page + j % page] = 0x7FC0
        t1[s, :(n - 20) // page] = [-7, 1 << 30, -(1 << 31)][s]

    def run(K, V, t, n, window):
        O, L = ttt.attention_decode(dev(Q, "bf16"), dev(K, "bf16"), dev(V, "bf16"), _i32(t), _i32(n),
                                    page, window=window, with_lse=True)
        torch.cuda.synchronize()
        return host_bits(O), host_bits(L)
    for a, b in zip(run(K1, V1, t1, lens, 20), run(Kc, Vc, table, lens, 20)):
        np.testing.assert_array_equal(a, b)
    t2 = table.copy()
    t2[0, 3], t2[1, 0], t2[2, :] = -1, len(Kc) // page, -1  # all of sequence 2's pages
    n2 = [200, 150, 64]
    O, L, A = oa.decode(_f(Q), _f(Kc), _f(Vc), t2, n2, page, dh ** -0.5)
    got = ttt.attention_decode(dev(Q, "bf16"), dev(Kc, "bf16"), dev(Vc, "bf16"), _i32(t2), _i32(n2),
                               page, with_lse=True)
    torch.cuda.synchronize()
    X = dh ** -0.5 * np.abs(_f(Q)).sum(-1) * _seen(Kc, table, lens, page)
    _check(*got, (O, L, A), X, dh, "bad pages")
    assert np.isneginf(L[2]).all()
    full = table.shape[1] * page  # the last page of each row is -1: cut there either way
    for a, b in zip(run(Kc, Vc, table, [full + 99, -5, -(1 << 31)], 0),
                    run(Kc, Vc, table, [full, 0, 0], 0)):
        np.testing.assert_array_equal(a, b)


def test_decode_pages_of_several_sequences():
    """A page may stand in several rows of the table (a shared prefix), and twice in one."""
    import torch
    print("case: decode shared pages", flush=True)
    rng = np.random.default_rng(11)
    page, Hq, Hkv, dh = 32, 4, 2, 64
    Kc, Vc = _draw(rng, 9 * page, Hkv, dh), _draw(rng, 9 * page, Hkv, dh)
    table = np.array([[4, 1, 7, -1], [4, 1, 2, 8], [5, 5, 5, 5]], np.int32)
    lens, Q = [80, 128, 100], _draw(rng, 3, Hq, dh)
    O, L = ttt.attention_decode(dev(Q, "bf16"), dev(Kc, "bf16"), dev(Vc, "bf16"), _i32(table),
                                _i32(lens), page, with_lse=True)
    torch.cuda.synchronize()
    X = dh ** -0.5 * np.abs(_f(Q)).sum(-1) * _seen(Kc, table, lens, page)
    _check(O, L, oa.decode(_f(Q), _f(Kc), _f(Vc), table, lens, page, dh ** -0.5), X, dh, "shared")


def test_decode_equals_the_packed_call_on_the_same_keys():
    import torch
    print("case: decode against packed", flush=True)
    rng = np.random.default_rng(6)
    lens, page, Hq, Hkv, dh = [70, 33, 256], 32, 4, 2, 128
    Kc, Vc, table = _cache(rng, lens, page, Hkv, dh)
    Q = _draw(rng, 3, Hq, dh)
    rows = [table[s, j // page] * page + j % page for s, n in enumerate(lens) for j in range(n)]
    a = ttt.attention_decode(dev(Q, "bf16"), dev(Kc, "bf16"), dev(Vc, "bf16"), _i32(table),
                             _i32(lens), page)
    b = ttt.attention_packed(dev(Q, "bf16"), dev(Kc[rows], "bf16"), dev(Vc[rows], "bf16"),
                             _i32([0, 1, 2, 3]), _i32(_cu(lens)))
    torch.cuda.synchronize()
    want, _, A = oa.decode(_f(Q), _f(Kc), _f(Vc), table, lens, page, dh ** -0.5)
    off = np.abs(host_f64(a) - host_f64(b))  # each is within 2^-8 (|o| + A) of the oracle
    assert (off <= 2 * 1.05 * 2.0 ** -8 * (np.abs(want) + A)).all()


def test_attention_refuses_what_it_cannot_check_on_the_device():
    import torch
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = _i32([0, 4])
    bad = [dict(K=q.float()), dict(V=q[:3]), dict(cu_q=cu.long()), dict(cu_k=_i32([0, 2, 4])),
           dict(K=q[:, :, :32]), dict(O=q.float()), dict(O=q[:2]), dict(cu_q=cu.cpu()),
           dict(lse=torch.zeros(4, 3, device="cuda")), dict(window=-1), dict(window=1 << 32),
           dict(scale=0.0), dict(Q=q.transpose(0, 1)), dict(Q=q[0]), dict(Q=q[:0])]
    for kw in bad:
        args = dict(Q=q, K=q, V=q, cu_q=cu)
        args.update(kw)
        with pytest.raises((ValueError, TypeError, ttt.TTTError)):
            ttt.attention_packed(**args)
    C, table = torch.zeros(64, 2, 64, dtype=torch.bfloat16, device="cuda"), _i32([[0, 1]] * 4)
    bad = [dict(K_cache=C[::2]), dict(V_cache=C[:32]), dict(page_table=table.long()),
           dict(page_table=table[:3]), dict(page_table=table[0]), dict(lengths=_i32([1, 2])),
           dict(page_size=24), dict(page_size=8), dict(page_size=0), dict(page_size=1 << 33),
           dict(page_size=128), dict(window=-2), dict(Q=q.float()), dict(O=q[:3]),
           dict(workspace=torch.zeros(64, dtype=torch.uint8))]
    for kw in bad:
        args = dict(Q=q, K_cache=C, V_cache=C.clone(), page_table=table, lengths=_i32([4] * 4),
                    page_size=32)
        args.update(kw)
        with pytest.raises((ValueError, TypeError, ttt.TTTError)):
            ttt.attention_decode(**args)


@pytest.mark.parametrize("seed", range(24))
def test_packed_random_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    dh, Hkv, G = int(rng.choice([64, 128])), int(rng.choice([1, 2, 3, 8])), int(rng.choice([1, 2, 4, 5]))
    n = int(rng.choice([1, 2, 5, 16, 17, 40, 63, 64, 80]))
    lq = rng.multinomial(int(rng.integers(1, 500)), rng.dirichlet(np.ones(n)))
    more = rng.integers(-20, int(rng.choice([1, 60, 600])), n) * int(rng.integers(0, 2))
    lk = np.maximum(lq + more, 0)
    window = int(rng.choice([0, 0, 1, 30, 100]))
    print(f"case: packed random {seed}: {n} sequences, {lq.sum()} queries, {lk.sum()} keys, "
          f"{Hkv * G}/{Hkv}x{dh} window={window}", flush=True)
    cu_q, cu_k = _cu(lq), _cu(lk)
    Q = _draw(rng, cu_q[-1], Hkv * G, dh)
    K, V = _draw(rng, max(cu_k[-1], 1), Hkv, dh), _draw(rng, max(cu_k[-1], 1), Hkv, dh)
    scale = float(rng.uniform(0.5, 2)) * dh ** -0.5
    O, L = _packed(Q, K, V, cu_q, cu_k, scale, window)
    _check(O, L, oa.packed(_f(Q), _f(K), _f(V), cu_q, cu_k, scale, window),
           _logit_size(_f(Q), _f(K), scale), dh, "packed")


@pytest.mark.parametrize("seed", range(16))
def test_decode_random_shapes(seed):
    import torch
    rng = np.random.default_rng(2000 + seed)
    dh, Hkv, G = int(rng.choice([64, 128])), int(rng.choice([1, 2, 3, 8])), int(rng.choice([1, 4, 7, 33]))
    S, page = int(rng.choice([1, 2, 9, 40])), int(rng.choice([16, 32, 128]))
    lens = [int(x) for x in rng.integers(0, int(rng.choice([40, 400, 2000])) // S ** 0.5 + 2, S)]
    window = int(rng.choice([0, 0, 1, 33, 200]))
    print(f"case: decode random {seed}: lens={lens[:8]} page={page} {Hkv * G}/{Hkv}x{dh} "
          f"window={window}", flush=True)
    Kc, Vc, table = _cache(rng, lens, page, Hkv, dh)
    Q, scale = _draw(rng, S, Hkv * G, dh), 1.2 * dh ** -0.5
    O, L = ttt.attention_decode(dev(Q, "bf16"), dev(Kc, "bf16"), dev(Vc, "bf16"), _i32(table),
                                _i32(lens), page, scale=scale, window=window, with_lse=True)
    torch.cuda.synchronize()
    X = scale * np.abs(_f(Q)).sum(-1) * _seen(Kc, table, lens, page)
    _check(O, L, oa.decode(_f(Q), _f(Kc), _f(Vc), table, lens, page, scale, window), X, dh, "decode")
