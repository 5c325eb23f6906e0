"""GPU parity of the gated delta rule against the fp64 oracle.

Tolerance, element by element, against the oracle's sums of sizes A of the state and B of the outputs
(each product by its size, each difference a sum). For one token: sums of dk products in fp32, in any order,
are off by at most dk half steps of fp32, 2^-24, of the sum of their sizes; the factors that normalise q and k by
at most dk / 2 + 4 half steps, the exponential by 4, and a dozen products by one each. Both S^T k and
then k u take such sums: 3 dk + 64 half steps of A (or of B) hold, and half a step of the output's type."""
import numpy as np
import pytest

import chunked_weight_sequence_amd as ttt
import gen
import oracle.serving as osv
from helpers import dev, host_bits, host_f64, requires_gpu
from test_gpu_attention import _f, _i32

pytestmark = [pytest.mark.gpu, requires_gpu]

EPS = 1e-6


def _draw(rng, N, Hk, Hv, dk, dv, unit=False):
    """bf16 bits of q, k, v (keys of a head have a direction in common), the gates and the steps."""
    q = rng.standard_normal((N, Hk, dk))
    k = rng.standard_normal((N, Hk, dk)) + 0.5 * rng.standard_normal((Hk, dk))
    if unit:  # keys that keep the state bounded without being divided by their norm
        q, k = q / np.sqrt(dk), k / (1.2 * np.sqrt(dk))
    v = rng.standard_normal((N, Hv, dv))
    rate = np.exp(rng.uniform(np.log(1e-3), 0, Hv))
    g = (-rate * np.log1p(np.exp(rng.standard_normal((N, Hv))))).astype(np.float32)
    beta = (1 / (1 + np.exp(-rng.standard_normal((N, Hv))))).astype(np.float32)
    return [gen.f32_to_bf16_bits(x.astype(np.float32)) for x in (q, k, v)] + [g, beta]


def _on_gpu(x):
    return [dev(a, "bf16") for a in x[:3]] + [dev(a, "f32") for a in x[3:]]


def _check(got, want, size, steps, half, what):
    got = host_f64(got) if not isinstance(got, np.ndarray) else got
    bound = 1.01 * half * np.abs(want) + steps * 2.0 ** -24 * size + 1e-37
    worst = float((np.abs(got - want) / bound).max()) if want.size else 0.0
    print(f"  {what}: {worst:.3f} of its bound", flush=True)
    assert np.isfinite(got).all() and worst <= 1.0, what


def _token_check(x, O, got_state, before, rows, states, scale, eps, dk):
    """Every sequence's token against the oracle: rows[i] of the inputs, state number states[i] (None: zero)."""
    for i, r in enumerate(rows):
        W0 = None if states[i] is None else before[states[i]]
        a = [_f(t[r:r + 1]) for t in x[:3]] + [t[r:r + 1] for t in x[3:]]
        o, w, b, size = osv.gated_delta(*a, W0, scale, eps)
        _check(O[r:r + 1], o, b, 3 * dk + 64, 2.0 ** -8, f"o of sequence {i}")
        if states[i] is not None:
            _check(got_state[states[i]], w, size, 3 * dk + 64, 0.0, f"state of sequence {i}")


@pytest.mark.parametrize("S,Hk,Hv,dk,dv", [(1, 1, 1, 64, 64), (1, 4, 8, 128, 128), (3, 2, 2, 64, 128), (2, 1, 4, 128, 64),
                                           (5, 2, 6, 128, 192), (40, 4, 8, 128, 256), (2, 2, 2, 64, 512),
                                           (150, 2, 4, 128, 128), (33, 8, 16, 64, 64)])
@pytest.mark.parametrize("normalize", [True, False])
def test_one_token(S, Hk, Hv, dk, dv, normalize):
    import torch
    print(f"case: delta token {S} x {Hk}/{Hv} heads {dk} x {dv} {normalize}", flush=True)
    rng = np.random.default_rng(S + Hv + dk + dv)
    x = _draw(rng, S, Hk, Hv, dk, dv, unit=not normalize)
    before = rng.standard_normal((S + 2, Hv, dk, dv)).astype(np.float32)
    at = rng.permutation(S + 2)[:S]
    pool, out = dev(before, "f32"), torch.full((S + 2, Hv, dk, dv), 7.0, device="cuda")
    O, st = ttt.gated_delta_decode(*_on_gpu(x), pool, state_out=out, slots=_i32(at), normalize=normalize,
                                   norm_eps=EPS)
    torch.cuda.synchronize()
    assert st is out
    np.testing.assert_array_equal(host_bits(pool), before)
    some = rng.permutation(S)[:6]
    eps = EPS if normalize else None
    _token_check(x, O, host_f64(out), before, some, at[some], dk ** -0.5, eps, dk)
    rest = np.setdiff1d(np.arange(S + 2), at)
    assert (host_f64(out)[rest] == 7).all()  # other slots as they were
    O2, st2 = ttt.gated_delta_decode(*_on_gpu(x), pool, slots=_i32(at), normalize=normalize, norm_eps=EPS)  # in place
    assert st2 is pool and torch.equal(O2, O) and torch.equal(pool[at], out[at])


def test_token_edges():
    """Padding slots, gates that forget everything or nothing, steps of zero, no slots, queries and keys of
    zeros, infinities in one sequence, slices of one buffer."""
    import torch
    print("case: delta token edges", flush=True)
    S, Hk, Hv, dk, dv = 7, 2, 4, 128, 128
    rng = np.random.default_rng(8)
    x = _draw(rng, S, Hk, Hv, dk, dv)
    x[3][1], x[3][2], x[4][2], x[4][3] = -np.inf, 0, 0, 0
    x[0][4], x[1][4] = 0, 0
    x[2][5, 1, 3] = 0x7F80  # an infinite value
    before = rng.standard_normal((S, Hv, dk, dv)).astype(np.float32)
    slots = [3, 0, 1, 2, 4, 5, -1]
    pool = dev(before, "f32")
    row = torch.cat([t.reshape(S, -1) for t in _on_gpu(x)[:3]], 1)
    q, k, v = row[:, :Hk * dk].view(S, Hk, dk), row[:, Hk * dk:2 * Hk * dk].view(S, Hk, dk), row[:, 2 * Hk * dk:].view(S, Hv, dv)
    wide = torch.full((S, 2 * Hv, dv), 7.0, dtype=torch.bfloat16, device="cuda")
    O, _ = ttt.gated_delta_decode(q, k, v, *_on_gpu(x)[3:], pool, slots=_i32(slots), scale=0.3, O=wide[:, :Hv])
    torch.cuda.synchronize()
    rows, states = [0, 1, 2, 3, 4, 6], [3, 0, 1, 2, 4, None]
    _token_check(x, O, host_f64(pool), before, rows, states, 0.3, EPS, dk)
    after = host_f64(pool)
    assert (wide[:, Hv:] == 7).all()
    np.testing.assert_array_equal(after[6], before[6])  # no sequence's: the padding wrote nothing
    np.testing.assert_array_equal(after[1], before[1])  # nothing forgotten, no step
    bad = np.zeros((Hv, dv), bool)
    bad[1, 3] = True
    assert (~np.isfinite(after[5]).all(axis=1) == bad).all() and (np.isfinite(host_f64(O)[5]) == ~bad).all()
    pool = dev(before, "f32")  # without slots each sequence has its own number's
    O, _ = ttt.gated_delta_decode(*_on_gpu(x), pool)
    _token_check(x, O, host_f64(pool), before, [0, 1, 2, 3, 4, 6], [0, 1, 2, 3, 4, 6], dk ** -0.5, EPS, dk)


def test_token_refusals():
    import torch
    print("case: delta token refusals", flush=True)
    S, Hk, Hv, dk, dv = 3, 2, 4, 64, 64
    x = _on_gpu(_draw(np.random.default_rng(0), S, Hk, Hv, dk, dv))
    st = torch.zeros(S, Hv, dk, dv, device="cuda")
    def call(i=None, t=None, state=st, **kw):
        a = list(x)
        if i is not None:
            a[i] = t
        return ttt.gated_delta_decode(*a, state, **kw)
    call()
    for kw, err in [
            (dict(i=0, t=x[0].float()), TypeError), (dict(i=1, t=x[1][:2]), ValueError),
            (dict(i=1, t=x[1][:, :1]), ValueError), (dict(i=2, t=x[2][:2]), ValueError),
            (dict(i=2, t=x[2][:, :3]), ValueError), (dict(i=3, t=x[3].double()), TypeError),
            (dict(i=4, t=x[4][:, :2]), ValueError), (dict(state=st[:2]), ValueError),
            (dict(state=st.half()), TypeError), (dict(state=st[0]), ValueError), (dict(state=st.cpu()), ValueError),
            (dict(state=st, state_out=torch.zeros(4, Hv, dk, dv, device="cuda")), ValueError),
            (dict(slots=_i32([0, 1])), ValueError), (dict(slots=torch.zeros(S, dtype=torch.int64, device="cuda")), TypeError),
            (dict(O=x[2]), ttt.TTTError), (dict(O=x[2].float()), TypeError), (dict(scale=float("nan")), ttt.TTTError),
            (dict(norm_eps=-1.0), ttt.TTTError)]:
        with pytest.raises(err):
            call(**kw)
    for dk2, dv2 in ((32, 64), (64, 32), (256, 64), (64, 576)):  # outside what is implemented
        y = _on_gpu(_draw(np.random.default_rng(0), S, Hk, Hv, dk2, dv2))
        with pytest.raises(ttt.TTTError):
            ttt.gated_delta_decode(*y, torch.zeros(S, Hv, dk2, dv2, device="cuda"))


def _chunk_sizes(x, S, scale, eps):
    """Of up to 64 tokens from the state S [Hv, dk, dv]: scale |q| |S| + 2 |A| |u| of every output."""
    q, k, v = (_f(t) for t in x[:3])
    g, beta = (t.astype(np.float64) for t in x[3:])
    n, Hk, dk = q.shape
    Hv = v.shape[1]
    out = np.zeros(v.shape)
    for h in range(Hv):
        a, b = q[:, h // (Hv // Hk)], k[:, h // (Hv // Hk)]
        if eps is not None:
            a, b = (t / np.sqrt((t * t).sum(1, keepdims=True) + eps) for t in (a, b))
        G = np.cumsum(np.maximum(g[:, h], -1000))
        low = np.tril(np.exp(np.minimum(G[:, None] - G[None], 0)))
        L = np.tril(beta[:, h, None] * (b @ b.T) * low, -1)
        u = np.linalg.solve(np.eye(n) + L, beta[:, h, None] * (v[:, h] - np.exp(G)[:, None] * (b @ S[h])))
        out[:, h] = abs(scale) * (np.exp(G)[:, None] * (np.abs(a) @ np.abs(S[h])) + 2 * np.abs((a @ b.T) * low) @ np.abs(u))
    return out


def _packed_check(x, O, lens, first, starts, ends, scale, eps):
    """O [N, Hv, dv] of the packed sequences, starts[s] [Hv, dk, dv] or None, ends[s] the states that came out (or
    None where they were not kept). Returns the worst relative error of a state."""
    got, at, worst, off = host_f64(O), first, 0.0, 0.0
    for s, n in enumerate(lens):
        Hv, dv, dk = x[2].shape[1], x[2].shape[2], x[0].shape[2]
        W = np.zeros((Hv, dk, dv)) if starts[s] is None else starts[s].astype(np.float64)
        for c in range(0, n, 64):
            part = [t[at + c:at + min(c + 64, n)] for t in x]
            size = _chunk_sizes(part, W, scale, eps)
            o, W, _, _ = osv.gated_delta(*[_f(t) for t in part[:3]], *part[3:], W, scale, eps)
            y = got[at + c:at + min(c + 64, n)]
            bound = 1.01 * 2.0 ** -8 * (np.abs(o) + size) + 2.0 ** -14 * (size + size.max(axis=2, keepdims=True)) + 1e-37
            worst = max(worst, float((np.abs(y - o) / bound).max()))
            assert np.isfinite(y).all()
        if ends[s] is not None:
            e = np.abs(ends[s] - W)
            for h in range(Hv):
                norm = np.linalg.norm(W[h])
                off = max(off, np.linalg.norm(e[h]) / norm if norm else float(e[h].max() > 0))
                assert (e[h] <= 64 * 2e-6 * (np.linalg.norm(W[h], axis=0) + norm / np.sqrt(dv)) / np.sqrt(dk) + 1e-37).all()
        at += n
    print(f"  o {worst:.3f} of its bound, states {off:.2e} off", flush=True)
    assert worst <= 1.0 and off <= 2e-6
    return off


def _packed(rng, lens, Hk, Hv, dk, dv, first=0, behind=0, normalize=True, state=True, scale=None, kept=True, edit=None):
    """Calls the operator on sequences of these lengths with states in slots of a pool, and checks everything."""
    import torch
    N, S = first + sum(lens) + behind, len(lens)
    x = _draw(rng, N, Hk, Hv, dk, dv, unit=not normalize)
    if edit:
        edit(x)
    cu = np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)
    before = rng.standard_normal((S + 2, Hv, dk, dv)).astype(np.float32)
    at = rng.permutation(S + 2)[:S]
    pool, out = dev(before, "f32"), torch.full((S + 2, Hv, dk, dv), 7.0, device="cuda")
    O = torch.full((N, Hv, dv), 7.0, dtype=torch.bfloat16, device="cuda")
    kw = dict(state=pool if state else None, slots=_i32(at), scale=scale, normalize=normalize, norm_eps=EPS, O=O)
    if not kept and not state:
        kw["slots"] = None
    _, st = ttt.gated_delta_packed(*_on_gpu(x), _i32(cu), state_out=out if kept else None, final_state=kept, **kw)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(host_bits(pool), before)
    assert (host_f64(O)[:first] == 7).all() and (host_f64(O)[N - behind:] == 7).all()
    after = host_f64(out)
    assert (st is out) == kept and (after[np.setdiff1d(np.arange(S + 2), at if kept else [])] == 7).all()
    _packed_check(x, O, lens, first, [before[a] if state else None for a in at],
                  [after[a] if kept else None for a in at], dk ** -0.5 if scale is None else scale,
                  EPS if normalize else None)
    return x, cu, before, at, O, out


@pytest.mark.parametrize("Hk,Hv,dk,dv", [(1, 1, 64, 64), (2, 4, 128, 128), (2, 2, 64, 128), (1, 3, 128, 64), (1, 2, 128, 192),
                                         (1, 1, 64, 512), (2, 2, 128, 256)])
def test_packed_sizes(Hk, Hv, dk, dv):
    """Sequences of no, one, 63 to 65 and more tokens, tokens of no sequence before and behind them."""
    print(f"case: delta packed {Hk}/{Hv} heads {dk} x {dv}", flush=True)
    rng = np.random.default_rng(Hv + dk + dv)
    _packed(rng, [64, 0, 1, 65, 63, 200, 0, 17], Hk, Hv, dk, dv, first=5, behind=3)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 48, 63, 64, 65, 127, 129])
def test_packed_one_sequence(n):
    print(f"case: delta packed, one sequence of {n}", flush=True)
    _packed(np.random.default_rng(n), [n], 1, 2, 128, 128)


@pytest.mark.parametrize("state,kept,normalize,scale", [(False, True, True, None), (True, False, True, 1.0), (False, False, False, None),
                                                        (True, True, False, -0.5)])
def test_packed_options(state, kept, normalize, scale):
    print(f"case: delta packed options {state} {kept} {normalize} {scale}", flush=True)
    _packed(np.random.default_rng(3), [100, 30], 2, 4, 128, 64, state=state, kept=kept, normalize=normalize, scale=scale)


@pytest.mark.parametrize("lens,Hk,Hv,dk,dv", [([700], 2, 2, 128, 128), ([30, 1, 100] * 12, 4, 8, 64, 128), ([3] * 70, 8, 8, 64, 64),
                                              ([70, 5] * 16, 4, 8, 128, 128), ([130] * 3, 16, 32, 128, 128)])
def test_packed_long_and_many(lens, Hk, Hv, dk, dv):
    """Every width of the workgroups' columns, more than 64 sequences."""
    print(f"case: delta packed long {lens[:3]} x {len(lens)} {Hk}/{Hv} {dk} x {dv}", flush=True)
    _packed(np.random.default_rng(len(lens)), lens, Hk, Hv, dk, dv)


@pytest.mark.parametrize("n", [2, 63, 64, 65, 129, 1023, 1024, 1025])
def test_packed_sequences_of_unlike_lengths(n):
    """The longest ones last and in the middle, many of one length, empty ones: on both sides of the number up to
    which sequences are taken in the order of their lengths."""
    print(f"case: delta packed, {n} sequences of unlike lengths", flush=True)
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 4, n)
    lens[n // 2], lens[-1] = 130, 300
    _packed(rng, [int(i) for i in lens], 1, 1, 64, 64, first=1)


def test_packed_gates_and_steps():
    """Gates of 0, of -inf (everything forgotten), of -1e5; steps of 0 and 1; keys and queries of zeros; the same
    key again and again."""
    print("case: delta packed gates", flush=True)

    def edit(x):
        q, k, v, g, b = x
        g[:40], b[3], b[7:9] = 0, 0, 1
        g[50, 0], g[50, 1], g[70] = -np.inf, -1e5, -np.inf
        g[64, -1] = -np.inf
        k[20], q[22], k[90:] = 0, 0, k[90]
        b[100:] = 1
        g[110:] = 0
    _packed(np.random.default_rng(12), [130, 20], 2, 4, 128, 128, edit=edit)
    _packed(np.random.default_rng(13), [130, 20], 1, 2, 64, 64, edit=edit)


def test_packed_in_pieces_and_by_tokens():
    """A prompt in pieces, in place in the pool, and single tokens after it: the result of one call over all of it
    (within the bounds of both), and slices of one buffer as inputs."""
    import torch
    print("case: delta packed in pieces", flush=True)
    rng = np.random.default_rng(5)
    Hk, Hv, dk, dv, lens, cuts = 2, 4, 128, 128, [150, 90], [64, 100, 131, 147]
    x = _draw(rng, sum(lens), Hk, Hv, dk, dv)
    t = _on_gpu(x)
    row = torch.cat([a.reshape(sum(lens), -1) for a in t[:3]], 1)
    q, k, v = row[:, :Hk * dk].view(-1, Hk, dk), row[:, Hk * dk:2 * Hk * dk].view(-1, Hk, dk), row[:, 2 * Hk * dk:].view(-1, Hv, dv)
    before = rng.standard_normal((4, Hv, dk, dv)).astype(np.float32)
    at, pool = _i32([2, 0]), dev(before, "f32")
    O = torch.zeros(sum(lens), Hv, dv, dtype=torch.bfloat16, device="cuda")
    last = 0
    for c in cuts:
        rows = [torch.arange(min(last, n), min(c, n), device="cuda") + o for n, o in zip(lens, (0, lens[0]))]
        cu = _i32([0, len(rows[0]), len(rows[0]) + len(rows[1])])
        r = torch.cat(rows)
        o, st = ttt.gated_delta_packed(*[a[r] for a in (q, k, v)], *[a[r] for a in t[3:]], cu, state=pool, slots=at, norm_eps=EPS)
        assert st is pool
        O[r] = o
        last = c
    for c in range(last, lens[0]):  # the second one has ended: its place is padding
        r = [c, 0]
        o, _ = ttt.gated_delta_decode(q[r], k[r], v[r], t[3][r], t[4][r], pool, slots=_i32([2, -1]), norm_eps=EPS)
        O[c] = o[0]
    torch.cuda.synchronize()
    after = host_f64(pool)
    _packed_check(x, O, lens, 0, [before[2], before[0]], [after[2], after[0]], dk ** -0.5, EPS)
    np.testing.assert_array_equal(after[[1, 3]], before[[1, 3]])
    whole, st = ttt.gated_delta_packed(q, k, v, *t[3:], _i32([0, 150, 240]), state=dev(before, "f32"), slots=at, norm_eps=EPS)
    _packed_check(x, whole, lens, 0, [before[2], before[0]], [host_f64(st)[2], host_f64(st)[0]], dk ** -0.5, EPS)


def test_packed_values_stay_in_their_sequence():
    """Infinities and NaN among one sequence's inputs and states reach no other sequence, no other head where they
    are of one head, and no chunk before their own."""
    import torch
    print("case: delta packed, infinities and NaN", flush=True)
    rng = np.random.default_rng(6)
    lens, Hk, Hv, dk, dv = [70, 150, 40], 2, 2, 128, 64
    x = _draw(rng, sum(lens), Hk, Hv, dk, dv)
    before = rng.standard_normal((3, Hv, dk, dv)).astype(np.float32)
    clean = ttt.gated_delta_packed(*_on_gpu(x), _i32([0, 70, 220, 260]), state=dev(before, "f32"))
    y = [a.copy() for a in x]
    y[2][70 + 100, 0, 5] = 0x7F80   # a value of the second sequence, head 0, in its second chunk
    y[1][70 + 140, 1, 3] = 0x7FC0   # a key of head 1, in its third
    dirty = ttt.gated_delta_packed(*_on_gpu(y), _i32([0, 70, 220, 260]), state=dev(before, "f32"))
    torch.cuda.synchronize()
    a, b = host_bits(clean[0]), host_bits(dirty[0])
    for rows, h in ((slice(0, 70), slice(None)), (slice(220, 260), slice(None)), (slice(70, 134), 0), (slice(70, 198), 1)):
        np.testing.assert_array_equal(a[rows, h], b[rows, h])
    np.testing.assert_array_equal(host_bits(clean[1])[[0, 2]], host_bits(dirty[1])[[0, 2]])
    assert not np.isfinite(host_f64(dirty[1])[1, 0, :, 5]).all() and np.isnan(host_f64(dirty[1])[1, 1]).any()


def test_packed_refusals():
    import torch
    print("case: delta packed refusals", flush=True)
    N, Hk, Hv, dk, dv = 40, 2, 4, 64, 64
    x = _on_gpu(_draw(np.random.default_rng(0), N, Hk, Hv, dk, dv))
    cu, st = _i32([0, 10, 40]), torch.zeros(2, Hv, dk, dv, device="cuda")
    O, new = ttt.gated_delta_packed(*x, cu)
    assert new.shape == (2, Hv, dk, dv)
    assert ttt.gated_delta_packed(*x, cu, final_state=False)[1] is None
    for cu2, kw, err in [
            (cu.long(), {}, TypeError), (cu[None], {}, ValueError), (cu.cpu(), {}, ValueError), (cu[:1], {}, ttt.TTTError),
            (cu, dict(state=st[:1]), ValueError), (cu, dict(slots=_i32([0, 1])), ValueError),
            (cu, dict(state_out=st, final_state=False), ValueError), (cu, dict(state=st, slots=_i32([0])), ValueError),
            (cu, dict(state=st, state_out=st.double()), TypeError), (cu, dict(O=x[2]), ttt.TTTError),
            (cu, dict(workspace=torch.empty(1000, dtype=torch.uint8, device="cuda")), ttt.TTTError)]:
        with pytest.raises(err):
            ttt.gated_delta_packed(*x, cu2, **kw)


def test_offsets_are_clamped_and_states_may_be_missing():
    """Offsets outside the buffers; one token without a state, kept or not."""
    import torch
    print("case: delta, clamped offsets, no states", flush=True)
    rng = np.random.default_rng(15)
    N, Hk, Hv, dk, dv = 100, 1, 2, 64, 128
    x = _draw(rng, N, Hk, Hv, dk, dv)
    O, st = ttt.gated_delta_packed(*_on_gpu(x), _i32([-7, 70, 1 << 30]), norm_eps=EPS)
    torch.cuda.synchronize()
    _packed_check(x, O, [70, 30], 0, [None, None], list(host_f64(st)), dk ** -0.5, EPS)
    one = [a[:3] for a in x]
    new = torch.full((3, Hv, dk, dv), 7.0, device="cuda")
    O, st = ttt.gated_delta_decode(*_on_gpu(one), None, state_out=new, norm_eps=EPS)
    O2, none = ttt.gated_delta_decode(*_on_gpu(one), None, norm_eps=EPS)
    torch.cuda.synchronize()
    assert st is new and none is None and torch.equal(O, O2)
    _packed_check(one, O, [1, 1, 1], 0, [None] * 3, list(host_f64(new)), dk ** -0.5, EPS)


def test_offsets_of_no_entry_are_refused():
    """As such, before a state for minus one sequences is made."""
    print("case: delta packed, no offsets", flush=True)
    x = _on_gpu(_draw(np.random.default_rng(0), 4, 1, 1, 64, 64))
    with pytest.raises(ValueError):
        ttt.gated_delta_packed(*x, _i32([]))


@pytest.mark.parametrize("beta,common,dk", [(0.01, 0.5, 128), (1e-4, 0.5, 64), (1.0, 3.0, 128)])
def test_a_long_state_that_forgets_nothing(beta, common, dk):
    """16384 tokens with gates of 0, against the recurrence in 64 bits. A chunk's products round a state's element 8 times,
    by a third of the square of half a step each: after 256 chunks sqrt(8 * 256 / 3) * 2^-24 = 1.6e-6 of its size at most, as
    roundings go their own ways; 2e-6 is what is stated. Tokens one by one round 64 times where a chunk does 8, and are to be
    no nearer where that counts: a step takes beta of what a state has along its key, 1 / dk of all of it, so a rounding lasts
    for dk / beta tokens, 100 chunks and more with steps of 0.01 and less, but two with steps of 1, whose 16 roundings are
    no more than those of u and T themselves, of which single tokens have fewer."""
    import torch
    print(f"case: delta packed, long state, {beta} {common} {dk}", flush=True)
    N, H, dv = 16384, 2, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(N, H, dk, generator=g, device="cuda").bfloat16()
    k = (torch.randn(N, H, dk, generator=g, device="cuda") + common * torch.randn(H, dk, generator=g, device="cuda")).bfloat16()
    v = (torch.randn(N, H, dv, generator=g, device="cuda") + 1).bfloat16()
    gates, steps = torch.zeros(N, H, device="cuda"), torch.full((N, H), beta, device="cuda")
    _, whole = ttt.gated_delta_packed(q, k, v, gates, steps, _i32([0, N]), norm_eps=EPS)
    one = torch.zeros(1, H, dk, dv, device="cuda")
    b, u = steps[0, 0].double(), k.double()
    u, w = u / ((u * u).sum(-1, keepdim=True) + EPS).sqrt(), v.double()
    want = torch.zeros(H, dk, dv, dtype=torch.float64, device="cuda")
    for t in range(N):
        want += u[t][..., None] * (b * (w[t] - (u[t][..., None] * want).sum(1)))[:, None]
        ttt.gated_delta_decode(q[t:t + 1], k[t:t + 1], v[t:t + 1], gates[:1], steps[:1], one, norm_eps=EPS)
    off = lambda x: [float((x[0, h].double() - want[h]).norm() / want[h].norm()) for h in range(H)]  # noqa: E731
    print(f"  states {max(off(whole)):.2e} off, token by token {max(off(one)):.2e}", flush=True)
    assert max(off(whole)) <= 2e-6
    assert beta > 0.01 or max(off(whole)) <= max(off(one))
