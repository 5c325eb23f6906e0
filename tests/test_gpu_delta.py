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
