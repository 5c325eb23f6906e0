"""Packed and one-token attention at the ends of their ranges, against the fp64 oracle: values near the
type's largest, scales near zero, logits past fp32, rows of very many keys, values that a row does not
see. Tolerances as in test_gpu_attention.py, where a test does not derive its own."""
import numpy as np
import pytest

import chunked_weight_sequence_amd as ttt
import gen
import oracle.attention as oa
from helpers import dev, host_bits, host_f64, requires_gpu
import test_gpu_norm_rope as norm_rope
from test_gpu_attention import _cache, _check, _cu, _draw, _f, _i32, _logit_size, _packed, _seen, _some_rows

pytestmark = [pytest.mark.gpu, requires_gpu]


def _large(rng, *shape):
    """Finite values of either sign up to 3.3e38 (bf16 ends at 3.39e38); channel 0 all of one sign."""
    x = rng.uniform(-3.3e38, 3.3e38, shape)
    x[..., 0] = rng.uniform(3.2e38, 3.3e38, shape[:-1])
    return gen.f32_to_bf16_bits(x.astype(np.float32))


@pytest.mark.parametrize("lq,more,Hq,Hkv,dh,window", [
    ([150], [0], 4, 2, 128, 0), ([90, 130], [30, 0], 3, 1, 64, 50),
    ([40], [3000], 2, 1, 128, 0), ([40], [3000], 2, 1, 64, 0),  # keys split, few pieces
    ([2], [9000], 4, 4, 128, 0),                                # keys split, many pieces
    ([4200], [0], 30, 15, 128, 0),                              # 256 rows to a workgroup
    ([256], [4200], 64, 8, 128, 0)])                            # the same, keys split
def test_packed_sums_of_large_values_stay_finite(lq, more, Hq, Hkv, dh, window):
    """A weighted mean of finite values is finite, although their sum before the division is not."""
    print(f"case: packed large values lq={lq} more={more} {Hq}/{Hkv}x{dh} window={window}", flush=True)
    rng = np.random.default_rng(sum(lq) + dh)
    cu_q, cu_k = _cu(lq), _cu(np.array(lq) + np.array(more))
    Q, K, V = _draw(rng, cu_q[-1], Hq, dh), _draw(rng, cu_k[-1], Hkv, dh), _large(rng, cu_k[-1], Hkv, dh)
    scale = dh ** -0.5
    O, L = _packed(Q, K, V, cu_q, cu_k, scale, window)
    tokens = sorted({0, 1, int(cu_q[-1]) - 1, *rng.integers(0, cu_q[-1], 30).tolist()})
    heads = sorted({0, Hq // 2, Hq - 1})
    q, k, v = _f(Q), _f(K), _f(V)
    _check(O[tokens][:, heads], L[tokens][:, heads],
           _some_rows(q, k, v, cu_q, cu_k, scale, window, tokens, heads),
           _logit_size(q[tokens], k, scale)[:, heads], dh, "large values")
    assert np.isfinite(host_f64(O)).all()


def test_packed_a_large_value_behind_the_first_maximum():
    """Weights relative to the first tile's maximum may reach 2^8: 2^7.8 times 2e36 passes fp32."""
    print("case: packed, large value in a later tile", flush=True)
    N, dh = 200, 64
    Q, K, V = (np.zeros((N, 1, dh)) for _ in range(3))
    Q[:, 0, 0], K[150, 0, 0], V[150, 0, 3] = 1.0, 5.40625, 2.0 ** 120.5
    Q, K, V = (gen.f32_to_bf16_bits(x.astype(np.float32)) for x in (Q, K, V))
    O, L = _packed(Q, K, V, [0, N], [0, N], 1.0, 0)
    _check(O, L, oa.packed(_f(Q), _f(K), _f(V), [0, N], [0, N], 1.0),
           _logit_size(_f(Q), _f(K), 1.0), dh, "later tile")


@pytest.mark.parametrize("lens,page,Hq,Hkv,dh", [
    ([0, 1, 33, 300], 16, 4, 4, 64), ([500, 129, 1000], 64, 14, 2, 128), ([2000], 256, 8, 8, 128),
    ([400, 0, 399, 1] * 25, 16, 32, 16, 128)])                  # two waves to a workgroup
def test_decode_sums_of_large_values_stay_finite(lens, page, Hq, Hkv, dh):
    import torch
    print(f"case: decode large values lens={lens[:8]} {Hq}/{Hkv}x{dh}", flush=True)
    rng = np.random.default_rng(sum(lens) + dh)
    Kc, Vc, table = _cache(rng, lens, page, Hkv, dh)
    Vc = np.where(Vc == 0x7F80, Vc, _large(rng, *Vc.shape))
    Q, scale = _draw(rng, len(lens), Hq, dh), dh ** -0.5
    O, L = ttt.attention_decode(dev(Q, "bf16"), dev(Kc, "bf16"), dev(Vc, "bf16"), _i32(table),
                                _i32(lens), page, scale=scale, with_lse=True)
    torch.cuda.synchronize()
    some = list(range(min(len(lens), 4)))
    want = oa.decode(_f(Q[some]), _f(Kc), _f(Vc), table[some], np.array(lens)[some], page, scale)
    X = scale * np.abs(_f(Q[some])).sum(-1) * _seen(Kc, table[some], np.array(lens)[some], page)
    _check(O[some], L[some], want, X, dh, "large values")
    assert np.isfinite(host_f64(O)).all()


@pytest.mark.parametrize("scale", [1e-38, 1e-40, 2.0 ** -149, 1e-30])
@pytest.mark.parametrize("Nq,Nk,Hq,Hkv,dh,window", [(300, 300, 4, 2, 128, 20), (200, 150, 2, 1, 64, 30),
                                                    (40, 3000, 2, 1, 128, 700), (4200, 4200, 30, 15, 128, 2500)])
def test_packed_scales_near_zero(Nq, Nk, Hq, Hkv, dh, window, scale):
    """All visible keys weigh the same: also for rows that see nothing of their first tile, whose window
    begins behind it."""
    print(f"case: packed scale={scale} {Nq}/{Nk} {Hq}/{Hkv}x{dh} window={window}", flush=True)
    rng = np.random.default_rng(Nq)
    Q, K, V = _draw(rng, Nq, Hq, dh), _draw(rng, Nk, Hkv, dh), _draw(rng, Nk, Hkv, dh)
    scale = float(np.float32(scale))
    O, L = _packed(Q, K, V, [0, Nq], [0, Nk], scale, window)
    tokens, heads = sorted({*range(0, Nq, max(1, Nq // 60)), Nq - 1}), sorted({0, Hq - 1})
    want = _some_rows(_f(Q), _f(K), _f(V), [0, Nq], [0, Nk], scale, window, tokens, heads)
    _check(O[tokens][:, heads], L[tokens][:, heads], want,
           _logit_size(_f(Q[tokens]), _f(K), scale)[:, heads], dh, "small scale")


def test_decode_scales_near_zero():
    import torch
    print("case: decode scales near zero", flush=True)
    rng = np.random.default_rng(12)
    lens, page, Hq, Hkv, dh = [70, 0, 900], 16, 4, 2, 64
    Kc, Vc, table = _cache(rng, lens, page, Hkv, dh)
    Q = _draw(rng, 3, Hq, dh)
    for scale in (1e-38, 2.0 ** -149, 1e-30):
        scale = float(np.float32(scale))
        O, L = ttt.attention_decode(dev(Q, "bf16"), dev(Kc, "bf16"), dev(Vc, "bf16"), _i32(table),
                                    _i32(lens), page, scale=scale, with_lse=True)
        torch.cuda.synchronize()
        X = scale * np.abs(_f(Q)).sum(-1) * _seen(Kc, table, lens, page)
        _check(O, L, oa.decode(_f(Q), _f(Kc), _f(Vc), table, lens, page, scale), X, dh, "small scale")


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("Nq,Nk,dh", [(70, 70, 64), (40, 3000, 128)])
def test_logits_past_fp32_are_not_taken_for_masked_ones(Nq, Nk, dh, sign):
    """A logit of 2.6e38 is finite, times log2(e) it is not in fp32: the row is NaN, never o = 0 with
    lse = -inf, which says that it sees nothing."""
    import torch
    print(f"case: logits of {sign} 2.6e38, {Nq}/{Nk}x{dh}", flush=True)
    Q, K = (np.zeros((n, 1, dh), np.float32) for n in (Nq, Nk))
    Q[..., 0], K[..., 0] = 1.6e19, sign * 1.6e19
    Q, K = gen.f32_to_bf16_bits(Q), gen.f32_to_bf16_bits(K)
    V = _draw(np.random.default_rng(1), Nk, 1, dh)
    O, L = _packed(Q, K, V, [0, Nq], [0, Nk], 1.0, 0)
    assert np.isnan(host_f64(O)).all() and not np.isneginf(host_f64(L)).any()
    page = 16
    Kc, Vc = (dev(x[:Nk // page * page], "bf16") for x in (K, V))
    table = _i32(np.arange(Nk // page)[None])
    O, L = ttt.attention_decode(dev(Q[:1], "bf16"), Kc, Vc, table, _i32([Nk // page * page]), page,
                                scale=1.0, with_lse=True)
    torch.cuda.synchronize()
    assert np.isnan(host_f64(O)).all() and not np.isneginf(host_f64(L)).any()


@pytest.mark.parametrize("scale", [0.9, 1.3, 1.7])
def test_decode_sums_of_many_equal_weights(scale):
    """262144 tokens in one piece, all with one logit: the weights of all tiles are the same, however
    many tiles pass without a new maximum. The sums are 4 of 2048 tiles' each: an addition is off by half
    a step of the sum, so a mean by 2048 2^-24 at most, and lse by 2048 2^-24 beside _check's terms."""
    import torch
    print(f"case: decode, many equal weights, scale {scale}", flush=True)
    S, Hkv, dh, page, n = 128, 8, 64, 64, 1 << 18
    g = torch.Generator(device="cuda").manual_seed(3)
    V = torch.randn((n, Hkv, dh), generator=g, device="cuda").to(torch.bfloat16)
    V[: n // 2, :, 0], V[n // 2:, :, 0] = 1.0, -1.0  # early against late tokens: mean 0
    key = _draw(np.random.default_rng(2), 1, Hkv, dh)
    K = dev(key, "bf16").expand(n, Hkv, dh).contiguous()
    q = _draw(np.random.default_rng(4), S, Hkv, dh, by=8.0)
    table = torch.arange(n // page, dtype=torch.int32, device="cuda").expand(S, n // page).contiguous()
    lens = np.ones(S, np.int32)
    lens[:3] = n
    assert ttt.lib().ttt_attention_decode_workspace(S, n // page, page, Hkv, Hkv, dh) == 0  # one piece
    O, L = ttt.attention_decode(dev(q, "bf16"), K, V, table, _i32(lens), page, scale=scale, with_lse=True)
    torch.cuda.synchronize()
    x = scale * (_f(q[:3]) * _f(key)).sum(-1)
    mean = V.double().mean(0).cpu().numpy()
    size = V.double().abs().mean(0).cpu().numpy()
    X = scale * (np.abs(_f(q[:3])) * np.abs(_f(key))).sum(-1)
    d = (dh + 4) * 2.0 ** -24 * X + 2048 * 2.0 ** -24
    off = np.abs(host_f64(L[:3]) - (x + np.log(n)))
    bound = d + 2.0 ** -20 + 4 * 2.0 ** -24 * (np.abs(x) + np.log(n) + X)
    print(f"  lse {float((off / bound).max()):.3f}", flush=True)
    ob = 1.01 * (2.0 ** -8 * (np.abs(mean) + size) + (4 * d[..., None] + 2.0 ** -19) * size)
    # equal weights are rounded alike: the mean of channel 0 holds no rounding of bf16 weights
    ob[..., 0] = 4 * 2048 * 2.0 ** -24
    o = float((np.abs(host_f64(O[:3]) - mean) / ob).max())
    print(f"  o {o:.3f}, channel 0 {np.abs(host_f64(O[:3, :, 0])).max():.2e}", flush=True)
    assert (off <= bound).all() and o <= 1.0


def test_packed_sums_of_many_equal_weights():
    """2^20 keys of one logit but for a larger one in the first tile, one piece: each lane adds up some
    2^18 equal weights. In sums of whole tiles (16384 of them) each addition is off by half a step: lse by
    16384 / 2 2^-24 on the mean of a growing sum, doubled for what the tiles' own 16 additions lose."""
    import torch
    print("case: packed, many equal weights", flush=True)
    Nq, Nk, Hq, dh = 256, 1 << 20, 128, 64
    K = torch.zeros(Nk, 1, dh, dtype=torch.bfloat16, device="cuda")
    K[0, 0, 0] = 1.0
    V = torch.ones_like(K)
    q = torch.zeros(Nq, Hq, dh, dtype=torch.bfloat16, device="cuda")
    top = torch.linspace(0.1, 2.0, Hq, device="cuda").to(torch.bfloat16)
    q[..., 0] = top
    O, L = ttt.attention_packed(q, K, V, _i32([0, Nq]), _i32([0, Nk]), scale=1.0, with_lse=True)
    torch.cuda.synchronize()
    x = top.double().cpu().numpy()[None]
    seen = Nk - Nq + 1 + np.arange(Nq)[:, None]  # keys of a row, the larger one among them
    want = np.log(np.exp(x) + seen - 1)
    off = np.abs(host_f64(L) - want).max()
    print(f"  lse off by {off:.2e}", flush=True)
    assert off <= 16384 * 2.0 ** -24 + 2.0 ** -20 + 8 * 2.0 ** -24 * 16
    # bf16(weight) / weight: at most 2^-8 off, and the result's own rounding
    assert np.abs(host_f64(O) - 1).max() <= 2.0 ** -7 + 2 * 16384 * 2.0 ** -24


@pytest.mark.parametrize("bad", [np.inf, np.nan])
@pytest.mark.parametrize("lq,more,Hq,Hkv,dh,window", [
    ([150], [0], 4, 2, 128, 0), ([150], [0], 4, 2, 64, 0), ([90, 130], [30, 0], 3, 1, 64, 50),
    ([40], [3000], 2, 1, 128, 0), ([40], [3000], 2, 1, 128, 1000),   # the keys are split
    ([4200], [0], 30, 15, 128, 0), ([1000], [3000], 64, 32, 128, 2500),  # 256 rows to a workgroup
    ([256], [4200], 64, 8, 128, 0)])                                 # the same, split
def test_packed_hidden_values_leave_the_bits_of_other_channels(lq, more, Hq, Hkv, dh, window, bad):
    """Beside an infinity or NaN the 32 channels that hold it may be summed again, at another reference
    maximum: every other channel, and every row of other heads and sequences, keeps its bits. The logits
    rise, so that weights are taken at several maxima."""
    print(f"case: packed hidden {bad}, bits, lq={lq} more={more} {Hq}/{Hkv}x{dh} window={window}", flush=True)
    rng = np.random.default_rng(sum(lq) + dh)
    cu_q, cu_k = _cu(lq), _cu(np.array(lq) + np.array(more))
    Q, K = _draw(rng, cu_q[-1], Hq, dh), _draw(rng, cu_k[-1], Hkv, dh)
    K = gen.f32_to_bf16_bits((_f(K) * np.linspace(0.2, 6, len(K))[:, None, None]).astype(np.float32))
    V = _draw(rng, cu_k[-1], Hkv, dh)
    at = int(cu_k[1]) - lq[0] // 2  # a key in the middle of the first sequence's own part
    V1 = V.copy()
    V1[at, 0, 5] = gen.f32_to_bf16_bits(np.float32([bad]))[0]
    want, got = (_packed(Q, K, v, cu_q, cu_k, dh ** -0.5, window) for v in (V, V1))
    np.testing.assert_array_equal(host_bits(got[1]), host_bits(want[1]))
    want, got = host_bits(want[0]), host_bits(got[0])
    last = np.arange(lq[0]) + more[0]
    sees = (last >= at) & ((last - at < window) if window else True)
    off = np.zeros(got.shape, bool)
    off[:lq[0], :Hq // Hkv, :32] = True
    assert 0 < sees.sum() < lq[0]
    np.testing.assert_array_equal(got[~off], want[~off])
    assert not np.isfinite(gen.bf16_bits_to_f32(got[:lq[0]][sees][:, :Hq // Hkv, 5])).any()


@pytest.mark.parametrize("layout,dh,rot", [("half", 64, 64), ("interleaved", 64, 16), ("half", 256, 128)])
def test_fp32_rotations_are_rounded_once(layout, dh, rot):
    """The pair (1, 0) turns into the cosine and the sine: half a step of fp32 from the exact ones, beside
    the fp64 angle's own error (2^20 times 2^-52 in radians)."""
    import torch
    print(f"case: fp32 rotation of (1, 0), {layout} {rot} of {dh}", flush=True)
    rng = np.random.default_rng(rot)
    N, half = 2000, rot // 2
    pos = np.concatenate([rng.integers(0, 1 << 20, N - 4), [0, 1, -7, (1 << 20) - 1]])
    a = np.arange(half) if layout == "half" else 2 * np.arange(half)
    b = a + half if layout == "half" else a + 1
    x = np.zeros((N, 1, dh), np.float32)
    x[:, 0, a] = 1
    freq, _ = oa.rope_frequencies(rot, 10000.0)
    Q, _ = ttt.qk_norm_rope(dev(x, "f32"), dev(x, "f32"), _i32(pos), torch.tensor(freq, device="cuda"),
                            layout=layout)
    torch.cuda.synchronize()
    got, angle = host_f64(Q)[:, 0], pos[:, None] * freq
    for at, want in ((a, np.cos(angle)), (b, np.sin(angle))):
        off = np.abs(got[:, at] - want) / (2.0 ** -24 * np.abs(want) + 2.0 ** -31)
        print(f"  {off.max():.3f} of the bound", flush=True)
        assert off.max() <= 1.0


@pytest.mark.parametrize("N,Hq,Hkv,dh,rot,layout,dtype,norm,first,scale", [
    (1024, 8, 2, 64, 32, "half", "bf16", "qk", 0, 1.0),        # four waves to a token, at most
    (1025, 8, 4, 64, 32, "half", "bf16", "qk", 0, 1.0),        # two
    (1025, 3, 3, 128, 16, "interleaved", "f32", "q", 77, 1.1),
    (2048, 8, 4, 64, 32, "half", "f32", "k", 0, 1.0)])
@pytest.mark.parametrize("how", ["plain", "in place"])
def test_norm_and_rotation_with_fewer_waves_to_a_token(N, Hq, Hkv, dh, rot, layout, dtype, norm, first,
                                                       scale, how):
    norm_rope.test_norm_and_rotation(N, Hq, Hkv, dh, rot, layout, dtype, norm, first, scale, how)


@pytest.mark.parametrize("Hq,Hkv,dh,more", [(32, 16, 64, 0), (32, 16, 128, 0), (20, 10, 128, 100)])
def test_packed_sequences_taken_longest_first(Hq, Hkv, dh, more):
    """Enough workgroups for that order; unlike lengths, two alike, empty sequences, rows of none."""
    import torch
    print(f"case: packed longest first {Hq}/{Hkv}x{dh} past {more}", flush=True)
    rng = np.random.default_rng(dh + more)
    lq = [0, 900, 33, 0, 1500, 128, 1, 900, 0]
    cu_q, cu_k = _cu(lq, 5), _cu([n + more * (n > 0) for n in lq], 3)
    Nq, Nk = cu_q[-1] + 7, cu_k[-1] + 2
    Q, K, V = _draw(rng, Nq, Hq, dh), _draw(rng, Nk, Hkv, dh), _draw(rng, Nk, Hkv, dh)
    O = torch.full((Nq, Hq, dh), 7.0, dtype=torch.bfloat16, device="cuda")
    L = torch.full((Nq, Hq), 7.0, device="cuda")
    _packed(Q, K, V, cu_q, cu_k, dh ** -0.5, 0, O=O, lse=L)
    for x in (O[:5], O[-7:], L[:5], L[-7:]):
        assert (x == 7).all()
    on = slice(5, -7)
    assert not (O[on] == 7).all(-1).any() and not (L[on] == 7).any()  # every row is written
    tokens = sorted({*(cu_q[:-1][np.diff(cu_q) > 0]).tolist(), *(cu_q[1:][np.diff(cu_q) > 0] - 1).tolist(),
                     *rng.integers(5, Nq - 7, 20).tolist()})
    heads = [0, 1, Hq - 1]
    q, k, v = _f(Q), _f(K), _f(V)
    _check(O[tokens][:, heads], L[tokens][:, heads],
           _some_rows(q, k, v, cu_q, cu_k, dh ** -0.5, 0, tokens, heads),
           _logit_size(q[tokens], k, dh ** -0.5)[:, heads], dh, "longest first")


def test_a_call_on_another_stream_without_torchs_own_functions(monkeypatch):
    """The public way to the stream gives the same handle, and a call through it the same bits."""
    import torch
    print("case: streams by the public interface", flush=True)
    current, stream = ttt._device_calls.__wrapped__(object())
    own = ttt._device_calls()
    side = torch.cuda.Stream()
    rng = np.random.default_rng(20)
    q, k, v = (dev(_draw(rng, 50, 2, 64), "bf16") for _ in range(3))
    want = host_bits(ttt.attention_packed(q, k, v, _i32([0, 50])))
    torch.cuda.synchronize()
    for s in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(s):
            assert current() == own[0]() == 0 and stream(0) == own[1](0) == s.cuda_stream
            monkeypatch.setattr(ttt, "_device_calls", lambda: (current, stream))
            got = ttt.attention_packed(q, k, v, _i32([0, 50]))
            monkeypatch.undo()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(host_bits(got), want)


def test_tensors_of_other_ranks_are_refused():
    import torch
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu, n = _i32([0, 4]), _i32([4] * 4)
    for bad in (cu[0], cu[None]):
        with pytest.raises(ValueError):
            ttt.attention_packed(q, q, q, bad)
        with pytest.raises(ValueError):
            ttt.attention_packed(q, q, q, cu, bad)
    f = torch.zeros(0, dtype=torch.float64, device="cuda")
    for bad in (q[0, 0, 0], q[0, 0], q[0], q[None]):
        with pytest.raises(ValueError):
            ttt.attention_decode(q, bad, q, _i32([[0]] * 4), n, 16)
        with pytest.raises(ValueError):
            ttt.attention_packed(q, bad, q, cu)
        with pytest.raises(ValueError):
            ttt.qk_norm_rope(q.clone(), q.clone(), _i32([0] * 4), f, V=q, K_cache=bad, V_cache=q, slots=n)


@pytest.mark.parametrize("dh,more,sign", [(64, 0, 1), (128, 0, -1), (128, 3000, 1)])
def test_means_of_the_largest_value_are_that_value(dh, more, sign):
    """Keys that all weigh the same and all hold bf16's largest value: however their weights round, the
    result does not pass it."""
    import torch
    print(f"case: largest values, dh {dh}, past {more}", flush=True)
    N, top = 300, float(torch.finfo(torch.bfloat16).max)
    Q = torch.zeros(N, 2, dh, dtype=torch.bfloat16, device="cuda")
    K = torch.zeros(N + more, 1, dh, dtype=torch.bfloat16, device="cuda")
    V = torch.full_like(K, sign * top)
    O = host_f64(ttt.attention_packed(Q, K, V, _i32([0, N]), _i32([0, N + more])))
    # every row: half a step of the weights, then of the result
    assert np.isfinite(O).all() and (np.abs(O - sign * top) <= 2.0 ** -7 * top).all()
    lens, page = list(range(1, 200)) + [more + N], 16
    pages = -(-(more + N) // page)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(len(lens), pages).contiguous()
    C, D = (torch.zeros(pages * page, 1, dh, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    D.fill_(sign * top)
    q = torch.zeros(len(lens), 2, dh, dtype=torch.bfloat16, device="cuda")
    O = host_f64(ttt.attention_decode(q, C, D, table, _i32(lens), page))
    torch.cuda.synchronize()
    assert np.isfinite(O).all() and (np.abs(O - sign * top) <= 2.0 ** -7 * top).all()
