"""GPU parity of ttt_qk_norm_rope against the fp64 oracle: both layouts and types, partial heads,
head sizes off the powers of two, far positions, strided and in-place calls, the cache write with
skipped slots, and what the binding refuses.

Tolerance, element by element, for y = r (a c - b s) w with |c|, |s| <= rope_scale: the sum of
squares of dh terms in fp32 is off by at most (dh / L + log2 L + 1) half steps (relative; L lanes),
half of that in its root; the root, the product by the weight, the rotation's products and sum and
the sine add a few half steps each, and the angle, a fraction of a turn in fp32, 2 pi 2^-25. With
n = dh / 2 + 32 half steps of fp32 relative to rope_scale (|a| + |b|) all of it is covered; the
output's rounding adds half a step of its type relative to the value."""
import numpy as np
import pytest

import chunked_weight_sequence_amd as ttt
import gen
import oracle.attention as oa
from helpers import dev, host_bits, host_f64, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]


def _draw(rng, shape, dtype):
    x = (1.5 * rng.standard_normal(shape)).astype(np.float32)
    return gen.f32_to_bf16_bits(x) if dtype == "bf16" else x


def _f(x):
    return (gen.bf16_bits_to_f32(x) if x.dtype == np.uint16 else x).astype(np.float64)


def _bound(X, w, eps, rot, layout, scale, want, dtype):
    """Allowed |error|, see the module's text."""
    y = np.abs(oa.norm_rope(X, w, eps, np.zeros(len(X)), np.zeros(0), layout, 1.0))
    mag, half, dh = y.copy(), rot // 2, X.shape[-1]
    a, b = ((slice(0, half), slice(half, rot)) if layout == "half"
            else (slice(0, rot, 2), slice(1, rot, 2)))
    mag[..., a] = mag[..., b] = max(1.0, scale) * (y[..., a] + y[..., b])
    return ((dh / 2 + 32) * 2.0 ** -24 * mag +
            (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(want) * 1.01)


def _check(got, want, bound, what):
    off = np.abs(host_f64(got) - want)
    worst = float((off / np.maximum(bound, 1e-300)).max())
    print(f"  {what}: largest error {worst:.3f} of its bound", flush=True)
    assert np.isfinite(host_f64(got)).all() and worst <= 1.0, what


CASES = [
    # N, Hq, Hkv, dh, rot, layout, dtype, norm, first position, rope_scale
    (1, 32, 8, 128, 128, "half", "bf16", "qk", 40000, 1.0),
    (1, 1, 1, 16, 16, "interleaved", "f32", "qk", 0, 1.0),
    (5, 3, 2, 80, 48, "half", "bf16", "qk", 100, 1.2),
    (7, 14, 2, 64, 64, "interleaved", "bf16", "q", -3, 1.0),
    (3, 5, 5, 112, 16, "interleaved", "f32", "k", 1 << 20, 1.0),
    (6, 2, 1, 256, 256, "half", "f32", "", (1 << 31) - 9, 0.7),
    (9, 4, 4, 96, 0, "half", "bf16", "qk", 5, 1.0),
    (2049, 4, 1, 64, 32, "half", "bf16", "qk", 1 << 18, 1.0),   # one wave per token
    (2050, 3, 2, 48, 48, "interleaved", "f32", "qk", 0, 1.0),
]


@pytest.mark.parametrize("N,Hq,Hkv,dh,rot,layout,dtype,norm,first,scale", CASES)
@pytest.mark.parametrize("how", ["plain", "slices", "in place"])
def test_norm_and_rotation(N, Hq, Hkv, dh, rot, layout, dtype, norm, first, scale, how):
    import torch
    print(f"case: N={N} {Hq}/{Hkv}x{dh} rot={rot} {layout} {dtype} norm={norm!r} {how}", flush=True)
    rng = np.random.default_rng(N + dh)
    row = _draw(rng, (N, (Hq + 2 * Hkv) * dh), dtype)
    Qh = row[:, :Hq * dh].reshape(N, Hq, dh)
    Kh = row[:, Hq * dh:(Hq + Hkv) * dh].reshape(N, Hkv, dh)
    qw = rng.uniform(0.5, 1.5, dh).astype(np.float32) if "q" in norm else None
    kw = rng.uniform(0.5, 1.5, dh).astype(np.float32) if "k" in norm else None
    pos = first + np.arange(N)
    inv, _ = oa.rope_frequencies(max(rot, 2), 1e4)
    inv = inv[:rot // 2]
    R = dev(row, dtype)
    if how == "plain":
        Q, K = dev(Qh, dtype), dev(Kh, dtype)
        out = {}
    else:
        Q = R[:, :Hq * dh].view(N, Hq, dh)
        K = R[:, Hq * dh:(Hq + Hkv) * dh].view(N, Hkv, dh)
        out = dict(Q_out=Q, K_out=K) if how == "in place" else {}
    q, k = ttt.qk_norm_rope(
        Q, K, torch.from_numpy(pos.astype(np.int32)).cuda(), torch.from_numpy(inv).cuda(),
        q_weight=None if qw is None else dev(qw, "f32"),
        k_weight=None if kw is None else dev(kw, "f32"), eps=1e-5, layout=layout, rope_scale=scale,
        **out)
    torch.cuda.synchronize()
    for got, X, w, what in ((q, _f(Qh), qw, "Q"), (k, _f(Kh), kw, "K")):
        want = oa.norm_rope(X, w, 1e-5, pos, inv, layout, scale)
        _check(got, want, _bound(X, w, 1e-5, rot, layout, scale, want, dtype), what)
    if how == "in place":
        assert q.data_ptr() == R.data_ptr()
        np.testing.assert_array_equal(host_bits(R)[:, (Hq + Hkv) * dh:], row[:, (Hq + Hkv) * dh:])
    if how == "slices":
        np.testing.assert_array_equal(host_bits(R), row)


@pytest.mark.parametrize("N,dtype", [(1, "bf16"), (13, "f32"), (130, "bf16"), (2500, "bf16")])
def test_cache_write_and_skipped_slots(N, dtype):
    import torch
    Hq, Hkv, dh, n_slots = 6, 2, 64, 3000
    print(f"case: cache write N={N} {dtype}", flush=True)
    rng = np.random.default_rng(N)
    Q, K, V = (_draw(rng, (N, h, dh), dtype) for h in (Hq, Hkv, Hkv))
    if dtype == "bf16":
        V.reshape(-1)[:3] = [0x7FC1, 0xFF80, 0x8000]  # NaN, -inf and -0 are copied as they are
    Kc, Vc = _draw(rng, (n_slots, Hkv, dh), dtype), _draw(rng, (n_slots, Hkv, dh), dtype)
    slots = rng.permutation(n_slots)[:N].astype(np.int32)
    for i, bad in zip(range(2, N, 5), [-1, n_slots, -(1 << 31), (1 << 31) - 1] * N):
        slots[i] = bad
    inv, _ = oa.rope_frequencies(64, 1e4)
    pos = torch.arange(N, dtype=torch.int32, device="cuda") + 17
    d = [dev(x, dtype) for x in (Q, K, V, Kc, Vc)]
    args = (pos, torch.from_numpy(inv).cuda())
    w = dict(q_weight=dev(np.ones(dh, np.float32), "f32"), k_weight=None)
    q0, k0 = ttt.qk_norm_rope(d[0], d[1], *args, **w)
    q, k = ttt.qk_norm_rope(d[0], d[1], *args, **w, V=d[2], K_cache=d[3], V_cache=d[4],
                            slots=torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    assert torch.equal(q, q0) and torch.equal(k, k0)
    on = (slots >= 0) & (slots < n_slots)
    Kw, Vw = Kc.copy(), Vc.copy()
    Kw[slots[on]], Vw[slots[on]] = host_bits(k)[on], V[on]
    np.testing.assert_array_equal(host_bits(d[3]).view(Kw.dtype), Kw)
    np.testing.assert_array_equal(host_bits(d[4]).view(np.uint8), Vw.view(np.uint8))


def test_bad_values_stay_in_their_head():
    import torch
    rng = np.random.default_rng(5)
    Q = _draw(rng, (4, 3, 64), "f32")
    ref = Q.copy()
    Q[1, 1, 40] = np.nan
    Q[2, 0, 3] = np.inf
    inv, _ = oa.rope_frequencies(32, 1e4)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    w = dev(np.ones(64, np.float32), "f32")
    for weight in (None, w):
        outs = [host_f64(ttt.qk_norm_rope(dev(x, "f32"), dev(ref, "f32"), pos,
                                          torch.from_numpy(inv).cuda(), q_weight=weight)[0])
                for x in (Q, ref)]
        same = np.ones((4, 3), bool)
        same[1, 1] = same[2, 0] = False
        np.testing.assert_array_equal(outs[0][same], outs[1][same])
    # without a norm, channels past the rotated ones are copies
    np.testing.assert_array_equal(
        host_bits(ttt.qk_norm_rope(dev(Q, "f32"), dev(ref, "f32"), pos,
                                   torch.from_numpy(inv).cuda())[0])[..., 32:].view(np.uint32),
        Q[..., 32:].view(np.uint32))


@pytest.mark.parametrize("case", ["k_dtype", "pos_dtype", "pos_len", "inv_dtype", "weight_dtype",
                                  "weight_len", "layout", "slots_alone", "cache_shape", "cache_alone",
                                  "out_shape", "heads_apart", "pos_cpu", "rot"])
def test_binding_refusals(case):
    import torch
    N, H, dh = 4, 2, 64
    Q = torch.zeros(N, H, dh, dtype=torch.bfloat16, device="cuda")
    K, pos = Q.clone(), torch.zeros(N, dtype=torch.int32, device="cuda")
    inv, kw = torch.zeros(32, dtype=torch.float64, device="cuda"), {}
    C = torch.zeros(8, H, dh, dtype=torch.bfloat16, device="cuda")
    if case == "k_dtype":
        K = K.float()
    elif case == "pos_dtype":
        pos = pos.long()
    elif case == "pos_len":
        pos = pos[:3]
    elif case == "inv_dtype":
        inv = inv.float()
    elif case == "weight_dtype":
        kw["q_weight"] = torch.ones(dh, dtype=torch.bfloat16, device="cuda")
    elif case == "weight_len":
        kw["k_weight"] = torch.ones(dh - 1, device="cuda")
    elif case == "layout":
        kw["layout"] = "other"
    elif case == "slots_alone":
        kw["slots"] = pos
    elif case == "cache_shape":
        kw.update(slots=pos, V=K, K_cache=C, V_cache=C[:4])
    elif case == "cache_alone":
        kw["K_cache"] = C
    elif case == "out_shape":
        kw["Q_out"] = Q[:3]
    elif case == "heads_apart":
        Q = torch.zeros(N, 2 * H, dh, dtype=torch.bfloat16, device="cuda")[:, ::2]
    elif case == "pos_cpu":
        pos = pos.cpu()
    elif case == "rot":
        inv = inv[:12].clone()  # 24 channels
    with pytest.raises((ValueError, TypeError, ttt.TTTError)):
        ttt.qk_norm_rope(Q, K, pos, inv, **kw)
