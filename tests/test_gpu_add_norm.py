"""GPU parity of ttt_add_rms_norm against the fp64 oracle.

Tolerance, element by element. A lane sums at most 64 squares one after the other, then 8 partial sums are
added: with the rounding of each h before it the sum of squares is off by at most 80 half steps of fp32,
2^-24 of itself, its root by half as many, the reciprocal root by 4 more, and three products and h itself
by one each: y is off by at most 50 half steps, and by half a step of its own type. In 8 bits the scale is
off as y is, plus two roundings, and a value by half a step of e4m3: 2^-4 of itself or 2^-10 scales.
S is the fp32 sum rounded once: the same bits."""
import numpy as np
import pytest

import chunked_weight_sequence_amd as ttt
import gen
import oracle.serving as osv
from helpers import dev, host_bits, host_f64, requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

STEP = 2.0 ** -24


def _draw(rng, dtype, *shape, by=1.0):
    x = (by * rng.standard_normal(shape)).astype(np.float32)
    return gen.f32_to_bf16_bits(x) if dtype == "bf16" else x


def _f(x, dtype):
    return gen.bf16_bits_to_f32(x) if dtype == "bf16" else x


def _dequantised(Y, scales, group):
    import torch
    codes = Y.view(torch.uint8).cpu().numpy()
    q = osv.e4m3_values()[codes]
    s = host_f64(scales)
    return q, np.repeat(s, group, axis=1) if group else s[:, None]


def _check(got, x, r, w, eps, dtype, group=None):
    """got: (Y, scales, S); group None: Y in dtype."""
    Y, scales, S = got
    want, _ = osv.add_rms_norm(_f(x, dtype), None if r is None else _f(r, dtype), w, eps)
    if r is not None:
        total = _f(x, dtype) + _f(r, dtype)  # numpy: fp32
        np.testing.assert_array_equal(host_bits(S), gen.f32_to_bf16_bits(total) if dtype == "bf16" else total)
    else:
        assert S is None
    if group is None:
        half = 2.0 ** -8 if dtype == "bf16" else STEP
        bound = (1.01 * half + 50 * STEP) * np.abs(want) + 1e-38
        worst = float((np.abs(host_f64(Y) - want) / bound).max())
    else:
        q, s = _dequantised(Y, scales, group)
        ws = osv.e4m3_scales(want, group)
        ws = np.repeat(ws, group, axis=1) if group else ws[:, None]
        assert (np.abs(s - ws) <= 52 * STEP * ws).all()
        bound = 1.01 * s * np.maximum(2.0 ** -4 * np.abs(want / s), 2.0 ** -10) + 53 * STEP * np.abs(want)
        worst = float((np.abs(q * s - want) / bound).max())
        assert np.abs(q).max() <= 448
    print(f"  {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D", [(1, 8), (1, 2560), (3, 64), (5, 1000), (2, 4096), (7, 4104), (2, 16384), (300, 2560),
                                 (2047, 136), (2048, 136), (4099, 1000), (4100, 520), (5000, 1032), (2100, 4096)])
def test_types_and_sizes(dtype, N, D):
    print(f"case: norm {dtype} {N} x {D}", flush=True)
    rng = np.random.default_rng(N + D)
    x, r = _draw(rng, dtype, N, D), _draw(rng, dtype, N, D, by=3.0)
    w = rng.uniform(-2, 2, D).astype(np.float32)
    _check(ttt.add_rms_norm(dev(x, dtype), dev(w, "f32"), residual=dev(r, dtype)), x, r, w, 1e-6, dtype)
    _check(ttt.add_rms_norm(dev(x, dtype), eps=0.5), x, None, None, 0.5, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D,group", [(1, 2560, 128), (1, 2560, 0), (3, 8, 0), (4, 16, 16), (5, 9728, 128), (5, 9728, 512),
                                       (2, 16384, 32), (2050, 1000, 0), (2050, 544, 32), (4099, 1280, 256), (3, 4224, 64)])
def test_eight_bits(dtype, N, D, group):
    print(f"case: norm e4m3 {dtype} {N} x {D} by {group}", flush=True)
    rng = np.random.default_rng(N + D + group)
    x, r = _draw(rng, dtype, N, D), _draw(rng, dtype, N, D)
    r[:, ::37] = _draw(rng, dtype, *r[:, ::37].shape, by=40.0)  # channels that are far larger
    w = rng.uniform(0.2, 2, D).astype(np.float32)
    got = ttt.add_rms_norm(dev(x, dtype), dev(w, "f32"), residual=dev(r, dtype), e4m3=True, group=group)
    _check(got, x, r, w, 1e-6, dtype, group)


@pytest.mark.parametrize("N", [5, 2053])
@pytest.mark.parametrize("e4m3", [False, True])
def test_values_at_the_ends_of_the_range(N, e4m3):
    """Rows whose squares leave fp32 at either end, rows of zeros, beside ordinary ones."""
    print(f"case: norm, ends of the range, {N} {e4m3}", flush=True)
    rng = np.random.default_rng(3)
    x = rng.standard_normal((N, 640)).astype(np.float32)
    x[0] *= np.float32(2.0 ** 100)
    x[1] *= np.float32(2.0 ** -100)
    x[2] = 0
    x[3, 5:] = 0
    x[3, :5] = [1e30, -1e-30, 1e20, 3, 0]
    w = rng.uniform(0.5, 2, 640).astype(np.float32)
    got = ttt.add_rms_norm(dev(x, "f32"), dev(w, "f32"), eps=0.0 if e4m3 else 1e-30, e4m3=e4m3)
    if e4m3:  # 0 / 0 of the row of zeros: NaN there, and only there
        y, s = host_f64(got[0].float()), host_f64(got[1])
        assert np.isnan(y[2]).all() and s[2] == 2.0 ** -126
        keep = np.arange(N) != 2
        assert np.isfinite(y[keep]).all()
        _check((got[0][keep], got[1][keep], None), x[keep], None, w, 0.0, "f32", 0)
    else:
        _check(got, x, None, w, 1e-30, "f32")


@pytest.mark.parametrize("N,D", [(4, 256), (2100, 256), (4, 4096)])
@pytest.mark.parametrize("size,weight", [(1e15, 1e25), (1e-15, 1e-28), (1e15, 1e-30), (1e-15, 1e30)])
def test_scales_of_weights_far_from_one(N, D, size, weight):
    """The product of a value and its weight may leave fp32 where the norm times the weight does not."""
    print(f"case: norm e4m3 {N} x {D}, values of {size}, weights of {weight}", flush=True)
    rng = np.random.default_rng(N + D)
    x = (size * rng.standard_normal((N, D))).astype(np.float32)
    x[1] = 0.5
    w = (weight * rng.uniform(0.5, 2, D)).astype(np.float32)
    for group in (0, 64):
        _check(ttt.add_rms_norm(dev(x, "f32"), dev(w, "f32"), eps=0.0, e4m3=True, group=group), x, None, w, 0.0, "f32", group)


def test_as_many_rows_as_a_launch_has_threads():
    """Rows times lanes past 2^32: rows of 8 channels, whose sums of squares are exact."""
    import torch
    N = (1 << 26) + 5
    print(f"case: norm, {N} rows", flush=True)
    sign = (torch.arange(N, device="cuda") % 3 - 1).to(torch.bfloat16)  # -1, 0, 1
    x = (2 * sign)[:, None].expand(N, 8).contiguous()
    Y, _, _ = ttt.add_rms_norm(x, eps=2.0 ** -126)
    assert torch.equal(Y, sign[:, None].expand(N, 8))
    Y, s, _ = ttt.add_rms_norm(x, eps=2.0 ** -126, e4m3=True)
    assert torch.equal(s > 2.0 ** -126, sign != 0)
    assert torch.equal(Y.view(torch.uint8)[:, 3], torch.where(sign == 0, 0, torch.where(sign > 0, 0x7E, 0xFE)).to(torch.uint8))


def test_infinities_and_nan_stay_in_their_rows():
    print("case: norm, infinities and NaN", flush=True)
    rng = np.random.default_rng(4)
    x = rng.standard_normal((6, 256)).astype(np.float32)
    clean = x.copy()
    x[1, 7], x[4, 200] = np.inf, np.nan
    for kw in (dict(), dict(e4m3=True), dict(e4m3=True, group=32)):
        y = host_f64(ttt.add_rms_norm(dev(x, "f32"), **kw)[0].float())
        c = host_f64(ttt.add_rms_norm(dev(clean, "f32"), **kw)[0].float())
        for n in (0, 2, 3, 5):
            np.testing.assert_array_equal(y[n], c[n])
        assert np.isnan(y[1, 7]) and (y[1, np.arange(256) != 7] == 0).all()
        assert np.isnan(y[4]).all()


@pytest.mark.parametrize("N", [9, 3000])
def test_slices_and_in_place(N):
    """Rows that are slices of wider buffers; the sum in place of the input or of the residual, the norm in
    place too; what lies between the slices stays."""
    import torch
    print(f"case: norm, slices, {N}", flush=True)
    rng = np.random.default_rng(N)
    D = 328
    wide = _draw(rng, "bf16", N, 3 * D)
    x, r = wide[:, D:2 * D].copy(), _draw(rng, "bf16", N, D)
    w = rng.uniform(0.5, 2, D).astype(np.float32)
    want = ttt.add_rms_norm(dev(x, "bf16"), dev(w, "f32"), residual=dev(r, "bf16"))
    _check(want, x, r, w, 1e-6, "bf16")
    B, R = dev(wide, "bf16"), dev(r, "bf16")
    out = torch.full((N, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    Y, _, S = ttt.add_rms_norm(B[:, D:2 * D], dev(w, "f32"), residual=R, S=B[:, D:2 * D], Y=out[:, :D])
    assert torch.equal(Y, want[0]) and torch.equal(S, want[2]) and (out[:, D:] == 7).all()
    np.testing.assert_array_equal(host_bits(B)[:, :D], wide[:, :D])
    np.testing.assert_array_equal(host_bits(B)[:, 2 * D:], wide[:, 2 * D:])
    X = dev(x, "bf16")
    Y, _, S = ttt.add_rms_norm(X, dev(w, "f32"), residual=R, S=R, Y=X)
    assert S is R and torch.equal(Y, want[0]) and torch.equal(S, want[2])
    q = torch.zeros(N, 2 * D, dtype=torch.float8_e4m3fn, device="cuda")
    Y, s, _ = ttt.add_rms_norm(dev(x, "bf16"), dev(w, "f32"), e4m3=True, Y=q[:, :D])
    _check((Y, s, None), x, None, w, 1e-6, "bf16", 0)
    assert (q[:, D:].view(torch.uint8) == 0).all()


def test_refusals():
    import torch
    print("case: norm refusals", flush=True)
    x = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    h = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    for args, kw, err in [
            ((x.half(),), {}, TypeError), ((x.cpu(),), {}, ValueError), ((x[0],), {}, ValueError),
            ((x.t(),), {}, ValueError), ((x, w[:32]), {}, ValueError), ((x, w.double()), {}, TypeError),
            ((x,), dict(residual=h), TypeError), ((x,), dict(residual=x[:2]), ValueError),
            ((x,), dict(S=x), ValueError), ((x,), dict(Y=h), TypeError), ((x,), dict(group=32), ValueError),
            ((x,), dict(e4m3=True, group=48), ValueError), ((x,), dict(e4m3=True, group=8), ttt.TTTError),
            ((x,), dict(e4m3=True, scales=torch.zeros(5, device="cuda")), ValueError),
            ((x,), dict(e4m3=True, Y=x), TypeError), ((x[:, :60].contiguous(),), {}, ttt.TTTError),
            ((x,), dict(eps=-1.0), ttt.TTTError), ((x,), dict(residual=x.clone(), S=x[:, :]), None),
            ((x[:3],), dict(residual=x[1:]), None), ((x[:3],), dict(residual=x[1:], S=x[1:]), ttt.TTTError)]:
        if err is None:
            ttt.add_rms_norm(*args, **kw)
        else:
            with pytest.raises(err):
                ttt.add_rms_norm(*args, **kw)


def test_values_beside_the_ties_of_eight_bits():
    """Codes are those of the quotient y / scale, rounded once to fp32 and once to e4m3, ties to even. Rows of +1 and
    -1 have a mean square of 1 and with eps = 0 a factor of exactly 1, so y is the weight with the row's signs, and
    the weights here are the fp32 numbers at and beside scale * (the middle between two codes)."""
    import torch
    rng = np.random.default_rng(21)
    values = osv.e4m3_values()
    up = np.unique(np.abs(values[np.isfinite(values)]))  # 0 .. 448
    middle = (up[1:] + up[:-1]) / 2
    for top in (1.0, 3.7, 0.0123, 448.0, 1e-20, 7e30, 1e-30, 1e36):
        print(f"case: norm e4m3, values beside ties, the largest {top}", flush=True)
        top = np.float32(top)
        scale = np.float32(top / np.float32(448))
        at = (middle * np.float64(scale)).astype(np.float32)
        w = np.concatenate([at, np.nextafter(at, np.float32(0)), np.nextafter(at, np.float32(np.inf))])
        w = np.concatenate([w[w < top], np.full(512, top, np.float32)])[:512]
        w = rng.permutation(w).astype(np.float32)
        w[::128] = top  # every group's scale is the row's
        x = np.where(rng.random((3, 512)) < 0.5, -1, 1).astype(np.float32)
        q = (np.abs(w) / scale).astype(np.float64)  # fp32 quotients
        lo = np.clip(np.searchsorted(up, q, side="right") - 1, 0, len(up) - 1)
        hi = np.minimum(lo + 1, len(up) - 1)
        d = (q - up[lo]) - (up[hi] - q)
        code = np.where((d > 0) | ((d == 0) & (lo % 2 == 1)), hi, lo)  # codes of the sizes are their numbers
        for dtype in ("f32", "bf16"):
            xs = dev(x if dtype == "f32" else gen.f32_to_bf16_bits(x), dtype)
            for group in (0, 128):
                Y, s, _ = ttt.add_rms_norm(xs, dev(w, "f32"), eps=0.0, e4m3=True, group=group)
                assert (host_f64(s) == np.float64(scale)).all()
                got = Y.view(torch.uint8).cpu().numpy()
                np.testing.assert_array_equal(got & 127, np.broadcast_to(code, got.shape))
                np.testing.assert_array_equal(got >> 7 == 1, x < 0)
