"""Pins of the attention oracle (oracle/attention.py) against facts fixed by the formulas, and the
library's host function ttt_rope_frequencies against it (no GPU)."""
import ctypes
import math

import numpy as np
import pytest

import chunked_weight_sequence_amd as ttt
import oracle.attention as oa


def _x(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_keeps_norms_and_depends_on_distances_only(layout):
    f, _ = oa.rope_frequencies(16, 1e4)
    q, k = _x(1, 1, 24), _x(1, 1, 24, seed=1)

    def at(x, p):
        return oa.norm_rope(x, None, 0.0, [p], f, layout, 1.0)
    np.testing.assert_array_equal(at(q, 0), q)
    np.testing.assert_array_equal(at(q, 9)[..., 16:], q[..., 16:])
    assert np.isclose(np.linalg.norm(at(q, 12345)), np.linalg.norm(q), rtol=1e-13)
    dots = [float((at(q, p + 7) * at(k, p)).sum()) for p in (0, 3, 1000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-11)


def test_rotation_by_a_quarter_turn_and_the_layouts():
    q = np.arange(1.0, 5.0).reshape(1, 1, 4)
    turn = np.array([math.pi / 2, 0.0])
    np.testing.assert_allclose(oa.norm_rope(q, None, 0, [1], turn, "half", 1.0)[0, 0],
                               [-3, 2, 1, 4], atol=1e-15)
    np.testing.assert_allclose(oa.norm_rope(q, None, 0, [1], turn, "interleaved", 2.0)[0, 0],
                               [-4, 2, 6, 8], atol=1e-15)


def test_norm_gives_unit_mean_square_times_the_weight():
    x, w = _x(3, 2, 32), _x(32, seed=2)
    y = oa.norm_rope(x, w, 0.0, [0, 0, 0], np.zeros(0), "half", 1.0)
    np.testing.assert_allclose(((y / w) ** 2).mean(-1), 1.0, rtol=1e-12)
    np.testing.assert_allclose(oa.norm_rope(7 * x, w, 0.0, [0] * 3, np.zeros(0), "half", 1.0), y,
                               rtol=1e-12)


def _library(rot, base, kind, factor=1.0, length=0, fast=32.0, slow=1.0):
    out, scale = (ctypes.c_double * max(1, rot // 2))(), ctypes.c_float()
    code = ttt.lib().ttt_rope_frequencies(ctypes.addressof(out), rot, base, kind, factor, length,
                                          fast, slow, ctypes.addressof(scale))
    return code, np.array(out), scale.value


@pytest.mark.parametrize("rot,base", [(2, 10.0), (16, 1e4), (96, 5e5), (128, 1e6), (256, 1e4)])
@pytest.mark.parametrize("kind,factor", [(None, 1.0), ("linear", 8.0), ("ntk", 4.0),
                                         ("yarn", 1.0), ("yarn", 16.0)])
def test_frequencies(rot, base, kind, factor):
    if kind == "ntk" and rot < 4:
        return
    code, f, s = _library(rot, base, ttt.ROPE_SCALINGS[kind], factor, 4096)
    want, scale = oa.rope_frequencies(rot, base, kind, factor, 4096)
    assert code == 0
    np.testing.assert_allclose(f, want, rtol=1e-12)
    assert np.isclose(s, scale, rtol=1e-6)
    assert np.isclose(f[0], 1.0 / factor if kind == "linear" else want[0], rtol=1e-12)
    if kind == "ntk":  # the slowest pair is interpolated by the whole factor
        assert np.isclose(f[-1], base ** (-(rot - 2) / rot) / factor, rtol=1e-12)
    if kind == "yarn" and factor > 1 and rot >= 96:  # fast pairs kept, slow ones interpolated
        plain = base ** (-2 * np.arange(rot // 2) / rot)
        assert f[0] == plain[0] and np.isclose(f[-1], plain[-1] / factor, rtol=1e-12)


@pytest.mark.parametrize("args", [
    (0, 1e4, 0), (3, 1e4, 0), (258, 1e4, 0), (64, 1.0, 0), (64, float("nan"), 0),
    (64, float("inf"), 0), (64, 1e4, 1, 0.5), (64, 1e4, 1, float("nan")), (2, 1e4, 2, 2.0),
    (64, 1e4, 3, 2.0, 0), (64, 1e4, 3, 2.0, 4096, 1.0, 1.0), (64, 1e4, 3, 2.0, 4096, 32.0, 0.0),
    (64, 1e4, 4), (64, 1e4, -1)])
def test_frequencies_refusals(args):
    assert _library(*args)[0] == 2  # TTT_E_SHAPE
    assert ttt.lib().ttt_rope_frequencies(None, 64, 1e4, 0, 1.0, 0, 32.0, 1.0, None) == 1


def test_one_key_equal_keys_and_two_keys():
    q, K, V = _x(4), _x(6, 4, seed=1), _x(6, 3, seed=2)
    o, lse, _ = oa.attend(q, K[:1], V[:1], 0.5)
    np.testing.assert_allclose(o, V[0], rtol=1e-15)
    assert np.isclose(lse, 0.5 * K[0] @ q)
    o, lse, a = oa.attend(q, np.tile(K[0], (6, 1)), V, 0.5)
    np.testing.assert_allclose(o, V.mean(0), rtol=1e-13)
    np.testing.assert_allclose(a, np.abs(V).mean(0), rtol=1e-13)
    assert np.isclose(lse, 0.5 * K[0] @ q + math.log(6))
    o, _, _ = oa.attend(q, K[:2], V[:2], 1.0)
    w = 1 / (1 + math.exp((K[1] - K[0]) @ q))
    np.testing.assert_allclose(o, w * V[0] + (1 - w) * V[1], rtol=1e-13)


def test_masks_windows_packing_and_groups():
    Q, K, V = _x(9, 4, 8), _x(9, 2, 8, seed=1), _x(9, 2, 8, seed=2)
    O, L, _ = oa.packed(Q, K, V, [0, 9], [0, 9], 0.3)
    np.testing.assert_allclose(O[0], V[0][[0, 0, 1, 1]], rtol=1e-14)     # the first sees itself
    K1, V1 = K.copy(), V.copy()
    K1[5:], V1[5:] = 9, 9
    O1, _, _ = oa.packed(Q, K1, V1, [0, 9], [0, 9], 0.3)
    np.testing.assert_array_equal(O1[:5], O[:5])                          # causality
    O2, L2, _ = oa.packed(Q, K, V, [0, 0, 4, 9], [0, 0, 4, 9], 0.3)        # packing
    for a, b in ((0, 4), (4, 9)):
        o, l, _ = oa.packed(Q[a:b], K[a:b], V[a:b], [0, b - a], [0, b - a], 0.3)
        np.testing.assert_allclose(O2[a:b], o, rtol=1e-14)
        np.testing.assert_allclose(L2[a:b], l, rtol=1e-14)
    O3, _, _ = oa.packed(Q, K, V, [0, 9], [0, 9], 0.3, window=1)           # only the own key
    np.testing.assert_allclose(O3, V[:, [0, 0, 1, 1]], rtol=1e-14)
    O4, _, _ = oa.packed(Q, K, V, [0, 9], [0, 9], 0.3, window=9)
    np.testing.assert_array_equal(O4, O)
    O5, L5, _ = oa.packed(Q, K[:4], V[:4], [0, 9], [0, 4], 0.3)            # 5 queries see nothing
    assert (O5[:5] == 0).all() and (L5[:5] == -np.inf).all()
    np.testing.assert_allclose(O5[5], V[0][[0, 0, 1, 1]], rtol=1e-14)
    O6, _, _ = oa.packed(Q[6:], K, V, [0, 3], [0, 9], 0.3)                 # a prompt's last piece
    np.testing.assert_allclose(O6, O[6:], rtol=1e-14)


def test_decode_is_the_last_row_of_a_packed_sequence():
    Q, K, V = _x(9, 4, 8), _x(9, 2, 8, seed=1), _x(9, 2, 8, seed=2)
    page, table = 4, np.array([[3, 0, 2]])
    Kc, Vc = np.full((16, 2, 8), np.nan), np.full((16, 2, 8), np.nan)
    for j in range(9):
        Kc[table[0, j // 4] * 4 + j % 4], Vc[table[0, j // 4] * 4 + j % 4] = K[j], V[j]
    for window in (0, 1, 4, 20):
        O, L, _ = oa.packed(Q, K, V, [0, 9], [0, 9], 0.3, window)
        o, l, _ = oa.decode(Q[8:], Kc, Vc, table, [9], page, 0.3, window)
        np.testing.assert_allclose(o, O[8:], rtol=1e-14)
        np.testing.assert_allclose(l, L[8:], rtol=1e-14)
    o, l, _ = oa.decode(Q[:1], Kc, Vc, table, [0], page, 0.3)
    assert (o == 0).all() and (l == -np.inf).all()
