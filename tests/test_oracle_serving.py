"""Pins of the oracle of the residual stream's norm and of the gated delta rule: closed forms, invariants,
and the separately written delta rule of TTT-Linear's oracle."""
import math

import numpy as np
import pytest

import oracle.attention as oa
import oracle.serving as osv
import oracle.ttt_linear as ol


def test_e4m3_codes():
    v = osv.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[7] == 7 * 2.0 ** -9 and v[8] == 2.0 ** -6
    assert v[0x38] == 1 and v[0x3C] == 1.5 and v[0x7E] == 448 and math.isnan(v[0x7F]) and v[0xFE] == -448
    assert (np.diff(v[:0x7F]) > 0).all()


def test_paged_is_packed_on_gathered_keys_and_decode_on_single_tokens():
    r = np.random.default_rng(2)
    page, Hq, Hkv, dh = 4, 4, 2, 6
    Kc, Vc = r.standard_normal((2, 8 * page, Hkv, dh))
    table, lens, new = np.array([[5, 1, 7], [0, 3, 2]]), [11, 6], [4, 6]
    Q, cu = r.standard_normal((10, Hq, dh)), [0, 4, 10]
    rows = [[t * page + i for t in table[s] for i in range(page)][:lens[s]] for s in range(2)]
    cat = rows[0] + rows[1]
    for window in (0, 3):
        got = osv.paged(Q, Kc, Vc, cu, table, lens, page, 0.4, window)
        want = oa.packed(Q, Kc[cat], Vc[cat], cu, [0, 11, 17], 0.4, window)
        for a, b in zip(got, want):
            np.testing.assert_allclose(a, b)
        one = osv.paged(Q[:2], Kc, Vc, [0, 1, 2], table, lens, page, 0.4, window)
        for a, b in zip(one, oa.decode(Q[:2], Kc, Vc, table, lens, page, 0.4, window)):
            np.testing.assert_allclose(a, b if a.ndim == b.ndim else b)
    hole = table.copy()
    hole[0, 1] = 99  # left out: the other keys' weights, of the same logits
    o, lse, _ = osv.paged(Q, Kc, Vc, cu, hole, lens, page, 0.4)
    keep = rows[0][:4] + rows[0][8:11]
    w = np.exp(0.4 * Kc[keep, 0] @ Q[3, 1])
    np.testing.assert_allclose(o[3, 1], w @ Vc[keep, 0] / w.sum())
    np.testing.assert_allclose(lse[3, 1], np.log(w.sum()))


def test_norm_closed_forms():
    y, h = osv.add_rms_norm([[3.0, -4.0]], [[0.0, 8.0]], None, 0.0)
    np.testing.assert_allclose(h, [[3, 4]])
    np.testing.assert_allclose(y, np.array([[3, 4]]) / math.sqrt(12.5))
    rng = np.random.default_rng(0)
    X = rng.standard_normal((5, 40))
    y, _ = osv.add_rms_norm(X, None, None, 0.0)
    np.testing.assert_allclose((y * y).mean(axis=1), 1)
    np.testing.assert_allclose(osv.add_rms_norm(7 * X, None, None, 0.0)[0], y)
    w = rng.standard_normal(40)
    np.testing.assert_allclose(osv.add_rms_norm(X, None, w, 0.0)[0], y * w)
    np.testing.assert_allclose(osv.add_rms_norm(X, None, None, 1e6)[0], X / 1e3, rtol=1e-5)  # eps decides
    assert osv.add_rms_norm(np.zeros((1, 8)), None, None, 1e-6)[0].max() == 0


def test_scales():
    y = np.array([[448.0, 1, -896, 2], [0, 0, 0, 0]])
    np.testing.assert_array_equal(osv.e4m3_scales(y), [2, 2.0 ** -126])
    np.testing.assert_array_equal(osv.e4m3_scales(y, 2), [[1, 2], [2.0 ** -126] * 2])


def _case(T=9, Hk=2, Hv=4, dk=6, dv=5, seed=0):
    r = np.random.default_rng(seed)
    return (r.standard_normal((T, Hk, dk)), r.standard_normal((T, Hk, dk)), r.standard_normal((T, Hv, dv)),
            -r.random((T, Hv)), r.random((T, Hv)), r.standard_normal((Hv, dk, dv)))


def test_without_decay_it_is_the_delta_rule():
    q, k, v, g, b, W = _case(Hk=4, dv=6)
    eta = 0.3
    o, w, _, _ = osv.gated_delta(q, k, v, 0 * g, 0 * b + eta, W, 1.0)
    o1, w1 = ol.delta_rule(q, k, v, W, eta)
    np.testing.assert_allclose(o, o1, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(w, w1, rtol=1e-12, atol=1e-12)


def test_orthonormal_keys_are_stored_and_read_back():
    n = 6
    k = np.eye(n)[:, None]
    v = np.random.default_rng(1).standard_normal((n, 1, 3))
    o, w, _, _ = osv.gated_delta(k, k, v, np.zeros((n, 1)), np.ones((n, 1)), None, 1.0)
    np.testing.assert_allclose(o, v)
    np.testing.assert_allclose(w[0], v[:, 0])
    # written twice: the newer value alone; half a step: the mean
    two = osv.gated_delta(k[[0, 0]], k[[0, 0]], v[:2], np.zeros((2, 1)), np.ones((2, 1)), None, 1.0)[0]
    np.testing.assert_allclose(two[1], v[1])
    half = osv.gated_delta(k[[0, 0]], k[[0, 0]], v[:2], np.zeros((2, 1)), np.array([[1], [0.5]]), None, 1.0)[0]
    np.testing.assert_allclose(half[1], (v[0] + v[1]) / 2)


def test_decay():
    q, k, v, g, b, W = _case()
    _, w, _, _ = osv.gated_delta(q, k, v, g, 0 * b, W, 1.0)  # no step: the decays alone
    np.testing.assert_allclose(w, np.exp(g.sum(axis=0))[:, None, None] * W)
    g2 = g.copy()
    g2[4] = -np.inf  # forgets all: a sequence of its own from there on
    o, w, _, _ = osv.gated_delta(q, k, v, g2, b, W, 0.5)
    o1, w1, _, _ = osv.gated_delta(q[4:], k[4:], v[4:], g[4:], b[4:], None, 0.5)
    np.testing.assert_allclose(o[4:], o1)
    np.testing.assert_allclose(w, w1)
    np.testing.assert_allclose(o[:4], osv.gated_delta(q[:4], k[:4], v[:4], g[:4], b[:4], W, 0.5)[0])


@pytest.mark.parametrize("eps", [None, 1e-6])
def test_pieces_groups_and_scale(eps):
    q, k, v, g, b, W = _case()
    o, w, size, wsize = osv.gated_delta(q, k, v, g, b, W, 0.5, eps)
    o1, w1, _, _ = osv.gated_delta(q[:5], k[:5], v[:5], g[:5], b[:5], W, 0.5, eps)
    o2, w2, _, _ = osv.gated_delta(q[5:], k[5:], v[5:], g[5:], b[5:], w1, 0.5, eps)
    np.testing.assert_allclose(np.concatenate([o1, o2]), o)
    np.testing.assert_allclose(w2, w)
    rep = [x.repeat(2, axis=1) for x in (q, k)]  # shared heads are heads of their own
    np.testing.assert_allclose(osv.gated_delta(*rep, v, g, b, W, 0.5, eps)[0], o)
    np.testing.assert_allclose(osv.gated_delta(q, k, v, g, b, W, 1.5, eps)[0], 3 * o)
    assert (np.abs(o) <= size * (1 + 1e-12)).all() and (np.abs(w) <= wsize * (1 + 1e-12)).all()


def test_normalised_keys_do_not_depend_on_their_length():
    q, k, v, g, b, W = _case()
    o, w, _, _ = osv.gated_delta(q, k, v, g, b, W, 1.0, 0.0)
    o1, w1, _, _ = osv.gated_delta(3 * q, 5 * k, v, g, b, W, 1.0, 0.0)
    np.testing.assert_allclose(o1, o)
    np.testing.assert_allclose(w1, w)
