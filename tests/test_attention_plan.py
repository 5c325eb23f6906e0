"""The rules that choose a form of the attention kernels: the cases that test a form on the GPU take it, and
no call needs more workspace than the queries say."""
import random

import pytest

import chunked_weight_sequence_amd as ttt
from attention_forms import DECODE, PACKED
from plan_shim import Plan


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    return Plan(tmp_path_factory.mktemp("plan"))


def test_packed_cases_take_their_forms(plan):
    for case, form in PACKED:
        p = plan.packed(*case)
        assert {k: p[k] for k in form} == form, (case, p)
        lq, more, *rest = case  # the GPU test adds five query rows of no sequence
        p = plan.packed(lq[:-1] + [lq[-1] + 5], more[:-1] + [more[-1] - 5], *rest)
        assert {k: p[k] for k in form} == form, (case, p)


def test_decode_cases_take_their_forms(plan):
    for (lens, pages, page, Hq, Hkv, dh, window), form in DECODE:
        p = plan.decode(len(lens), pages, page, Hq, Hkv, dh, window)
        assert {k: p[k] for k in form} == form, (lens[:4], pages, Hq, Hkv, dh, window, p)
        assert max(lens) <= pages * page


def test_the_forms_are_all_there():
    """Every kernel and every way of joining, each size of head, split and whole, with a window and without."""
    packed = {(f["qt"], c[4], f["splits"] > 1) for c, f in PACKED}
    assert packed == {(q, d, s) for q, d in ((1, 64), (1, 128), (2, 128)) for s in (False, True)}
    assert {(c[4], f["join"]) for c, f in PACKED if f["splits"] > 1} >= {
        (64, 16), (64, 1), (64, 4), (128, 8), (128, 1), (128, 4)}
    assert {c[4] for c, f in PACKED if f.get("reversed")} == {64, 128}
    assert {f["qt"] for c, f in PACKED if c[5] and f["splits"] > 1} == {1, 2}
    assert {f["qt"] for c, f in PACKED if f.get("longest")} == {1, 2}
    decode = {(c[5], f["waves"], f["splits"] > 1, c[6] > 0) for c, f in DECODE}
    assert decode >= {(128, 2, s, w) for s in (False, True) for w in (False, True)}
    assert decode >= {(64, 4, True, True), (128, 4, True, True), (64, 4, True, False), (128, 4, True, False)}
    assert {f.get("join") for c, f in DECODE} >= {1, 4, 8, 16}


def test_sequences_are_taken_longest_first_where_it_pays(plan):
    assert plan.packed([1100] * 8, [0] * 8, 16, 8, 128, 0)["longest"]           # 1100 workgroups
    assert plan.packed([0, 900, 33, 0, 1500, 128, 1, 900, 0], [0] * 9, 32, 16, 64, 0)["longest"]
    assert not plan.packed([32] * 16, [0] * 16, 32, 8, 128, 0)["longest"]       # all on the chip at once
    assert not plan.packed([180] * 24, [0] * 24, 32, 8, 128, 0)["longest"]      # rows of three tiles
    assert not plan.packed([1024] * 16, [0] * 16, 32, 32, 64, 512)["longest"]   # many times around


def test_no_call_needs_more_workspace_than_the_queries_say(plan):
    """The queries do not know the window, which decides the number of pieces too."""
    rng = random.Random(5)

    def log(lo, hi):
        return int(lo * (hi / lo) ** rng.random())
    for _ in range(20000):
        Hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
        Hq, dh = Hkv * rng.choice([1, 2, 4, 7, 8, 40]), rng.choice([64, 128])
        n, window = log(1, 90), rng.choice([0, log(1, 30000)])
        Nq, Nk = log(1, 40000), log(1, 200000)
        p = plan.packed([Nq] + [0] * (n - 1), [Nk - Nq] + [0] * (n - 1), Hq, Hkv, dh, window)
        need = p["splits"] * Nq * Hq * (dh + 2) * 4 if p["splits"] > 1 else 0
        assert need <= p["workspace"], (n, Nq, Nk, Hq, Hkv, dh, window, p)
        assert p["workspace"] == ttt.lib().ttt_attention_packed_workspace(n, Nq, Nk, Hq, Hkv, dh)
        assert 1 <= p["splits"] <= 64 and 0 <= p["half"] <= p["tiles"]
        S, page = log(1, 500), rng.choice([16, 64, 256])
        pages = log(1, 100000 // page)
        d = plan.decode(S, pages, page, Hq, Hkv, dh, window)
        need = d["splits"] * S * Hq * (dh + 2) * 4 if d["splits"] > 1 else 0
        assert need <= d["workspace"], (S, pages, page, Hq, Hkv, dh, window, d)
        assert d["workspace"] == ttt.lib().ttt_attention_decode_workspace(S, pages, page, Hq, Hkv, dh)
        assert 1 <= d["splits"] <= 64
