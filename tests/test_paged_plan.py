"""The rules by which attention of new tokens over a paged cache chooses its form (csrc/attn_plan.hpp), compiled for
the host: no call needs more workspace than the query says, and the forms that the GPU tests mean are taken."""
import ctypes
import random
import subprocess

import pytest

import chunked_weight_sequence_amd as ttt
from plan_shim import CSRC

SOURCE = """
#include "attn_plan.hpp"
using namespace ttt;
extern "C" void paged(int n, int Nq, int max_pages, int page, int Hq, int Hkv, int dh, int window, long* out) {
  const PackedPlan p = paged_plan(n, Nq, max_pages, page, Hq, Hkv, dh, window);
  out[0] = p.qt, out[1] = p.splits, out[2] = p.tiles, out[3] = p.half;
  out[4] = long(paged_workspace(n, Nq, max_pages, page, Hq, Hkv, dh));
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("paged") / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "-x", "c++", "-", "-o", so],
                   input=SOURCE, text=True, check=True)
    fn = ctypes.CDLL(so).paged

    def ask(*args):
        out = (ctypes.c_long * 5)()
        fn(*(ctypes.c_int(int(x)) for x in args), out)
        return dict(zip(("qt", "splits", "tiles", "half", "workspace"), out))
    return ask


def test_no_call_needs_more_workspace_than_the_query_says(plan):
    rng = random.Random(7)

    def log(lo, hi):
        return int(lo * (hi / lo) ** rng.random())
    for _ in range(20000):
        Hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
        Hq, dh = Hkv * rng.choice([1, 2, 4, 7, 8, 40]), rng.choice([64, 128])
        n, window, page = rng.choice([1, log(1, 300)]), rng.choice([0, log(1, 30000)]), rng.choice([16, 64, 256])
        Nq, pages = log(1, 40000), log(1, 200000 // page)
        p = plan(n, Nq, pages, page, Hq, Hkv, dh, window)
        need = p["splits"] * Nq * Hq * (dh + 2) * 4 if p["splits"] > 1 else 0
        assert need <= p["workspace"], (n, Nq, pages, page, Hq, Hkv, dh, window, p)
        assert p["workspace"] == ttt.lib().ttt_attention_paged_workspace(n, Nq, pages, page, Hq, Hkv, dh)
        assert 1 <= p["splits"] <= 64 and 0 <= p["half"] <= p["tiles"] and p["qt"] in (1, 2)


def test_forms(plan):
    """Rows by 128 and by 256, whole and in pieces, of one and of several sequences."""
    got = {name: plan(*a) for name, a in dict(
        one=(1, 512, 256, 64, 32, 8, 128, 0), drafts=(16, 48, 500, 16, 16, 4, 64, 0), whole=(4, 8000, 32, 256, 32, 32, 64, 2048),
        mixed=(16, 526, 375, 32, 32, 8, 128, 0), wide=(5, 1539, 160, 16, 32, 8, 128, 0), few=(8, 135, 250, 16, 32, 8, 128, 0), prompt=(1, 2100, 33, 64, 32, 8, 128, 0),
        short=(16, 790, 19, 16, 32, 8, 128, 0)).items()}
    assert (got["one"]["qt"], got["one"]["splits"]) == (2, 4)
    assert got["drafts"]["qt"] == 1 and got["drafts"]["splits"] >= 8
    assert (got["whole"]["qt"], got["whole"]["splits"]) == (1, 1)
    assert (got["mixed"]["qt"], got["mixed"]["splits"]) == (1, 3)
    assert (got["wide"]["qt"], got["wide"]["splits"]) == (2, 1)
    assert got["few"]["qt"] == 1 and got["few"]["splits"] > 1
    assert got["short"]["splits"] == 1 and got["prompt"]["splits"] == 1


def test_what_is_judged_is_what_is_launched(tmp_path):
    """Of several sequences 256 rows are taken only where the workgroups of the pieces that are launched fill at least 9 of
    10 places of the chip each time around, in pieces of at least 1024 keys, and an order by length only where more than
    512 and at most 3200 are launched, each with a key tile at least for every sequence that it ranks."""
    so = str(tmp_path / "forms.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "-x", "c++", "-", "-o", so], input="""
#include "attn_plan.hpp"
using namespace ttt;
extern "C" void form(int n, int Nq, int max_pages, int page, int Hq, int Hkv, int window, long* out) {
  const PackedPlan p = paged_plan(n, Nq, max_pages, page, Hq, Hkv, 128, window);
  const long Nk = paged_keys(n, max_pages, page), wgs = packed_wgs(p.qt, n, Nq, Hq, Hkv);
  const long v[] = {p.qt, p.splits, p.longest, wgs, packed_seen(n, Nq, Nk, window), packed_keys(n, Nk, window)};
  for (int i = 0; i < 6; ++i) out[i] = v[i];
}
""", text=True, check=True)
    fn = ctypes.CDLL(so).form

    def ask(*args):
        out = (ctypes.c_long * 6)()
        fn(*(ctypes.c_int(int(x)) for x in args), out)
        return list(out)
    rng, forms = random.Random(11), set()
    for _ in range(40000):
        Hkv, n = rng.choice([1, 2, 4, 8, 16]), rng.randint(2, 40)
        a = (n, int(n * 2000 ** rng.random()), rng.randint(1, 1000), 16, Hkv * rng.choice([1, 2, 4, 8]), Hkv,
             rng.choice([0, 0, rng.randint(1, 9000)]))
        qt, splits, longest, wgs, seen, keys = ask(*a)
        forms.add((qt, splits > 1, bool(longest)))
        if qt == 2:
            around = -(-wgs * splits // 256)
            assert 10 * wgs * splits >= 9 * 256 * around and seen >= 1024 * splits, (a, qt, splits, wgs)
        if longest:
            assert 512 < wgs * splits <= 3200 and (splits == 1 or n <= keys // 64 // splits), (a, splits, wgs)
    assert {(1, False, False), (1, False, True), (1, True, False), (1, True, True), (2, False, False), (2, True, False)} <= forms
    # 2 x 260 tokens on 8000: 3 pieces would fill the chip, 4 are launched; the GPU tests' sequences in several pieces of 256 rows
    assert ask(2, 520, 500, 16, 32, 8, 0)[:2] == [1, 4]
    assert ask(3, 409, 266, 16, 32, 4, 0)[:2] == [2, 4]
    assert ask(2, 1224, 410, 16, 8, 2, 0)[:2] == [2, 6]


def test_few_rows_of_one_sequence_stay_in_one_tile_of_128(plan):
    """However long the keys, or the table that has room for them, are."""
    for new in (1, 5, 32):
        for keys in (4096, 32768, 49152, 131072, 1 << 20):
            assert plan(1, new, keys // 64, 64, 32, 8, 128, 0)["qt"] == 1, (new, keys)
    assert plan(1, 40, 1024, 64, 32, 8, 128, 0)["qt"] == 2 and plan(1, 128, 1024, 64, 8, 8, 128, 0)["qt"] == 1
