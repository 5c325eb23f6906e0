"""The rules by which the attention calls choose their kernels (csrc/attn_plan.hpp), compiled for the host."""
import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "chunked_weight_sequence_amd", "csrc")

SOURCE = """
#include "attn_plan.hpp"
using namespace ttt;
extern "C" void packed(int n, int Nq, int Nk, int Hq, int Hkv, int dh, int window, long* out) {
  const PackedPlan p = packed_plan(n, Nq, Nk, Hq, Hkv, dh, window);
  const long v[] = {p.qt, p.splits, p.tiles, p.half, p.longest, join_rows(p.splits, long(Nq) * Hq, dh),
                    long(packed_workspace(n, Nq, Nk, Hq, Hkv, dh))};
  for (int i = 0; i < 7; ++i) out[i] = v[i];
}
extern "C" void decode(int n, int max_pages, int page, int Hq, int Hkv, int dh, int window, long* out) {
  const DecodePlan p = decode_plan(n, max_pages, page, Hkv, Hq / Hkv, dh, window);
  const long v[] = {p.waves, p.splits, join_rows(p.splits, long(n) * Hq, dh),
                    long(decode_workspace(n, max_pages, page, Hq, Hkv, dh))};
  for (int i = 0; i < 4; ++i) out[i] = v[i];
}
"""


class Plan:
    def __init__(self, folder):
        so = os.path.join(str(folder), "plan.so")
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "-x", "c++", "-", "-o", so],
                       input=SOURCE, text=True, check=True)
        self.lib = ctypes.CDLL(so)

    def _ask(self, fn, args, names):
        out = (ctypes.c_long * len(names))()
        fn(*(ctypes.c_int(int(x)) for x in args), out)
        return dict(zip(names, out))

    def packed(self, lq, more, Hq, Hkv, dh, window):
        """Of a call with these queries and further keys of each sequence."""
        Nk = sum(max(a + b, 0) for a, b in zip(lq, more))
        p = self._ask(self.lib.packed, (len(lq), sum(lq), max(Nk, 1), Hq, Hkv, dh, window),
                      ("qt", "splits", "tiles", "half", "longest", "join", "workspace"))
        p["reversed"], p["longest"] = p["half"] < p["tiles"], bool(p["longest"])
        return p

    def decode(self, n_seq, max_pages, page, Hq, Hkv, dh, window):
        return self._ask(self.lib.decode, (n_seq, max_pages, page, Hq, Hkv, dh, window),
                         ("waves", "splits", "join", "workspace"))
