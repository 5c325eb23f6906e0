"""The listed cases of perf/more_operators.py, whose times are published, through the package against their 64-bit
results, every element.

Bounds as in test_gpu_add_norm.py, test_gpu_attention.py (the sums of weight * |v| from the plain form with |V| in place
of V, 2^-7 off with room to spare) and test_gpu_delta.py: states 2e-6 of their size in the 2-norm, each head's. Outputs
of the delta rule here by their 2-norm too: half a step of their own, 2^-8 at most, and half a step of A's entries,
whose products with u are as large as the outputs in the mean over a head's tokens and channels (neither keys nor
values have a mean that would cancel): 2^-7 of the norm, where roundings are as large as they can be."""
import importlib.util
import os

import pytest

from helpers import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")
_SPEC = importlib.util.spec_from_file_location("serving_cases", _PATH)
ops = importlib.util.module_from_spec(_SPEC)
_SPEC.loader.exec_module(ops)


def _within(got, want, bound, what):
    worst = float(((got.double() - want).abs() / bound).max())
    print(f"  {what}: {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0, what


@pytest.mark.parametrize("case", ops.listed(), ids=lambda c: c["name"])
def test_listed_case(case, monkeypatch):
    import torch
    print(f"case: {case['name']}", flush=True)
    seed, step = 2, 2.0 ** -24
    want = ops.exact(case, seed)
    state = ops.prepare(case, seed)
    monkeypatch.setattr(ops, "own", True)
    got = ops.run(state)
    if case["op"] == "norm":
        half = {"bf16": 2.0 ** -8, "f32": step}[case["dtype"]]
        _within(got[-1], want[-1], (1.01 * half + step) * want[-1].abs() + 1e-38, "sum")
        if case["out"] != "e4m3":
            _within(got[0], want[0], (1.01 * half + 50 * step) * want[0].abs() + 1e-38, "y")
            return
        _within(got[1], want[1], 52 * step * want[1], "scales")
        q = got[0].float().double()
        _within(q, want[0], 1.01 * torch.clamp(2.0 ** -4 * want[0].abs(), min=2.0 ** -10) + 110 * step * want[0].abs(), "y")
        return
    if case["op"] == "paged":
        monkeypatch.setattr(ops, "own", False)
        size = ops.run(dict(state, Vc=state["Vc"].abs()))[0].double() * (1 + 2.0 ** -7)
        X = case["dh"] ** -0.5 * float(state["Q"].float().norm(dim=-1).max()) * float(state["Kc"].float().norm(dim=-1).max())
        d = (case["dh"] + 4) * step * X
        _within(got[0], want[0], 1.01 * (2.0 ** -8 * (want[0].abs() + size) + (4 * d + 2.0 ** -19) * size) + 1e-38, "o")
        _within(got[1], want[1], d + 2.0 ** -20 + 4 * step * (want[1].abs() + X), "lse")
        return
    o, w = got[0].double(), want[0]
    off = (o - w).flatten(2).norm(dim=(0, 2)) / w.flatten(2).norm(dim=(0, 2))
    at = state["slots"].long()
    S, W = got[1][at].double(), want[1][at]
    soff = (S - W).norm(dim=(2, 3)) / W.norm(dim=(2, 3))
    rest = torch.ones(len(got[1]), dtype=torch.bool, device=S.device)
    rest[at] = False
    print(f"  o {float(off.max()):.2e}, states {float(soff.max()):.2e} off", flush=True)
    assert torch.isfinite(o).all() and float(off.max()) <= 2.0 ** -7 and float(soff.max()) <= 2e-6
    assert (got[1][rest] == 0).all()
