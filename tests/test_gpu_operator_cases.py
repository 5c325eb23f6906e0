"""The listed cases of perf/operators.py, whose times are published, through the package against their
64-bit results, every element.

Bounds as in test_gpu_attention.py and test_gpu_norm_rope.py. The sums of weight * |v| come from the plain
form with |V| in place of V (in fp32, rounded to bf16: at most 2^-7 off with room to spare), sum |q_c k_c|
is at most the product of the norms, and |a| + |b| of a pair at most the root of 2 times its norm, which
the rotation keeps."""
import importlib.util
import math
import os

import pytest

from helpers import requires_gpu

pytestmark = [pytest.mark.gpu, requires_gpu]

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")
_SPEC = importlib.util.spec_from_file_location("operator_cases", _PATH)
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
    seed, half_step = 2, {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[case.get("dtype", "bf16")]
    want = ops.exact(case, seed)
    state = ops.prepare(case, seed)
    monkeypatch.setattr(ops, "own", True)
    got = ops.run(state)
    if case["op"] == "rope":
        half = case["rot"] // 2
        for y, w, what in zip(got[:2], want[:2], "qk"):
            size = w.abs()
            a, b = ((slice(0, half), slice(half, 2 * half)) if case["layout"] == "half" else
                    (slice(0, 2 * half, 2), slice(1, 2 * half, 2)))
            size[..., a] = size[..., b] = math.sqrt(2) * torch.hypot(w[..., a], w[..., b])
            _within(y, w, (case["dh"] / 2 + 32) * 2.0 ** -24 * size + 1.01 * half_step * w.abs() + 1e-38, what)
        if case["cache"]:
            at = state["slots"].long()
            assert torch.equal(got[2][at], got[1]) and torch.equal(got[3], want[3].to(got[3].dtype))
            rest = torch.ones(len(got[2]), dtype=torch.bool, device=got[2].device)
            rest[at] = False
            assert torch.equal(got[2][rest], want[2][rest].to(got[2].dtype))  # other slots as they were
        return
    assert torch.equal(torch.isneginf(got[1]), torch.isneginf(want[1]))
    key, value = ("K", "V") if case["op"] == "packed" else ("Kc", "Vc")
    monkeypatch.setattr(ops, "own", False)
    size = ops.run(dict(state, **{value: state[value].abs()}))[0].double() * (1 + 2.0 ** -7)
    X = case["dh"] ** -0.5 * float(state["Q"].float().norm(dim=-1).max()) * \
        float(state[key].float().norm(dim=-1).max())
    d = (case["dh"] + 4) * 2.0 ** -24 * X
    _within(got[0], want[0], 1.01 * (half_step * (want[0].abs() + size) + (4 * d + 2.0 ** -19) * size) + 1e-38,
            "o")
    lse = torch.where(torch.isneginf(want[1]), 0.0, want[1])
    _within(torch.where(torch.isneginf(got[1]), 0.0, got[1]), lse,
            d + 2.0 ** -20 + 4 * 2.0 ** -24 * (lse.abs() + X), "lse")
