"""Norm and rotation at the stated limits: sizes of heads whose squares leave fp32."""
import numpy as np
import pytest

import chunked_weight_sequence_amd as ttt
import gen
import oracle.attention as oa
from helpers import dev, host_f64, requires_gpu
from test_gpu_attention import _f, _i32

pytestmark = [pytest.mark.gpu, requires_gpu]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,by,eps", [(128, 1e25, 1e-6), (128, 2.0 ** 127, 1e-6), (80, 1e19, 0.0), (64, 1e-25, 0.0),
                                       (256, 1e-36, 0.0), (64, 1e-22, 1e-40), (64, 1e-25, 1e-6)])
def test_norms_of_very_large_and_small_heads(dtype, dh, by, eps):
    """x / sqrt(mean(x^2) + eps) is of ordinary size wherever x lies in its type's range. Bound: the sum's
    dh / 2 half steps and 16 more for the root, the products and a scaling, then the output's rounding."""
    import torch
    print(f"case: norm of heads of size {by} {dtype} dh={dh} eps={eps}", flush=True)
    rng = np.random.default_rng(dh)
    x = (by * rng.uniform(-1, 1, (5, 3, dh))).astype(np.float32)
    x[1, 1] /= 1e12 if by > 1 else 1  # an ordinary head among them, in the same waves
    x[2, 0] = 1.5
    if dtype == "bf16":
        x = gen.f32_to_bf16_bits(x)
    w = rng.uniform(0.5, 1.5, dh).astype(np.float32)
    X = _f(x) if dtype == "bf16" else x.astype(np.float64)
    e = float(np.float32(eps))
    Q, _ = ttt.qk_norm_rope(dev(x, dtype), dev(x, dtype), _i32([0] * 5),
                            torch.zeros(0, dtype=torch.float64, device="cuda"), q_weight=dev(w, "f32"),
                            eps=eps)
    torch.cuda.synchronize()
    want = oa.norm_rope(X, w, e, [0] * 5, np.zeros(0), "half", 1.0)
    bound = ((dh / 2 + 16) * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)) * np.abs(want) + 2e-38
    off = np.abs(host_f64(Q) - want) / bound
    print(f"  {off.max():.3f} of the bound", flush=True)
    assert np.isfinite(host_f64(Q)).all() and off.max() <= 1.0
