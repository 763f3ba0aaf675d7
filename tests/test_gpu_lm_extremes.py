"""GPU: the 8-bit operators at the ends of their types' ranges.

Tolerances, derived before any run: those of tests/test_gpu_lm.py, from its own checks.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("no CUDA device", allow_module_level=True)

from dac_vocoder_decode_gb300 import binding as V  # noqa: E402
from tests import test_gpu_lm as T  # noqa: E402

SYNC = V.VOC_FLAG_SYNC


# ------------------------------------------------------------------ rows
def _large(g, d, t):
    """Rows whose largest magnitudes lie from 2^126 to the type's largest value."""
    top = torch.finfo(t).max
    x = (torch.rand(6, d, generator=g, device="cuda", dtype=torch.float64) * 2 - 1) * top
    x[1] *= 0.3
    x[2] /= x[2].abs().max() / 2.0 ** 127
    x[3] = torch.randn(d, generator=g, device="cuda", dtype=torch.float64)
    x[3, d // 2] = -top
    x[4] = 0
    x[4, d - 1] = 2.0 ** 127
    x[5, 0] = top
    return x.to(t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [1, 40, 1024, 1031, 5000, 20000])
def test_rows_largest_magnitudes(dtype, d):
    """Magnitudes from 2^126 to the type's largest value, as inputs and as sums with a residual."""
    t = T.TYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(d)
    x = _large(g, d, t)
    w = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(t)
    for eps in (1e-6, 0.0):
        T._check_rows(x, "rms", w, None, eps, V.rows_fp8(x, weight=w, eps=eps, flags=SYNC), d)
    T._check_rows(x, "none", None, None, 0, V.rows_fp8(x, V.VOC_LM_NONE, flags=SYNC), d)
    half = (x.double() / 2).to(t)
    rest = (x.double() - half.double()).to(t)
    got = V.rows_fp8(half, weight=w, residual=rest, eps=1e-6, flags=SYNC)
    T._check_rows(half, "rms", w, rest, 1e-6, got, d)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [[1, 1], [5, 64], [129, 64]])
def test_attention_largest_queries(d, new):
    """bf16 queries from 2^126 to the largest value, over keys so small that scores stay finite."""
    bt = T.Batch([400, 64], new, 2, d, seed=8)
    bt.ks = np.full_like(bt.ks, 2.0 ** -90)
    bt.cache.k_scale.copy_(torch.from_numpy(bt.ks).cuda())
    q = bt.rng.uniform(-1, 1, (bt.total, 4, d)) * float(torch.finfo(torch.bfloat16).max)
    q[0, 1, 5] = 2.0 ** 126
    q[1] *= 2.0 ** -3
    T._check_attention(bt, torch.from_numpy(q).cuda().bfloat16(), scale=2.0 ** -49)
