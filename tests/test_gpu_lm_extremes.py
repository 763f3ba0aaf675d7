"""GPU: the 8-bit operators at the ends of their types' ranges.

Tolerances, derived before any run: those of tests/test_gpu_lm.py, from its own checks.  Gates far
below zero: e^-|g| by an exponential whose argument, up to 128 in powers of two, is off by half its
last place (2^-18) and by 2^-25 of itself, together below 5e-6 of the result, and 8 more roundings;
1e-5 in all.
"""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("no CUDA device", allow_module_level=True)

from dac_vocoder_decode_gb300 import binding as V  # noqa: E402
from tests import lm_ref as R  # noqa: E402
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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [40, 1024, 1031, 4100, 20000])
def test_rows_gates_far_below_zero(dtype, d):
    """silu(g) u where e^g is below the smallest normal number and u is large."""
    t = T.TYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(d)
    rows = 6
    lo = torch.tensor([-90.0, -100.0, -120.0, -88.0, -150.0, -95.0], device="cuda")[:, None]
    gate = lo + 8 * torch.rand(rows, d, generator=g, device="cuda")
    gate[5, ::2] = torch.randn(gate[5, ::2].shape, generator=g, device="cuda")  # beside usual ones
    up = (0.5 + torch.rand(rows, d, generator=g, device="cuda")) * 2.0 ** 120
    up *= 1 - 2 * (torch.rand(rows, d, generator=g, device="cuda") < 0.5).float()
    up[5, ::2] *= 2.0 ** -240
    x = torch.cat([gate, up], 1).to(t)
    q, scale, _ = V.rows_fp8(x, V.VOC_LM_GATED, flags=SYNC)
    n, ref, _ = R.rows(T._np(x), "gated")
    s = T._np(scale)
    np.testing.assert_allclose(s, ref, rtol=1e-5, atol=0)
    v = n / s[:, None]
    with np.errstate(divide="ignore"):
        half = np.maximum(np.exp2(np.floor(np.log2(np.abs(v))) - 4), 2.0 ** -10)
    assert np.all(np.abs(T._np(q) - v) <= half * (1 + 1e-4) + 1e-5 * np.abs(v))


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


@pytest.mark.parametrize("top", [0, 4, 8])
@pytest.mark.parametrize("d,heads", [(64, 2), (128, 1), (128, 12)])
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 130, 20]])
def test_attention_value_scales_at_both_ends(top, d, heads, new):
    """Blocks of the smallest value scale (zeros have it) beside blocks of scales up to the largest of
    f16 values: the former add nothing to the sum of values, and all of their weight to the sum of
    weights.  (What the header leaves open starts 2^104 apart.)"""
    bt = T.Batch([500, 130, 300], new, 1, d, seed=4)
    e = np.where(bt.rng.random(bt.vs.shape) < 0.5, -96, bt.rng.integers(top - 4, top + 1, bt.vs.shape))
    e[bt.table[0, 0]], e[bt.table[1, 0]], e[bt.table[2, 0]] = -96, top, -96
    e[bt.table[0, 1]], e[bt.table[1, 1]], e[bt.table[2, 1]] = top, -96, top
    bt.vs = np.exp2(e).astype(np.float32)
    bt.cache.v_scale.copy_(torch.from_numpy(bt.vs).cuda())
    T._check_attention(bt, T._queries(bt, heads))
    T._check_attention(bt, T._queries(bt, heads), max_kv=4000)
