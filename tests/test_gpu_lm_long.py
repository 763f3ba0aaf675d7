"""GPU: the 8-bit operators' kernels for many tokens and long caches, over what only large sizes
reach: rings that wrap, further tiles of a pair.

Tolerances are those of tests/test_gpu_lm.py.  A test that is written for one kernel asserts that its
call launches it.
"""
from __future__ import annotations

import os
import warnings

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("no CUDA device", allow_module_level=True)

from dac_vocoder_decode_gb300 import binding as V  # noqa: E402
from tests import test_gpu_lm as T  # noqa: E402

SYNC = V.VOC_FLAG_SYNC


def _launched(tmp_path, call):
    """Text that names every kernel that `call` launches: the call's graph, captured and written out
    after a first pass outside of it."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    graph.enable_debug_mode()
    with torch.cuda.graph(graph):
        call()
    path = os.path.join(str(tmp_path), "graph.dot")
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")  # it announces itself
        graph.debug_dump(path)
    with open(path) as f:
        return f.read()


# ------------------------------------------------------------------ product of many tokens
def _operands(m, k, n, bias, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, w = T._codes(g, m, k), T._codes(g, n, k)
    xs = torch.rand(m, generator=g, device="cuda") / 16 + 0.01
    ws = torch.rand(n, generator=g, device="cuda") / (16 * k ** 0.5) + 0.001
    return x, xs, w, ws, torch.randn(n, generator=g, device="cuda") if bias else None


# 289 tiles on 76 pairs of SMs and 8 chunks of K, the last one ragged; 45 tiles and 13 chunks; 102
# tiles of one chunk more than the ring holds; 32 tiles, the fewest, and one short chunk
MANY = [(4100, 1000, 4200, True), (2100, 1537, 1030, False), (4100, 900, 1300, True),
        (2000, 70, 900, True)]


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,k,n,bias", MANY)
def test_linear_many(tmp_path, out, m, k, n, bias):
    x, xs, w, ws, b = _operands(m, k, n, bias, seed=m + k)
    call = lambda: V.linear_fp8(x, xs, w, ws, bias=b, out_dtype=T.TYPES[out])  # noqa: E731
    assert "linear_many_kernel" in _launched(tmp_path, call)
    y = V.linear_fp8(x, xs, w, ws, bias=b, out_dtype=T.TYPES[out], flags=SYNC)
    T._check_linear(x, xs, w, ws, b, y)


@pytest.mark.parametrize("at,ld", [(3, 1309), (2, 1306)])
def test_linear_many_into_a_strided_output(at, ld):
    m, k, n = 4100, 900, 1300
    x, xs, w, ws, b = _operands(m, k, n, True, seed=ld)
    buf = torch.full((m, ld), -7.0, dtype=torch.bfloat16, device="cuda")
    V.linear_fp8(x, xs, w, ws, bias=b, out=buf[:, at:at + n], flags=SYNC)
    T._check_linear(x, xs, w, ws, b, buf[:, at:at + n])
    assert torch.all(buf[:, :at] == -7) and torch.all(buf[:, at + n:] == -7)


def test_linear_many_nan_stays_alone_and_repeats_bit_for_bit():
    m, k, n = 4100, 900, 1300
    x, xs, w, ws, _ = _operands(m, k, n, False, seed=5)
    clean = V.linear_fp8(x, xs, w, ws, flags=SYNC)
    for _ in range(3):
        assert torch.equal(V.linear_fp8(x, xs, w, ws, flags=SYNC), clean)
    x.view(torch.uint8)[4000, 899] = 0x7f
    w.view(torch.uint8)[1290, 0] = 0xff
    xs[130] = float("nan")
    y = V.linear_fp8(x, xs, w, ws, flags=SYNC)
    bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    bad[4000], bad[130], bad[:, 1290] = True, True, True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,k,n,bias", [(70, 2048, 9000, True), (128, 9000, 1500, False),
                                        (250, 4000, 256, True), (64, 1200, 20000, False)])
def test_linear_few_over_many_chunks(tmp_path, out, m, k, n, bias):
    """Rings that wrap several times (whole K on a CTA) and rings that never fill (K split)."""
    x, xs, w, ws, b = _operands(m, k, n, bias, seed=m + k)
    call = lambda: V.linear_fp8(x, xs, w, ws, bias=b, out_dtype=T.TYPES[out])  # noqa: E731
    assert "linear_few_kernel" in _launched(tmp_path, call)
    y = V.linear_fp8(x, xs, w, ws, bias=b, out_dtype=T.TYPES[out], flags=SYNC)
    T._check_linear(x, xs, w, ws, b, y)
