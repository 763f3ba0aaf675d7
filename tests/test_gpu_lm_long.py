"""GPU: the 8-bit operators' kernels for many tokens and long caches, over what only large sizes
reach: rings that wrap, further tiles of a pair, scales handed over in groups, tiles in many parts.

Tolerances are those of tests/test_gpu_lm.py.  The attention's 64-bit reference is taken on the GPU
in plain products (`_reference`), by the same definition as tests/lm_ref.py; one test holds the two
together.  A test that is written for one kernel asserts that its
call launches it.
"""
from __future__ import annotations

import os
import warnings

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
# tiles of two chunks more than the ring holds; 33 tiles, the fewest, and one short chunk
MANY = [(4100, 1000, 4200, True), (2100, 1537, 1030, False), (4100, 900, 1300, True),
        (2700, 70, 700, True)]


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


# ------------------------------------------------------------------ attention over long caches
class Pool:
    """Sequences whose blocks are drawn from one small pool, so that long caches take little memory;
    every block and head has scales of its own."""

    def __init__(self, lens, new, kv_heads, d, pages=300, seed=0):
        rng = np.random.default_rng(seed)
        self.lens, self.new, self.kv_heads, self.d, self.rng = lens, new, kv_heads, d, rng
        self.total, self.max_q = sum(new), max(new)
        cols = max(-(-n // 64) for n in lens)
        self.table = torch.from_numpy(rng.integers(0, pages, (len(lens), cols)).astype(np.int32)).cuda()
        grid = lambda *s: torch.from_numpy(  # noqa: E731
            R.e4m3_round(rng.standard_normal(s) * 100).astype(np.float32)).cuda().to(T.F8)
        scale = lambda lo, hi: torch.from_numpy(  # noqa: E731
            np.exp2(rng.integers(lo, hi, (pages, kv_heads))).astype(np.float32)).cuda()
        self.cache = V.KVCacheFP8(grid(pages, kv_heads, 64, d), grid(pages, kv_heads, d, 64),
                                  scale(-9, -5), scale(-12, -5))
        self.t_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.cu = None if len(set(new)) == 1 else torch.from_numpy(cu).cuda()

    def args(self):
        return dict(page_table=self.table, kv_lens=self.t_lens, cu_q=self.cu, max_q=self.max_q)

    def queries(self, heads, dtype="bf16"):
        q = self.rng.standard_normal((self.total, heads, self.d))
        return torch.from_numpy(q).cuda().to(T.TYPES[dtype])


def _reference(bt, q, window=0, causal=True):
    """(o, sum of weights times |v|, largest sum of |q k| times the scale) in 64 bits."""
    heads, d, scale = q.shape[1], bt.d, bt.d ** -0.5
    group = heads // bt.kv_heads
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mag, smax = torch.zeros_like(o), torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(bt.lens, bt.new)):
        pages = bt.table[b, :-(-n // 64)].long()
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")[None]
        seen = (key <= pos) if causal else torch.ones(m, n, dtype=torch.bool, device="cuda")
        if window:
            seen = seen & (key > pos - window)
        for hk in range(bt.kv_heads):
            k = bt.cache.k[:, hk].double()[pages] * bt.cache.k_scale[:, hk].double()[pages][:, None, None]
            v = bt.cache.v[:, hk].double()[pages] * bt.cache.v_scale[:, hk].double()[pages][:, None, None]
            k, v = k.reshape(-1, d)[:n], v.transpose(1, 2).reshape(-1, d)[:n]
            for h in range(hk * group, (hk + 1) * group):
                qq = q[at:at + m, h].double()
                s = (qq @ k.T * scale).masked_fill(~seen, -float("inf"))
                w = torch.softmax(s, 1)
                o[at:at + m, h], mag[at:at + m, h] = w @ v, w @ v.abs()
                smax[at:at + m, h] = (qq.abs() @ k.abs().T * scale).masked_fill(~seen, 0).amax(1)
        at += m
    return o, mag, smax


def _check(bt, q, window=0, causal=True, **kw):
    o = V.attention_fp8(q, bt.cache, window=window, causal=causal, flags=SYNC, **bt.args(), **kw)
    ref, mag, s = _reference(bt, q, window, causal)
    rel = 2.0 ** -11 + 2.0 ** -16 + 2 * 1.5 * bt.d * 2.0 ** -24 * s
    tol = rel[..., None] * mag + T.UNIT[q.dtype] * ref.abs() + 2.0 ** -30
    off = (o.double() - ref).abs()
    assert bool(torch.isfinite(o).all())
    assert bool((off <= tol).all()), float((off / tol).max())
    return o


def test_the_two_references_agree():
    bt = Pool([130, 70, 64], [40, 1, 64], 2, 64, seed=1)
    q = bt.queries(4)
    ref, mag, s = R.attention(T._np(q), T._np(bt.cache.k), T._np(bt.cache.v), T._np(bt.cache.k_scale),
                              T._np(bt.cache.v_scale), bt.table.cpu().numpy(), bt.lens, bt.new, 0.125,
                              window=50)
    for a, b in zip(_reference(bt, q, window=50), (ref, mag, s)):
        np.testing.assert_allclose(T._np(a), b, rtol=1e-10, atol=1e-12)


# 20 sequences x 4 key heads: more tiles than half the SMs, so that keys are not split and one CTA
# walks over up to 141 key tiles; 64 and 200 rows a key head (one and both tiles of 128)
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("bf16", 64)])
@pytest.mark.parametrize("rows", [64, 200])
@pytest.mark.parametrize("window", [0, 8300])
def test_attention_prompt_tiles_over_long_caches(tmp_path, dtype, d, rows, window):
    lens = [9000 - 211 * i for i in range(20)]  # 141 to 78 blocks: both sides of 128 and of 96
    bt = Pool(lens, [rows // 2] * 20, 4, d, seed=rows + d)
    q = bt.queries(8, dtype)
    text = _launched(tmp_path, lambda: V.attention_fp8(q, bt.cache, window=window, **bt.args()))
    assert "attn_prompt_kernel" in text and "attn_join" not in text
    _check(bt, q, window=window)


def test_attention_prompt_tiles_over_long_caches_not_causal():
    bt = Pool([8200 + 64 * i for i in range(20)], [33] * 20, 4, 64, seed=3)
    _check(bt, bt.queries(4), causal=False)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_whole_prompt_of_many_key_tiles(d):
    """One prompt, its last tiles over 130 key tiles."""
    bt = Pool([8300], [8300], 2, d, seed=d)
    _check(bt, bt.queries(4))


@pytest.mark.parametrize("d", [64, 128])
def test_attention_prompt_tiles_in_long_parts(tmp_path, d):
    """Parts of 60 key tiles and more, which start anywhere."""
    bt = Pool([17000 - 150 * i for i in range(8)], [40] * 8, 4, d, seed=d)
    q = bt.queries(8)
    text = _launched(tmp_path, lambda: V.attention_fp8(q, bt.cache, **bt.args()))
    assert "attn_prompt_kernel" in text and "attn_join_tiles_kernel" in text
    _check(bt, q)


@pytest.mark.parametrize("d,heads", [(64, 1), (128, 8), (64, 9), (128, 16)])
@pytest.mark.parametrize("n", [2300, 9000, 17000])
def test_attention_single_tokens_in_many_parts(tmp_path, d, heads, n):
    """One sequence and key head: 11, 37 and 68 parts of a tile, so the join takes them in one, two
    and three turns of 32, for tiles of 8 and of 16 rows."""
    bt = Pool([n], [1], 1, d, seed=n)
    q = bt.queries(heads)
    text = _launched(tmp_path, lambda: V.attention_fp8(q, bt.cache, **bt.args()))
    assert "attn_rows_kernel" in text and "attn_join_kernel" in text
    _check(bt, q)


def test_attention_long_beside_short():
    """A tile in more than 32 parts beside tiles that a CTA has whole."""
    bt = Pool([17000, 5, 64, 3000, 1], [1] * 5, 1, 64, seed=9)
    _check(bt, bt.queries(4))
