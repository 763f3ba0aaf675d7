"""GPU: the 8-bit operators of a token model against their 64-bit restatements (tests/lm_ref.py).

Tolerances, derived before any run:
  rows       scale: 32-bit sums of at most d/32 + 32 positive terms in a row, half of whose
             relative error reaches the norm, and 16 more roundings.  Codes: half an e4m3 step
             (2^-4 of the binade, 2^-10 in the subnormals) around n / scale, widened by 1e-5 for
             the 32-bit chain.  The sum is exact: one 32-bit addition, one rounding.
  linear     e4m3 products are exact in 32 bits; K/32 accumulations and 4 more roundings of at most
             2^-23 of sum |x w| each, and one rounding to the output's type.
  append     exact: the scales are powers of two, every rounding is defined.
  attention  weights carry 11 bits (2^-11), scores the error of a 32-bit sum over d (1.5 d 2^-24
             of sum |q k|, twice: maximum and value), the exponential and sums 2^-16; all act on
             sum w |v|; one rounding to the output's type.
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

F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SYNC = V.VOC_FLAG_SYNC


def _np(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _strided(t, extra):
    """The same values with `extra` more elements between rows."""
    if not extra:
        return t
    buf = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), device=t.device).to(t.dtype)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


# ------------------------------------------------------------------ rows
def _check_rows(x, mode, weight, residual, eps, got, d):
    q, scale, total = got
    n, ref, _ = R.rows(_np(x), mode, None if weight is None else _np(weight),
                       None if residual is None else _np(residual), eps)
    rel = ((d / 32 + 32) / 2 + 16) * 2.0 ** -24
    s = _np(scale)
    np.testing.assert_allclose(s, ref, rtol=rel, atol=0)
    v = n / s[:, None]
    with np.errstate(divide="ignore"):
        half = np.maximum(np.exp2(np.floor(np.log2(np.abs(v))) - 4), 2.0 ** -10)
    assert np.all(np.abs(_np(q) - v) <= half * (1 + 1e-4) + 1e-5 * np.abs(v))
    if residual is not None:
        assert torch.equal(total, (x.float() + residual.float()).to(x.dtype))
    else:
        assert total is None


MODES = {"rms": V.VOC_LM_RMS, "none": V.VOC_LM_NONE, "gated": V.VOC_LM_GATED}


@pytest.mark.parametrize("mode", ["rms", "none", "gated"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,d,extra,res", [
    (1, 1, 0, True), (3, 7, 0, True), (5, 64, 0, False), (8, 1024, 0, True), (2, 1000, 8, True),
    (9, 1536, 0, True), (4, 1537, 3, True), (3, 2056, 0, False), (2, 4100, 12, True),
    (1, 8192, 0, True), (2, 16392, 0, True), (1, 70000, 0, False), (700, 96, 0, True)])
def test_rows(mode, dtype, rows, d, extra, res):
    t = TYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(rows * 1000 + d)
    width = 2 * d if mode == "gated" else d
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(t)  # noqa: E731
    x = _strided(mk(rows, width) * 3, extra)
    residual = _strided(mk(rows, width), extra) if res and mode != "gated" else None
    weight = (1 + 0.3 * mk(d)).to(t) if mode == "rms" else None
    got = V.rows_fp8(x, MODES[mode], weight=weight, residual=residual, eps=1e-5, flags=SYNC)
    _check_rows(x, mode, weight, residual, 1e-5, got, d)
    assert got[0].stride(0) % 16 == 0 or rows == 1


@pytest.mark.parametrize("d", [40, 1024, 1031, 5000])
@pytest.mark.parametrize("big", [1e30, 3e4, 1e-12, 1e-30])
def test_rows_far_magnitudes(d, big):
    """Squares that would overflow or vanish in 32 bits."""
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(4, d, generator=g, device="cuda") * big
    x[1] = 0
    w = torch.ones(d, device="cuda")
    for eps in (1e-6, 0.0):
        _check_rows(x, "rms", w, None, eps, V.rows_fp8(x, weight=w, eps=eps, flags=SYNC), d)
    _check_rows(x, "none", None, None, 0, V.rows_fp8(x, V.VOC_LM_NONE, flags=SYNC), d)


@pytest.mark.parametrize("d", [24, 1024, 1025, 9000])
def test_rows_nonfinite_rows_stay_alone(d):
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(6, d, generator=g, device="cuda").bfloat16()
    w = torch.ones(d, device="cuda").bfloat16()
    clean = V.rows_fp8(x, weight=w, flags=SYNC)
    y = x.clone()
    y[1, d // 2] = float("nan")
    y[4, d - 1] = float("inf")
    q, scale, _ = V.rows_fp8(y, weight=w, flags=SYNC)
    keep = [0, 2, 3, 5]
    assert torch.equal(scale[keep], clean[1][keep])
    assert torch.equal(q[keep].view(torch.uint8), clean[0][keep].view(torch.uint8))
    assert torch.isnan(scale[1]) and torch.isnan(q[1].float()).all()
    assert torch.isnan(q[4].float() * scale[4]).all()


@pytest.mark.parametrize("d", [1024, 1030])
def test_rows_sum_in_place(d):
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r = (torch.randn(70, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.rand(d, generator=g, device="cuda").bfloat16()
    ref = V.rows_fp8(x, weight=w, residual=r, flags=SYNC)
    for place in (x, r):
        args = dict(x=x.clone(), residual=r.clone())
        out = args["x"] if place is x else args["residual"]
        q, s, total = V.rows_fp8(args["x"], weight=w, residual=args["residual"], sum_out=out,
                                 flags=SYNC)
        assert total is out and torch.equal(out, ref[2])
        assert torch.equal(s, ref[1]) and torch.equal(q.view(torch.uint8), ref[0].view(torch.uint8))


def test_rows_empty():
    q, s, _ = V.rows_fp8(torch.zeros(0, 64, device="cuda"), V.VOC_LM_NONE, flags=SYNC)
    assert q.shape == (0, 64) and s.shape == (0,)


# ------------------------------------------------------------------ linear
def _codes(g, rows, k, extra=0):
    pad = (k + 15) // 16 * 16 + extra
    v = torch.randn(rows, k, generator=g, device="cuda") * 90
    buf = torch.full((rows, pad), 0x7f, dtype=torch.uint8, device="cuda")  # NaN beyond the row
    buf[:, :k] = v.clamp(-448, 448).to(F8).view(torch.uint8)
    return buf.view(F8)[:, :k]


def _check_linear(x, xs, w, ws, bias, y):
    X, W = _np(x) * _np(xs)[:, None], _np(w) * _np(ws)[:, None]
    ref, mag = X @ W.T, np.abs(X) @ np.abs(W).T
    if bias is not None:
        ref, mag = ref + _np(bias), mag + np.abs(_np(bias))
    tol = (x.shape[1] / 32 + 4) * 2.0 ** -23 * mag + UNIT[y.dtype] * np.abs(ref)
    assert np.all(np.abs(_np(y) - ref) <= tol)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,k,n,bias,extra", [
    (1, 1, 1, True, 0), (1, 16, 7, False, 16), (3, 100, 129, True, 0), (8, 1024, 1536, True, 0),
    (16, 257, 64, False, 32), (17, 128, 128, True, 0), (33, 4096, 200, False, 0),
    (100, 2000, 131, True, 48), (128, 640, 256, False, 0), (129, 384, 513, True, 0),
    (257, 512, 300, True, 0), (300, 1537, 1030, False, 0), (520, 256, 256, True, 0),
    (1000, 1024, 768, False, 0), (2049, 144, 515, True, 0)])
def test_linear(out, m, k, n, bias, extra):
    g = torch.Generator(device="cuda").manual_seed(m + 7 * k + n)
    x, w = _codes(g, m, k, extra), _codes(g, n, k, extra)
    xs = torch.rand(m, generator=g, device="cuda") / 16 + 0.01
    ws = torch.rand(n, generator=g, device="cuda") / (16 * k ** 0.5) + 0.001
    b = torch.randn(n, generator=g, device="cuda") if bias else None
    y = V.linear_fp8(x, xs, w, ws, bias=b, out_dtype=TYPES[out], flags=SYNC)
    _check_linear(x, xs, w, ws, b, y)


@pytest.mark.parametrize("m", [5, 300, 700])
def test_linear_into_a_strided_output(m):
    """Rows of a wider buffer at an odd stride; what lies between stays."""
    g = torch.Generator(device="cuda").manual_seed(m)
    x, w = _codes(g, m, 320), _codes(g, 259, 320)
    xs, ws = torch.rand(m, device="cuda"), torch.rand(259, device="cuda") / 100
    buf = torch.full((m, 267), -7.0, dtype=torch.bfloat16, device="cuda")
    V.linear_fp8(x, xs, w, ws, out=buf[:, 3:262], flags=SYNC)
    _check_linear(x, xs, w, ws, None, buf[:, 3:262])
    assert torch.all(buf[:, :3] == -7) and torch.all(buf[:, 262:] == -7)


@pytest.mark.parametrize("m", [9, 400])
def test_linear_nan_rows_and_channels_stay_alone(m):
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = _codes(g, m, 288), _codes(g, 300, 288)
    xs, ws = torch.ones(m, device="cuda"), torch.ones(300, device="cuda") / 100
    clean = V.linear_fp8(x, xs, w, ws, flags=SYNC)
    x.view(torch.uint8)[4, 100] = 0x7f
    w.view(torch.uint8)[17, 287] = 0xff
    xs[2] = float("nan")
    y = V.linear_fp8(x, xs, w, ws, flags=SYNC)
    bad = torch.zeros(m, 300, dtype=torch.bool, device="cuda")
    bad[4], bad[2], bad[:, 17] = True, True, True
    assert torch.equal(torch.isnan(y), bad)
    assert torch.equal(y[~bad], clean[~bad])


def test_linear_repeats_bit_for_bit():
    g = torch.Generator(device="cuda").manual_seed(9)
    for m, k, n in ((7, 4096, 512), (600, 1024, 640)):
        x, w = _codes(g, m, k), _codes(g, n, k)
        xs, ws = torch.rand(m, device="cuda"), torch.rand(n, device="cuda")
        y = [V.linear_fp8(x, xs, w, ws, out_dtype=torch.float32, flags=SYNC) for _ in range(3)]
        assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])


def test_linear_empty():
    g = torch.Generator(device="cuda").manual_seed(9)
    w = _codes(g, 8, 32)
    y = V.linear_fp8(w[:0], torch.ones(0, device="cuda"), w, torch.ones(8, device="cuda"))
    assert y.shape == (0, 8)


# ------------------------------------------------------------------ cache
class Batch:
    """Sequences over a shuffled pool whose unused slots hold NaN codes."""

    def __init__(self, lens, new, kv_heads, d, seed=0, spare_cols=1, filled=True):
        rng = np.random.default_rng(seed)
        self.lens, self.new, self.kv_heads, self.d = lens, new, kv_heads, d
        blocks = [max(0, (n + 63) // 64) for n in lens]
        self.pages = sum(blocks) + 2
        order = rng.permutation(self.pages)
        cols = max(blocks + [0]) + spare_cols
        self.table = np.full((len(lens), cols), -1, np.int32)
        at = 0
        for b, n in enumerate(blocks):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.spare = order[at:]
        # values on the e4m3 grid, scales of their own for every block and head
        self.ks, self.vs = (np.exp2(rng.integers(-9, -5, (self.pages, kv_heads))).astype(np.float32)
                            for _ in range(2))
        self.kc = R.e4m3_round(rng.standard_normal((self.pages, kv_heads, 64, d)) * 100)
        self.vc = R.e4m3_round(rng.standard_normal((self.pages, kv_heads, d, 64)) * 100)
        used = np.zeros((self.pages, 64), bool)
        for b, n in enumerate(lens):
            held = n if filled else n - new[b]
            for j in range(max(0, held)):
                used[self.table[b, j // 64], j % 64] = True
        self.kc = np.where(used[:, None, :, None], self.kc, np.nan)
        self.vc = np.where(used[:, None, None, :], self.vc, np.nan)
        f8 = lambda a: torch.from_numpy(a.astype(np.float32)).cuda().to(F8)  # noqa: E731
        self.cache = V.KVCacheFP8(f8(self.kc), f8(self.vc), torch.from_numpy(self.ks).cuda(),
                                  torch.from_numpy(self.vs).cuda())
        self.t_table = torch.from_numpy(self.table).cuda()
        self.t_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        equal = len(set(new)) == 1
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.cu = None if equal else torch.from_numpy(cu).cuda()
        self.total, self.max_q = sum(new), max(new)
        self.rng = rng

    def args(self):
        return dict(page_table=self.t_table, kv_lens=self.t_lens, cu_q=self.cu, max_q=self.max_q)


def _check_append(bt, k, v):
    """Appends on both sides and compares everything, untouched slots included."""
    V.kv_append_fp8(bt.cache, k, v, flags=SYNC, **bt.args())
    R.append(bt.kc, bt.vc, bt.ks, bt.vs, _np(k).astype(np.float32), _np(v).astype(np.float32),
             bt.table, bt.lens, bt.new)
    np.testing.assert_array_equal(bt.cache.k_scale.cpu().numpy(), bt.ks)
    np.testing.assert_array_equal(bt.cache.v_scale.cpu().numpy(), bt.vs)
    np.testing.assert_array_equal(_np(bt.cache.k), bt.kc)
    np.testing.assert_array_equal(_np(bt.cache.v), bt.vc)


APPENDS = [([1], [1]), ([64], [64]), ([65], [1]), ([130], [129]), ([63, 200, 1], [63, 73, 1]),
           ([250, 249, 64, 1], [1, 1, 1, 1]), ([100, 64, 90], [3, 0, 26]), ([70, 1, 128], [2, 2, 2]),
           ([300], [237])]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,heads", [(64, 1), (128, 3)])
@pytest.mark.parametrize("lens,new", APPENDS)
def test_append(dtype, d, heads, lens, new):
    bt = Batch(lens, new, heads, d, seed=len(lens) + lens[0], filled=False)
    k, v = (torch.from_numpy(bt.rng.standard_normal((bt.total, heads, d)) *
                             np.exp2(bt.rng.integers(-3, 4, (bt.total, 1, 1)))).cuda()
            .to(TYPES[dtype]) for _ in range(2))
    _check_append(bt, k, v)


@pytest.mark.parametrize("d", [64, 128])
def test_append_from_a_fused_projection(d):
    """k and v as slices of one q|k|v buffer."""
    bt = Batch([70, 20, 140], [6, 20, 1], 2, d, filled=False)
    qkv = torch.from_numpy(bt.rng.standard_normal((bt.total, 8, d))).cuda().bfloat16()
    _check_append(bt, qkv[:, 4:6], qkv[:, 6:8])


@pytest.mark.parametrize("lens,new", [([40], [40]), ([40], [3]), ([130], [100])])
def test_append_nonfinite_and_extremes(lens, new):
    bt = Batch(lens, new, 2, 64, filled=False)
    k, v = (torch.from_numpy(bt.rng.standard_normal((bt.total, 2, 64))).cuda().bfloat16()
            for _ in range(2))
    k[0, 0, 3], k[1, 0, 5] = float("inf"), float("nan")
    v[2, 1, 7], v[1, 1, 8] = float("nan"), -float("inf")
    k[2, 1] *= 1e30
    v[0, 0] *= 1e-35
    _check_append(bt, k, v)
    assert not torch.isnan(bt.cache.v.float()[torch.from_numpy(bt.table[0, :1]).long().cuda()]
                           [..., :lens[0] % 64 or 64]).any() or lens[0] > 64


def test_append_zeros_and_whole_blocks_of_inf():
    bt = Batch([64, 64], [64, 64], 1, 64, filled=False)
    k = torch.zeros(128, 1, 64, device="cuda").bfloat16()
    v = torch.full_like(k, float("inf"))
    _check_append(bt, k, v)


def test_append_skips_what_has_no_page():
    """Pages outside the pool and blocks beyond the table take nothing."""
    bt = Batch([200, 64], [200, 64], 1, 64, filled=False, spare_cols=0)
    bt.table[0, 1], bt.table[0, 2] = bt.pages, -5
    bt.table = np.ascontiguousarray(bt.table[:, :3])
    bt.t_table = torch.from_numpy(bt.table).cuda()
    k, v = (torch.from_numpy(bt.rng.standard_normal((264, 1, 64))).cuda().bfloat16()
            for _ in range(2))
    _check_append(bt, k, v)


def test_append_more_tokens_than_the_length():
    """kv_len below the number of new tokens: the first ones have negative positions and go."""
    bt = Batch([5], [8], 1, 64, filled=False)
    k, v = (torch.from_numpy(bt.rng.standard_normal((8, 1, 64))).cuda().bfloat16()
            for _ in range(2))
    _check_append(bt, k, v)


# ------------------------------------------------------------------ attention
def _check_attention(bt, q, causal=True, window=0, scale=None, max_kv=None, **kw):
    scale = bt.d ** -0.5 if scale is None else scale
    o = V.attention_fp8(q, bt.cache, softmax_scale=scale, causal=causal, window=window,
                        max_kv=max_kv, flags=SYNC, **bt.args(), **kw)
    ref, mag, s = R.attention(_np(q), bt.kc, bt.vc, bt.ks.astype(np.float64),
                              bt.vs.astype(np.float64), bt.table, bt.lens, bt.new, scale, causal,
                              window)
    rel = 2.0 ** -11 + 2.0 ** -16 + 2 * 1.5 * bt.d * 2.0 ** -24 * s
    tol = rel[..., None] * mag + UNIT[q.dtype] * np.abs(ref) + 2.0 ** -30
    got = _np(o)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-30)))
    return o


def _queries(bt, heads, dtype="bf16", amp=1.0):
    return (torch.from_numpy(bt.rng.standard_normal((bt.total, heads, bt.d))) * amp).cuda().to(
        TYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,heads,kv_heads", [(64, 16, 16), (64, 4, 1), (128, 8, 2), (128, 7, 1),
                                              (64, 40, 2), (128, 3, 3)])
@pytest.mark.parametrize("lens", [[1], [64], [65, 1, 63], [250, 31, 129, 700], [2000, 5]])
def test_attention_single_tokens(dtype, d, heads, kv_heads, lens):
    bt = Batch(lens, [1] * len(lens), kv_heads, d, seed=lens[0])
    _check_attention(bt, _queries(bt, heads, dtype))


CHUNKS = [([5], [5]), ([64], [64]), ([200, 37, 1], [17, 37, 1]), ([130, 300], [129, 3]),
          ([333], [333]), ([90, 64, 70], [0, 64, 5]), ([700, 129], [150, 129])]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,heads,kv_heads", [(64, 4, 2), (128, 4, 1), (128, 2, 2), (64, 7, 1)])
@pytest.mark.parametrize("lens,new", CHUNKS)
def test_attention_chunks(dtype, d, heads, kv_heads, lens, new):
    bt = Batch(lens, new, kv_heads, d, seed=lens[0])
    _check_attention(bt, _queries(bt, heads, dtype))


@pytest.mark.parametrize("window", [1, 2, 63, 64, 72, 250, 5000])
@pytest.mark.parametrize("lens,new", [([300, 64, 1], [1, 1, 1]), ([333, 200], [200, 70]),
                                      ([900], [129])])
def test_attention_window(window, lens, new):
    bt = Batch(lens, new, 2, 64, seed=window)
    _check_attention(bt, _queries(bt, 4), window=window)


@pytest.mark.parametrize("lens,new", [([300, 64], [1, 1]), ([200, 130], [60, 130])])
@pytest.mark.parametrize("window", [0, 100])
def test_attention_not_causal(lens, new, window):
    bt = Batch(lens, new, 2, 128, seed=5)
    _check_attention(bt, _queries(bt, 4), causal=False, window=window)


@pytest.mark.parametrize("lens,new", [([0, 70], [1, 1]), ([3, 200], [6, 6]), ([0, 200], [9, 150]),
                                      ([10, 300], [150, 150])])
def test_attention_rows_without_keys_are_zero(lens, new):
    """Empty sequences, and queries whose position would be negative."""
    bt = Batch(lens, new, 2, 64)
    o = _check_attention(bt, _queries(bt, 4))
    empty = new[0] - lens[0]
    assert torch.all(o[:empty] == 0)


def test_attention_missing_pages_hold_no_tokens():
    for new in ([1, 1], [70, 200]):
        bt = Batch([300, 330], new, 2, 64)
        bt.table[0, 1], bt.table[1, 0], bt.table[1, 5] = -1, bt.pages, -7
        bt.t_table = torch.from_numpy(bt.table).cuda()
        _check_attention(bt, _queries(bt, 4))


def test_attention_length_beyond_the_table():
    for new in ([1], [140]):
        bt = Batch([300], new, 1, 64, spare_cols=0)
        bt.table = np.ascontiguousarray(bt.table[:, :3])
        bt.t_table = torch.from_numpy(bt.table).cuda()
        _check_attention(bt, _queries(bt, 2), causal=False)


@pytest.mark.parametrize("new", [[1, 1], [40, 170]])
def test_attention_strided_queries_and_output(new):
    """q as a slice of a fused projection at an odd offset, the output into a wider buffer."""
    bt = Batch([200, 170], new, 2, 64)
    buf = torch.from_numpy(bt.rng.standard_normal((bt.total, 9, 65))).cuda().bfloat16()
    q = buf[:, 1:7, 1:]
    out = torch.full((bt.total, 8, 66), -3.0, device="cuda").bfloat16()
    o = _check_attention(bt, q, out=out[:, 1:7, :64])
    assert o.data_ptr() == out[:, 1:7].data_ptr()
    assert torch.all(out[:, 0] == -3) and torch.all(out[:, 7] == -3)
    assert torch.all(out[:, :, 64:] == -3)


@pytest.mark.parametrize("new", [[1, 1, 1], [1, 130, 20]])
def test_attention_block_scales_far_apart(new):
    """Blocks whose scales differ by many powers of two, scores from sharp to flat."""
    bt = Batch([500, 130, 300], new, 1, 64, seed=4)
    e = bt.rng.integers(-40, 41, bt.vs.shape)
    bt.vs = np.exp2(e).astype(np.float32)
    bt.cache.v_scale.copy_(torch.from_numpy(bt.vs).cuda())
    bt.ks = (bt.ks * np.exp2(bt.rng.integers(-3, 4, bt.ks.shape))).astype(np.float32)
    bt.cache.k_scale.copy_(torch.from_numpy(bt.ks).cuda())
    _check_attention(bt, _queries(bt, 2))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("amp", [1e-4, 20.0])
@pytest.mark.parametrize("new", [[1, 1], [129, 64]])
def test_attention_query_magnitudes(dtype, amp, new):
    bt = Batch([400, 64], new, 2, 64, seed=8)
    _check_attention(bt, _queries(bt, 4, dtype, amp))


@pytest.mark.parametrize("new", [[1, 1], [150, 64]])
def test_attention_nan_stays_with_who_sees_it(new):
    """A NaN query poisons its own row; a token appended with a NaN poisons the queries that see
    it and no other."""
    bt = Batch([220, 64], new, 1, 64, seed=3, filled=False)
    k, v = (torch.from_numpy(bt.rng.standard_normal((bt.total, 1, 64))).cuda().bfloat16()
            for _ in range(2))
    k2, v2 = k.clone(), v.clone()
    tok = new[0] // 2  # of the first sequence
    v2[tok, 0, 9] = float("nan")
    q = _queries(bt, 2)
    V.kv_append_fp8(bt.cache, k, v, flags=SYNC, **bt.args())
    clean = V.attention_fp8(q, bt.cache, flags=SYNC, **bt.args())
    assert torch.isfinite(clean).all()
    V.kv_append_fp8(bt.cache, k2, v2, flags=SYNC, **bt.args())
    q2 = q.clone()
    q2[bt.total - 1, 1, 3] = float("nan")
    o = V.attention_fp8(q2, bt.cache, flags=SYNC, **bt.args())
    bad = torch.zeros(bt.total, 2, dtype=torch.bool, device="cuda")
    bad[tok:new[0]] = True
    bad[bt.total - 1, 1] = True
    assert torch.equal(torch.isnan(o).all(-1), bad) and torch.equal(torch.isnan(o).any(-1), bad)
    assert torch.equal(o[~bad], clean[~bad])


def test_attention_repeats_bit_for_bit_and_any_split():
    """The same call gives the same bits; another max_kv (another split) the same within the
    tolerance."""
    bt = Batch([3000, 17], [1, 1], 1, 64, seed=6)
    q = _queries(bt, 4)
    a = _check_attention(bt, q, max_kv=3000)
    b = _check_attention(bt, q, max_kv=3000)
    assert torch.equal(a, b)
    _check_attention(bt, q, max_kv=100)
    _check_attention(bt, q, max_kv=100000)


def test_attention_own_workspace_and_its_refusal():
    bt = Batch([4000], [1], 1, 64, seed=6)
    q = _queries(bt, 4)
    need = V.load_library().vocoder_lm_attention_ws_bytes(1, 1, 4, 1, 64, 4000, 0)
    if need == 0:
        pytest.skip("this call needs no workspace")
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    _check_attention(bt, q, max_kv=4000, ws=ws)
    with pytest.raises(V.VocoderError) as e:
        V.attention_fp8(q, bt.cache, max_kv=4000, ws=ws[:need - 16], **bt.args())
    assert e.value.status == V.VOC_WORKSPACE_TOO_SMALL


def test_attention_far_offsets():
    """A pool beyond 2^32 bytes: pages at both ends of it."""
    pages = (1 << 32) // (4 * 64 * 128) + 40
    if torch.cuda.mem_get_info()[0] < 3 * (pages * 4 * 64 * 128):
        pytest.skip("not enough device memory")
    bt = Batch([200, 100], [1, 1], 4, 128, seed=2)
    at = np.concatenate([np.arange(3), np.arange(pages - bt.pages + 3, pages)])
    big = V.KVCacheFP8.empty(pages, 4, 128)
    idx = torch.from_numpy(at).cuda()
    for name in ("k", "v"):
        getattr(big, name).view(torch.uint8)[idx] = getattr(bt.cache, name).view(torch.uint8)
    for name in ("k_scale", "v_scale"):
        getattr(big, name)[idx] = getattr(bt.cache, name)
    table = torch.from_numpy(np.where(bt.table >= 0, at[bt.table], -1).astype(np.int32)).cuda()
    q = _queries(bt, 8)
    ref = V.attention_fp8(q, bt.cache, flags=SYNC, **bt.args())
    got = V.attention_fp8(q, big, table, bt.t_lens, flags=SYNC)
    assert torch.equal(ref, got)
    k, v = (torch.randn(2, 4, 128, device="cuda").bfloat16() for _ in range(2))
    V.kv_append_fp8(bt.cache, k, v, flags=SYNC, **bt.args())
    V.kv_append_fp8(big, k, v, table, bt.t_lens, flags=SYNC)
    assert torch.equal(big.k.view(torch.uint8)[idx], bt.cache.k.view(torch.uint8))
    assert torch.equal(big.v.view(torch.uint8)[idx], bt.cache.v.view(torch.uint8))


RAGGED = [[1, 40, 3000, 0, 64, 17, 1500, 700], [2900, 1], [5, 5, 5, 2048], [1, 0, 2, 4100]]


@pytest.mark.parametrize("d,heads,kv_heads", [(64, 8, 8), (128, 7, 1), (128, 20, 2), (64, 1, 1)])
@pytest.mark.parametrize("lens", RAGGED)
def test_attention_shares_of_ragged_lengths(d, heads, kv_heads, lens):
    """Long and short sequences side by side: CTAs whose share ends inside a tile, before its first
    block, or holds many tiles; tiles in more than 32 parts."""
    bt = Batch(lens, [1] * len(lens), kv_heads, d, seed=3)
    q = _queries(bt, heads)
    _check_attention(bt, q, max_kv=16000)
    if len(lens) > 2:
        bt.table[2, 0] = -1  # and a page that holds no tokens
        bt.t_table = torch.from_numpy(bt.table).cuda()
        _check_attention(bt, q, max_kv=16000)


MANY = [([333], [333]), ([200, 130, 700], [200, 1, 150]), ([0, 520], [9, 300])]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,heads,kv_heads", [(64, 16, 16), (128, 16, 16), (64, 32, 16)])
@pytest.mark.parametrize("lens,new", MANY)
def test_attention_many_rows_and_heads(dtype, d, heads, kv_heads, lens, new):
    bt = Batch(lens, new, kv_heads, d, seed=lens[0])
    _check_attention(bt, _queries(bt, heads, dtype))


@pytest.mark.parametrize("lens,new", [([900, 3, 70, 500], [200, 3, 40, 1]), ([1000], [700]),
                                      ([600, 600], [33, 600])])
@pytest.mark.parametrize("window", [0, 90])
def test_attention_short_caches_with_many_rows(lens, new, window):
    """Up to 16 blocks of keys: tiles of 16 rows while they all run at once, tiles of 256 beyond."""
    for heads, kv_heads in ((4, 1), (16, 4), (12, 12)):
        bt = Batch(lens, new, kv_heads, 64, seed=heads)
        _check_attention(bt, _queries(bt, heads), window=window)


@pytest.mark.parametrize("n_seq", [600])
def test_attention_many_sequences(n_seq):
    """More sequences than CTAs count through; a tile or two for each."""
    lens = [40 + i % 50 for i in range(n_seq)]
    new = [min(n, 36 + i % 3) for i, n in enumerate(lens)]
    bt = Batch(lens, new, 1, 64, seed=1)
    _check_attention(bt, _queries(bt, 1))


@pytest.fixture
def long_announced(monkeypatch):
    """Announces every length as 4000: more than 32 rows then take tiles of 256 rows, their keys in
    parts, and fewer rows shares."""
    real = V.attention_fp8
    monkeypatch.setattr(V, "attention_fp8",
                        lambda *a, max_kv=None, **kw: real(*a, max_kv=max_kv or 4000, **kw))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,heads,kv_heads", [(64, 4, 2), (128, 4, 1), (128, 2, 2), (64, 7, 1)])
@pytest.mark.parametrize("lens,new", CHUNKS + MANY)
def test_attention_chunks_in_parts(long_announced, dtype, d, heads, kv_heads, lens, new):
    test_attention_chunks(dtype, d, heads, kv_heads, lens, new)


@pytest.mark.parametrize("window", [1, 2, 63, 64, 72, 250])
@pytest.mark.parametrize("lens,new", [([300, 64, 1], [1, 1, 1]), ([333, 200], [200, 70]),
                                      ([900], [129])])
def test_attention_window_in_parts(long_announced, window, lens, new):
    test_attention_window(window, lens, new)


@pytest.mark.parametrize("case,args", [
    (test_attention_not_causal, ([200, 130], [60, 130], 0)),
    (test_attention_not_causal, ([200, 130], [60, 130], 100)),
    (test_attention_rows_without_keys_are_zero, ([0, 200], [9, 150])),
    (test_attention_rows_without_keys_are_zero, ([10, 300], [150, 150])),
    (test_attention_missing_pages_hold_no_tokens, ()),
    (test_attention_length_beyond_the_table, ()),
    (test_attention_strided_queries_and_output, ([40, 170],)),
    (test_attention_block_scales_far_apart, ([1, 130, 20],)),
    (test_attention_query_magnitudes, ("bf16", 1e-4, [129, 64])),
    (test_attention_query_magnitudes, ("f16", 20.0, [129, 64])),
    (test_attention_nan_stays_with_who_sees_it, ([1, 1],)),
    (test_attention_nan_stays_with_who_sees_it, ([150, 64],))],
    ids=lambda v: v.__name__[5:] if callable(v) else "-".join(map(str, v)))
def test_attention_in_parts(long_announced, case, args):
    case(*args)


def test_attention_workspace_holds_for_any_number_of_tokens():
    """The size asked for without the number of tokens covers the fewest and the most."""
    lib = V.load_library()
    for new in ([200, 1, 1], [200, 200, 200], [1, 200, 90]):
        bt = Batch([700, 650, 900], new, 2, 64, seed=2)
        q = _queries(bt, 2)
        need = lib.vocoder_lm_attention_ws_bytes(3, 200, 2, 2, 64, 4000, 0)
        ws = torch.full((max(need, 16),), 0xff, dtype=torch.uint8, device="cuda")
        _check_attention(bt, q, max_kv=4000, ws=ws)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,at,ld", [(515, 0, 515), (514, 0, 514), (513, 1, 514), (512, 3, 520),
                                     (500, 4, 504), (516, 2, 518)])
def test_linear_output_rows_on_any_start(out, n, at, ld):
    """Rows of every alignment from many tokens; what lies beside them stays."""
    g = torch.Generator(device="cuda").manual_seed(n + at)
    m, k = 4100, 64
    x, w = _codes(g, m, k), _codes(g, n, k)
    xs, ws = (torch.rand(r, generator=g, device="cuda") / 8 + 0.01 for r in (m, n))
    buf = torch.full((m, ld), -7.0, dtype=TYPES[out], device="cuda")
    V.linear_fp8(x, xs, w, ws, out=buf[:, at:at + n], flags=SYNC)
    _check_linear(x, xs, w, ws, None, buf[:, at:at + n])
    assert torch.all(buf[:, :at] == -7) and torch.all(buf[:, at + n:] == -7)


# ------------------------------------------------------------------ streams and empties
def test_empty_batches():
    bt = Batch([70], [1], 1, 64)
    none = torch.zeros(0, 1, 64, device="cuda").bfloat16()
    t0, l0 = bt.t_table[:0], bt.t_lens[:0]
    V.kv_append_fp8(bt.cache, none, none, t0, l0, max_q=0, flags=SYNC)
    assert V.attention_fp8(none, bt.cache, t0, l0, max_q=0, flags=SYNC).shape == (0, 1, 64)


def test_operators_on_a_stream_of_their_own():
    """A layer's chain on a side stream, tensors made there, against the default stream."""
    bt = Batch([300, 64], [1, 1], 2, 64, seed=11)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, 256, generator=g, device="cuda").bfloat16()
    w, ws = _codes(g, 256, 256), torch.rand(256, generator=g, device="cuda") / 100
    nw = torch.ones(256, device="cuda").bfloat16()

    def chain(stream=None):
        q8, s, _ = V.rows_fp8(x, weight=nw, stream=stream)
        y = V.linear_fp8(q8, s, w, ws, stream=stream)
        return V.attention_fp8(y.view(2, 4, 64), bt.cache, bt.t_table, bt.t_lens, stream=stream)

    ref = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = []
    for _ in range(20):
        out.append(chain(side))
        junk = torch.full((1 << 16,), 3.0, device="cuda")  # may reuse what the chain dropped
        del junk
    side.synchronize()
    with torch.cuda.stream(side):
        out.append(chain())
    side.synchronize()
    for o in out:
        assert torch.equal(o, ref)


# ------------------------------------------------------------------ the binding's two ways
def test_compiled_and_python_marshalling_agree(monkeypatch):
    """The compiled binding and the Python one make the same calls, with defaults and with every
    operand given; both refuse wrong tensors with VOC_INVALID_ARG."""
    V._lm_setup()
    if V._LM.fast is None:
        pytest.skip("lm_torch.so is not built")
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r = (torch.randn(5, 96, generator=g, device="cuda").bfloat16() for _ in range(2))
    w8, ws = _codes(g, 70, 96), torch.rand(70, generator=g, device="cuda")
    bias = torch.randn(70, generator=g, device="cuda")
    nw = torch.rand(96, generator=g, device="cuda").bfloat16()

    def calls():
        bt = Batch([70, 300, 64], [6, 1, 64], 2, 64, seed=1, filled=False)
        single = Batch([900, 5], [1, 1], 2, 64, seed=2)
        k, v = (torch.from_numpy(bt.rng.standard_normal((bt.total, 2, 64))).cuda().bfloat16()
                for _ in range(2))
        out = [*V.rows_fp8(x, weight=nw, residual=r),
               *V.rows_fp8(x, V.VOC_LM_NONE, scale=torch.empty(5, device="cuda"),
                           out=torch.empty(5, 96, device="cuda").to(F8))[:2],
               *V.rows_fp8(x[:, :70], V.VOC_LM_GATED)[:2]]
        for kw in (dict(), dict(bias=bias, out_dtype=torch.float32),
                   dict(out=torch.empty(5, 75, device="cuda").half()[:, :70])):
            out.append(V.linear_fp8(out[0], out[1], w8, ws, **kw))
        V.kv_append_fp8(bt.cache, k, v, **bt.args())
        q, q1 = _queries(bt, 4), _queries(single, 6, "f16")
        out += [bt.cache.k, bt.cache.v, bt.cache.k_scale, bt.cache.v_scale,
                V.attention_fp8(q, bt.cache, **bt.args()),
                V.attention_fp8(q, bt.cache, window=20, causal=False, softmax_scale=0.3,
                                out=torch.empty_like(q), max_kv=300, **bt.args()),
                V.attention_fp8(q1, single.cache, **single.args()),
                V.attention_fp8(q1, single.cache, max_kv=900, ws=torch.empty(
                    1 << 20, dtype=torch.uint8, device="cuda"), **single.args())]
        torch.cuda.synchronize()
        for bad in (lambda: V.rows_fp8(x.double()), lambda: V.rows_fp8(x, weight=nw[:9]),
                    lambda: V.rows_fp8(x.T), lambda: V.rows_fp8(x, weight=nw.float()),
                    lambda: V.rows_fp8(x, V.VOC_LM_NONE, sum_out=x),
                    lambda: V.rows_fp8(x), lambda: V.rows_fp8(x.cpu(), V.VOC_LM_NONE),
                    lambda: V.linear_fp8(out[0], out[1][:3], w8, ws),
                    lambda: V.linear_fp8(out[0], out[1], w8[:, :90], ws),
                    lambda: V.linear_fp8(out[0], out[1], w8, ws, out_dtype=torch.int32),
                    lambda: V.linear_fp8(out[0][:, 3:], out[1], w8[:, 3:], ws),
                    lambda: V.KVCacheFP8(bt.cache.k, bt.cache.k, bt.cache.k_scale, bt.cache.v_scale)
                    if bt.cache.k.shape != bt.cache.v.shape else V.rows_fp8(x),
                    lambda: V.kv_append_fp8(bt.cache, k, v.half(), **bt.args()),
                    lambda: V.kv_append_fp8(bt.cache, k, v, bt.t_table.long(), bt.t_lens),
                    lambda: V.kv_append_fp8(bt.cache, k, v, bt.t_table, bt.t_lens, max_q=1),
                    lambda: V.attention_fp8(q[:, :3], bt.cache, **bt.args()),
                    lambda: V.attention_fp8(q, bt.cache, window=-1, **bt.args()),
                    lambda: V.attention_fp8(q, bt.cache, out=q[:, :2], **bt.args())):
            with pytest.raises(V.VocoderError) as e:
                bad()
            assert e.value.status == V.VOC_INVALID_ARG
        return out

    fast = calls()
    monkeypatch.setattr(V._LM, "fast", None)
    slow = calls()
    assert len(fast) == len(slow)
    for a, b in zip(fast, slow):
        assert (a is None and b is None) or (
            a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride() and
            torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)))
