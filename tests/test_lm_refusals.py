"""CPU: what the 8-bit operators refuse.  Every argument is checked before any device work, so
these calls return on a machine without a GPU; the addresses are never used.  The 64-bit
restatements of tests/lm_ref.py are pinned here as well."""
from __future__ import annotations

import numpy as np
import pytest

from dac_vocoder_decode_gb300 import binding as V
from dac_vocoder_decode_gb300 import build as B
from tests import lm_ref as R

PTR = 1 << 20  # an address that passes the alignment checks


@pytest.fixture(scope="module")
def lib():
    B.build()
    return V.load_library()


def _refused(lib, name, args, text, status=V.VOC_INVALID_ARG):
    assert getattr(lib, name)(*args) == status, text
    assert text in V.vocoder_last_error(), V.vocoder_last_error()


ROWS = dict(x=PTR, ldx=64, residual=PTR, ldr=64, weight=PTR, dtype=V.VOC_LM_BF16,
            mode=V.VOC_LM_RMS, rows=4, d=64, eps=1e-6, sum_out=PTR, lds=64, out8=PTR, ldo=64,
            scale=PTR, stream=None, flags=0)


@pytest.mark.parametrize("change,text", [
    (dict(dtype=3), "dtype"), (dict(mode=3), "mode"), (dict(rows=-1), "sizes"),
    (dict(d=0), "sizes"), (dict(d=1 << 25, ldx=1 << 25), "sizes"), (dict(weight=None), "weight"),
    (dict(mode=V.VOC_LM_NONE), "weight"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(mode=V.VOC_LM_GATED, weight=None), "residual"),
    (dict(residual=None), "sum_out"), (dict(ldx=63), "stride"), (dict(ldr=63), "stride"),
    (dict(lds=63), "stride"), (dict(ldo=63), "stride"), (dict(x=None), "NULL"),
    (dict(out8=None), "NULL"), (dict(scale=None), "NULL"), (dict(x=PTR + 1), "aligned"),
    (dict(dtype=V.VOC_LM_F32, residual=PTR + 2), "aligned"), (dict(scale=PTR + 2), "aligned"),
    (dict(flags=V.VOC_FLAG_PROFILE), "flags"),
    (dict(mode=V.VOC_LM_GATED, weight=None, residual=None, sum_out=None), "stride")])
def test_rows_refusals(lib, change, text):
    _refused(lib, "vocoder_lm_rows_fp8", {**ROWS, **change}.values(), text)


LINEAR = dict(x8=PTR, ldx=64, x_scale=PTR, w8=PTR, ldw=64, w_scale=PTR, bias=PTR, M=4, N=8, K=64,
              out=PTR, ldo=8, out_dtype=V.VOC_LM_BF16, stream=None, flags=0)


@pytest.mark.parametrize("change,text", [
    (dict(out_dtype=-1), "out_dtype"), (dict(M=-1), "sizes"), (dict(N=-1), "sizes"),
    (dict(K=0), "sizes"), (dict(ldx=48), "stride"), (dict(ldw=48), "stride"),
    (dict(ldo=7), "stride"), (dict(ldx=72), "multiples of 16"), (dict(ldw=65), "multiples of 16"),
    (dict(x8=PTR + 8), "16-byte"), (dict(w8=PTR + 1), "16-byte"), (dict(x8=None), "NULL"),
    (dict(w_scale=None), "NULL"), (dict(out=None), "NULL"), (dict(out=PTR + 1), "aligned"),
    (dict(bias=PTR + 2), "aligned"), (dict(flags=1), "flags")])
def test_linear_refusals(lib, change, text):
    _refused(lib, "vocoder_lm_linear_fp8", {**LINEAR, **change}.values(), text)


APPEND = dict(kc=PTR, vc=PTR, ks=PTR, vs=PTR, n_pages=8, kv_heads=2, head_dim=64, k=PTR, ldk=128,
              hsk=64, v=PTR, ldv=128, hsv=64, dtype=V.VOC_LM_BF16, table=PTR, ldt=4, cols=4,
              lens=PTR, cu=PTR, n_seq=2, n_tokens=6, max_q=5, stream=None, flags=0)
CACHE_BAD = [
    (dict(dtype=V.VOC_LM_F32), "dtype", V.VOC_INVALID_ARG),
    (dict(head_dim=96), "head_dim", V.VOC_UNSUPPORTED),
    (dict(n_pages=0), "sizes", V.VOC_INVALID_ARG), (dict(kv_heads=0), "sizes", V.VOC_INVALID_ARG),
    (dict(cols=0), "sizes", V.VOC_INVALID_ARG), (dict(ldt=3), "sizes", V.VOC_INVALID_ARG),
    (dict(n_seq=-1), "batch", V.VOC_INVALID_ARG), (dict(n_seq=70000), "batch", V.VOC_INVALID_ARG),
    (dict(n_seq=0), "without sequences", V.VOC_INVALID_ARG),
    (dict(cu=None), "max_q", V.VOC_INVALID_ARG), (dict(max_q=7), "max_q", V.VOC_INVALID_ARG),
    (dict(kc=None), "NULL", V.VOC_INVALID_ARG), (dict(lens=None), "NULL", V.VOC_INVALID_ARG),
    (dict(vc=PTR + 8), "alignment", V.VOC_INVALID_ARG),
    (dict(table=PTR + 2), "alignment", V.VOC_INVALID_ARG),
    (dict(flags=4), "flags", V.VOC_INVALID_ARG)]


@pytest.mark.parametrize("change,text,status", CACHE_BAD + [
    (dict(k=None), "NULL", V.VOC_INVALID_ARG), (dict(k=PTR + 8), "16-byte", V.VOC_INVALID_ARG),
    (dict(ldv=130), "multiples of 8", V.VOC_INVALID_ARG),
    (dict(hsk=68), "multiples of 8", V.VOC_INVALID_ARG)])
def test_append_refusals(lib, change, text, status):
    _refused(lib, "vocoder_lm_kv_append", {**APPEND, **change}.values(), text, status)


ATTN = dict(q=PTR, ldq=256, hsq=64, dtype=V.VOC_LM_BF16, heads=4, kc=PTR, vc=PTR, ks=PTR, vs=PTR,
            n_pages=8, kv_heads=2, head_dim=64, table=PTR, ldt=4, cols=4, lens=PTR, cu=PTR,
            n_seq=2, n_tokens=6, max_q=5, max_kv=256, softmax_scale=0.125, causal=1, window=0,
            out=PTR, ldo=256, hso=64, ws=None, ws_bytes=0, stream=None, flags=0)


@pytest.mark.parametrize("change,text,status", CACHE_BAD + [
    (dict(heads=3), "multiple of kv_heads", V.VOC_INVALID_ARG),
    (dict(heads=0), "multiple of kv_heads", V.VOC_INVALID_ARG),
    (dict(max_kv=-1), "max_kv", V.VOC_INVALID_ARG), (dict(window=-1), "window", V.VOC_INVALID_ARG),
    (dict(causal=2), "causal", V.VOC_INVALID_ARG),
    (dict(softmax_scale=float("inf")), "softmax_scale", V.VOC_INVALID_ARG),
    (dict(q=None), "NULL", V.VOC_INVALID_ARG), (dict(out=None), "NULL", V.VOC_INVALID_ARG),
    (dict(q=PTR + 1), "alignment", V.VOC_INVALID_ARG),
    (dict(ws=PTR + 4), "alignment", V.VOC_INVALID_ARG)])
def test_attention_refusals(lib, change, text, status):
    _refused(lib, "vocoder_lm_attention", {**ATTN, **change}.values(), text, status)


def test_attention_refuses_rows_beyond_its_counters(lib):
    """heads / kv_heads times max_q rows share a key head; they are counted in 32 bits."""
    call = {**ATTN, "heads": 65536, "kv_heads": 1, "max_q": 1 << 16, "n_tokens": 1 << 18}
    _refused(lib, "vocoder_lm_attention", call.values(), "too many rows", V.VOC_UNSUPPORTED)


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    f8 = torch.zeros(4, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s4 = torch.ones(4)
    for bad in (lambda: V.rows_fp8(torch.zeros(4, 8, dtype=torch.float64)),
                lambda: V.rows_fp8(torch.zeros(8, 4).T),
                lambda: V.rows_fp8(torch.zeros(4, 7), V.VOC_LM_GATED),
                lambda: V.rows_fp8(torch.zeros(4, 8), weight=torch.zeros(7)),
                lambda: V.rows_fp8(torch.zeros(4, 8), weight=torch.zeros(8)),  # CPU tensors
                lambda: V.linear_fp8(f8, s4, f8[:, :32], s4),
                lambda: V.linear_fp8(f8, s4[:3], f8, s4),
                lambda: V.linear_fp8(f8.float(), s4, f8, s4),
                lambda: V.linear_fp8(f8, s4, f8, s4, bias=torch.zeros(3)),
                lambda: V.linear_fp8(f8, s4, f8, s4, out_dtype=torch.float64),
                lambda: V.KVCacheFP8(f8.view(1, 1, 4, 64), f8, s4, s4)):
        with pytest.raises(V.VocoderError) as e:
            bad()
        assert e.value.status == V.VOC_INVALID_ARG


# ------------------------------------------------------------------ the restatements
def test_e4m3_round_is_the_format():
    """Every code's value is a fixed point, midpoints go to even, as torch's conversion does."""
    torch = pytest.importorskip("torch")
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    fin = codes[np.isfinite(codes)]
    np.testing.assert_array_equal(R.e4m3_round(fin), fin)
    grid = np.unique(fin)
    mid = (grid[1:] + grid[:-1]) / 2
    rng = np.random.default_rng(5)
    v = np.concatenate([mid, rng.uniform(-448, 448, 4000), rng.uniform(-0.1, 0.1, 4000)])
    v = v.astype(np.float32)
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(R.e4m3_round(v), ref)
    assert R.e4m3_round(np.inf) == 448 and np.isnan(R.e4m3_round(np.nan))


def test_block_scale():
    assert R.block_scale(0.0) == 2.0 ** -96
    assert R.block_scale(448.0) == 1.0 and R.block_scale(448.1) == 2.0
    assert R.block_scale(7.0) == 2.0 ** -6


def test_append_tokenwise_equals_blockwise():
    """Power-of-two scales: appending one token at a time leaves what one append leaves, but for
    codes that pass through the subnormals."""
    rng = np.random.default_rng(2)
    n, d = 70, 8
    k, v = (rng.standard_normal((n, 1, d)).astype(np.float32) for _ in range(2))
    table = np.array([[1, 0]])
    mk = lambda: [np.zeros((2, 1, 64, d)), np.zeros((2, 1, d, 64)), np.zeros((2, 1)),  # noqa: E731
                  np.zeros((2, 1))]
    one, many = mk(), mk()
    R.append(*one, k, v, table, [n], [n])
    for i in range(n):
        R.append(*many, k[i:i + 1], v[i:i + 1], table, [i + 1], [1])
    np.testing.assert_array_equal(one[2], many[2])
    assert np.max(np.abs(one[0] - many[0])) <= 2.0 ** -9  # one subnormal step


def test_attention_restatement_on_one_key():
    """With one visible key the output is that key's value."""
    kc, vc = np.full((1, 1, 64, 64), 2.0), np.zeros((1, 1, 64, 64))
    vc[0, 0, :, 0] = np.arange(64)
    ks = vs = np.array([[0.5]])
    q = np.ones((1, 2, 64), np.float32)
    o, _, _ = R.attention(q, kc, vc, ks, vs, np.array([[0]]), [1], [1], 0.125)
    np.testing.assert_array_equal(o[0, 1], np.arange(64) * 0.5)
