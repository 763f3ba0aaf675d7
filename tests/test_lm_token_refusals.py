"""CPU: what the operators beside the 8-bit ones refuse (heads turned by position, low-rank adapters, log
probabilities).  Every argument is checked before any device work, so these calls return on a machine without
a GPU; the addresses are never used."""
from __future__ import annotations

import math

import pytest

from dac_vocoder_decode_gb300 import binding as V
from dac_vocoder_decode_gb300 import build as B

PTR = 1 << 20  # an address that passes the alignment checks
BAD, NOT = V.VOC_INVALID_ARG, V.VOC_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    B.build()
    return V.load_library()


def _refused(lib, name, args, text, status=BAD):
    assert getattr(lib, name)(*args) == status, text
    assert text in V.vocoder_last_error(), V.vocoder_last_error()


ROTATE = dict(q=PTR, ldq=256, hsq=64, heads=4, k=PTR, ldk=128, hsk=64, kv_heads=2, head_dim=64,
              dtype=V.VOC_LM_BF16, q_weight=PTR, k_weight=PTR, eps=1e-6, positions=PTR, ldp=5, axes=3,
              turns=PTR, axis=PTR, pairs=32, neighbours=0, n_tokens=5, q_out=PTR, ldqo=256, hsqo=64,
              k_out=PTR, ldko=128, hsko=64, stream=None, flags=0)


@pytest.mark.parametrize("change,text,status", [
    (dict(dtype=V.VOC_LM_F32), "dtype", BAD), (dict(head_dim=8), "head_dim", NOT),
    (dict(head_dim=72), "head_dim", NOT), (dict(head_dim=272), "head_dim", NOT),
    (dict(pairs=40), "pairs", NOT), (dict(pairs=12), "pairs", NOT), (dict(pairs=-8), "pairs", NOT),
    (dict(heads=-1), "heads", BAD), (dict(heads=0, kv_heads=0), "heads", BAD),
    (dict(heads=65537), "heads", BAD), (dict(n_tokens=-1), "tokens", BAD),
    (dict(n_tokens=1 << 30), "tokens", BAD), (dict(axes=0), "axes", BAD), (dict(axes=17), "axes", BAD),
    (dict(ldp=4), "positions", BAD), (dict(neighbours=2), "neighbours", BAD), (dict(flags=1), "flags", BAD),
    (dict(eps=-1.0), "eps", BAD), (dict(eps=math.inf), "eps", BAD), (dict(q=None), "NULL", BAD),
    (dict(k_out=None), "NULL", BAD), (dict(positions=None), "NULL", BAD), (dict(turns=None), "NULL", BAD),
    (dict(q=PTR + 8), "16-byte", BAD), (dict(k_weight=PTR + 2), "16-byte", BAD),
    (dict(hsk=68), "multiples of 8", BAD), (dict(ldqo=260), "multiples of 8", BAD),
    (dict(positions=PTR + 2), "aligned", BAD), (dict(turns=PTR + 4), "aligned", BAD)])
def test_rotate_refusals(lib, change, text, status):
    _refused(lib, "vocoder_lm_rotate", {**ROTATE, **change}.values(), text, status)


ADAPTERS = dict(x8=PTR, ldx=64, x_scale=PTR, y=PTR, ldy=40, y_dtype=V.VOC_LM_BF16, a=PTR, lda=64,
                sa=1024, b=PTR, ldb=16, sb=640, dtype=V.VOC_LM_BF16, scale=PTR, ranks=PTR, rank=16, pool=4,
                ids=PTR, M=3, N=40, K=64, out=PTR + 4096, ldo=40, stream=None, flags=0)


@pytest.mark.parametrize("change,text,status", [
    (dict(dtype=V.VOC_LM_F32, y_dtype=V.VOC_LM_F32), "dtype", BAD), (dict(y_dtype=V.VOC_LM_F16), "y_dtype", BAD),
    (dict(y_dtype=7), "y_dtype", BAD), (dict(M=-1), "sizes", BAD), (dict(K=0), "sizes", BAD),
    (dict(N=1 << 29), "sizes", BAD), (dict(N=(1 << 24) + 1, ldy=1 << 25, ldo=1 << 25), "sizes", BAD),
    (dict(rank=0), "rank", NOT), (dict(rank=12), "rank", NOT),
    (dict(rank=136), "rank", NOT), (dict(pool=0), "pool", BAD), (dict(flags=4), "flags", BAD),
    (dict(ldx=48), "stride", BAD), (dict(ldy=39), "stride", BAD), (dict(ldo=39), "stride", BAD),
    (dict(lda=56), "stride", BAD), (dict(ldb=8), "stride", BAD), (dict(ldx=72), "multiple of 16", BAD),
    (dict(lda=68), "multiples of 8", BAD), (dict(sb=644), "multiples of 8", BAD),
    (dict(x8=None), "NULL", BAD), (dict(ids=None), "NULL", BAD), (dict(scale=None), "NULL", BAD),
    (dict(x8=PTR + 8), "16-byte", BAD), (dict(b=PTR + 2), "16-byte", BAD),
    (dict(ids=PTR + 1), "aligned", BAD), (dict(y_dtype=V.VOC_LM_F32, y=PTR + 2), "aligned", BAD),
    (dict(out=PTR, ldo=48), "y's place", BAD)])
def test_adapters_refusals(lib, change, text, status):
    _refused(lib, "vocoder_lm_adapters", {**ADAPTERS, **change}.values(), text, status)


LOGPROBS = dict(logits=PTR, ldl=100, dtype=V.VOC_LM_BF16, rows=3, vocab=100, temperature=1.0, tokens=PTR,
                logprob=PTR, entropy=PTR, top=5, top_logprobs=PTR, top_tokens=PTR, stream=None, flags=0)


@pytest.mark.parametrize("change,text,status", [
    (dict(dtype=3), "dtype", BAD), (dict(rows=-1), "sizes", BAD), (dict(vocab=0), "sizes", BAD),
    (dict(vocab=1 << 29, ldl=1 << 29), "sizes", BAD), (dict(temperature=0.0), "temperature", BAD),
    (dict(temperature=-1.0), "temperature", BAD), (dict(temperature=math.nan), "temperature", BAD),
    (dict(temperature=math.inf), "temperature", BAD), (dict(top=-1), "top", BAD),
    (dict(top=8, vocab=7), "top", BAD), (dict(top=33), "32 alternatives", NOT), (dict(flags=1), "flags", BAD),
    (dict(ldl=99), "stride", BAD), (dict(tokens=None), "go together", BAD),
    (dict(logprob=None), "go together", BAD), (dict(logits=None), "NULL", BAD),
    (dict(top_tokens=None), "NULL", BAD), (dict(logits=PTR + 1), "aligned", BAD),
    (dict(tokens=PTR + 4), "aligned", BAD), (dict(top_tokens=PTR + 4), "aligned", BAD)])
def test_logprobs_refusals(lib, change, text, status):
    _refused(lib, "vocoder_lm_logprobs", {**LOGPROBS, **change}.values(), text, status)


@pytest.mark.parametrize("name,call,work", [
    ("vocoder_lm_rotate", ROTATE, "n_tokens"), ("vocoder_lm_adapters", ADAPTERS, "M"),
    ("vocoder_lm_logprobs", LOGPROBS, "rows")])
def test_nothing_to_do_is_no_fault_of_the_arguments(lib, name, call, work):
    """A call without tokens gets as far as the device (there is none on a CPU)."""
    st = getattr(lib, name)(*{**call, work: 0}.values())
    assert st in (V.VOC_OK, V.VOC_CUDA_ERROR), V.vocoder_last_error()


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    f8 = torch.zeros(4, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    h = torch.zeros(4, 2, 64).bfloat16()
    pos, turns = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.int64)
    y, a, b = torch.zeros(4, 8), torch.zeros(2, 8, 64), torch.zeros(2, 8, 8)
    for bad in (lambda: V.rotate_heads(h, h, pos, turns),  # CPU tensors
                lambda: V.rotate_heads(h.double(), h, pos, turns),
                lambda: V.rotate_heads(h[0], h, pos, turns),
                lambda: V.adapters_fp8(y, f8, torch.ones(4), a, b, torch.ones(2), pos),
                lambda: V.adapters_fp8(y[0], f8, torch.ones(4), a, b, torch.ones(2), pos),
                lambda: V.logprobs(torch.zeros(4, 8)), lambda: V.logprobs(torch.zeros(8)),
                lambda: V.logprobs(torch.zeros(4, 8, dtype=torch.int32))):
        with pytest.raises(V.VocoderError) as e:
            bad()
        assert e.value.status == V.VOC_INVALID_ARG


def test_rotation_turns():
    """Turns reproduce position * rate modulo a turn where 32 bits would not."""
    torch = pytest.importorskip("torch")
    rates = torch.tensor([1.0, 0.1, 1e-4, 3.0, 4.0, -1.0, 0.0, 2 * math.pi * 1.25], dtype=torch.float64)
    turns = V.rotation_turns(rates)
    assert turns.dtype == torch.int64 and turns.shape == (8,)
    for pos in (0, 1, 77, 1_000_003, -5):
        for r, t in zip(rates.tolist(), turns.tolist()):
            got = ((pos * t) % 2 ** 64) / 2 ** 64
            off = (got - pos * r / (2 * math.pi)) % 1
            assert min(off, 1 - off) < 1e-9 * (1 + abs(pos)) ** 0.5
    half = V.rotation_turns([math.pi])  # half a turn either way
    assert half.item() in (-2 ** 63, 2 ** 63 - 1) or abs(abs(half.item()) - 2 ** 63) < 2 ** 12
