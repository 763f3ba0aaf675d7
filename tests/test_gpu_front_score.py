"""GPU: codes that Front.score takes, what it refuses, and what a refused call leaves; voices that are assigned."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("no CUDA device", allow_module_level=True)

from dac_vocoder_decode_gb300 import binding as V  # noqa: E402
from dac_vocoder_decode_gb300.front import Front  # noqa: E402
from tests.test_gpu_front_token import TOKEN, _codes, _voices  # noqa: E402


def _same(a, b):
    return all(x is None and y is None or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("how", ["transposed", "int32", "strided", "host"])
def test_score_takes_the_codes_that_a_prompt_takes(how):
    """The same codes as [B, books, T] seen the other way round, in 32 bits, as a part of a larger tensor, on the host."""
    codes = _codes(2, 30, seed=7)
    wide = torch.zeros(2, 40, 6, dtype=torch.int64, device="cuda")
    wide[:, 3:33, 1:5] = codes
    given = {"transposed": codes.transpose(1, 2).contiguous().transpose(1, 2), "int32": codes.int(),
             "strided": wide[:, 3:33, 1:5], "host": codes.cpu()}[how]
    front = Front(TOKEN, 2, 30)
    _voices(front, 0, -1)
    want = [t.clone() for t in front.score(codes, top=4)]
    front.reset()
    latent = front.prompt(codes)
    front.reset()
    assert torch.equal(front.prompt(given), latent)
    front.reset()
    assert _same(front.score(given, top=4), want)


@pytest.mark.parametrize("change", [dict(top=33), dict(top=65), dict(top=-1), dict(temperature=0.0),
                                    dict(temperature=float("nan")), dict(books=3), dict(sequences=1),
                                    dict(frames=99), dict(floats=True)])
def test_a_refused_score_takes_no_frames(change):
    """The sequence goes on where it was: the score after the refusal is that of a stack that never saw it."""
    codes = _codes(2, 70, seed=8)
    front, other = Front(TOKEN, 2, 70), Front(TOKEN, 2, 70)
    for f in (front, other):
        _voices(f, -1, 2)
        f.prompt(codes[:, :20])
    bad = _codes(2, change.pop("frames", 50), seed=9)
    bad = bad[:change.pop("sequences", 2), :, :change.pop("books", 4)]
    if change.pop("floats", False):
        bad = bad.float()
    with pytest.raises(V.VocoderError) as e:
        front.score(bad, **change)
    assert e.value.status in (V.VOC_INVALID_ARG, V.VOC_UNSUPPORTED)
    assert front.frames == 20 and front.lens.tolist() == [20, 20]
    assert _same(front.score(codes[:, 20:], top=3), other.score(codes[:, 20:], top=3))


@pytest.mark.parametrize("how", ["list", "int32", "int64", "host"])
def test_assigned_voices_reach_captured_steps(how):
    """The graph of a step reads the voices that were assigned behind its capture."""
    codes = _codes(2, 6, seed=10)
    front, other = Front(TOKEN, 2, 6), Front(TOKEN, 2, 6)
    _voices(other, 2, -1)
    want = [other.step(codes[:, i]).clone() for i in range(6)]
    front.step(codes[:, 0])
    front.reset()
    given = torch.tensor([2, -1], dtype=torch.int32 if how == "int32" else torch.int64,
                         device="cpu" if how == "host" else "cuda")
    front.voice = given.tolist() if how == "list" else given
    assert front.voice.tolist() == [2, -1] and front.voice.dtype == torch.int32
    assert _same([front.step(codes[:, i]).clone() for i in range(6)], want)
    for bad in ([0], [[0, 1]], [0.5, 1.0], 1):
        with pytest.raises(V.VocoderError):
            front.voice = bad
    assert front.voice.tolist() == [2, -1]
