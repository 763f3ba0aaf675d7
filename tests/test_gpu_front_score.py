"""GPU: codes that Front.score takes, what it refuses, and what a refused call leaves; voices that are assigned."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("no CUDA device", allow_module_level=True)

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
