"""GPU: low-rank adapters and log probabilities at the launch shapes and ends of ranges that small calls do not
reach, against 64-bit forms.  Tolerances as in test_gpu_lm_token.py unless a test derives its own."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("no CUDA device", allow_module_level=True)

from dac_vocoder_decode_gb300 import binding as V  # noqa: E402
from tests import test_gpu_lm_token as T  # noqa: E402

SYNC = V.VOC_FLAG_SYNC
SMS = torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------------ low-rank adapters
@pytest.mark.parametrize("dtype,y_dtype", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("M,N,K,rank", [(6, 70, 64, 8), (40, 33, 96, 16), (150, 64, 300, 32), (70, 40, 64, 128)])
def test_adapters_infinite_low_rank_values_stay_infinite(M, N, K, rank, dtype, y_dtype):
    """An infinity in A: the formula's infinities, their signs and its NaN (0 times an infinity, two of unlike sign);
    finite low-rank values beside them, beyond 16 bits too, take nothing away.  Tokens of others are ordinary."""
    c = T.Adapters(M, N, K, rank, 3, dtype, y_dtype, ids=torch.arange(M, device="cuda") % 4 - 1)
    c.a[1] *= 1000
    c.a[1, 2, 5] = math.inf
    c.a[2, 0, 1], c.a[2, 3, 9] = math.inf, -math.inf
    c.x8[3::8, 5] = 0
    got = c.run()
    ref = c.y.double()
    for i in range(3):
        rows = torch.nonzero(c.ids == i)[:, 0]
        x = c.x[rows].double() * c.x_scale[rows].double()[:, None]
        ref[rows] += float(c.scale[i]) * (x @ c.a[i].double().T) @ c.b[i].double().T
    far = (c.ids == 1) | (c.ids == 2)
    assert bool(torch.isinf(ref[far]).any()) and bool(torch.isnan(ref[far]).any())
    assert not bool(torch.isfinite(ref[far]).any())
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(got[far].double().nan_to_num(0, 1, -1), ref[far].nan_to_num(0, 1, -1))
    c.a[1:] = 0
    again = c.run()
    assert torch.equal(again[~far], got[~far])
    c.check(again)


@pytest.mark.parametrize("rank,M", [(8, 3), (32, 70), (64, 1), (128, 20)])
def test_adapters_32_bit_outputs_of_bf16_keep_the_low_rank_bits(rank, M):
    """A low-rank value of 21 bits, exact in every sum: what is lost is what the parts between the products drop.  Two
    parts of 8 bits would drop the last, 2^-20; an accumulation may drop 2^-22 of the value."""
    c = T.Adapters(M, 40, 48, rank, 1, "bf16", "f32", ids=torch.zeros(M, device="cuda"))
    c.x8[:] = torch.ones(1, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    c.x_scale.fill_(1)
    c.y.zero_()
    c.a.zero_()
    c.b.zero_()
    c.scale.fill_(1)
    c.a[0, 5, 0], c.a[0, 5, 1], c.a[0, 5, 2] = 1, 2.0 ** -10, 2.0 ** -20
    c.b[0, :, 5] = 1
    got = c.run().double()
    assert float((got - (1 + 2.0 ** -10 + 2.0 ** -20)).abs().max()) <= 2.0 ** -22


# ------------------------------------------------------------------ log probabilities
@pytest.mark.parametrize("temperature", [0.7, 1.0, 1.3, 4.0])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(5, 50), (5, 3000), (4 * SMS + 3, 2048), (3, 9001), (3, 70001)])
def test_logprobs_of_the_lowest_value_beside_ordinary_ones(rows, vocab, dtype, temperature):
    """A mask of the type's lowest value: its tokens' log probabilities as far as 32 bits hold them, -infinity beyond.

    1 / temperature, the difference and their product round by 2^-24 each, the sum by one more: below 2^-21 of
    the result, beside the sums' error of an ordinary row, far below 1e-4."""
    t, g = T.TYPES[dtype], T._gen(vocab)
    x = T._randn(g, rows, vocab) * 3
    x = x.to(t)
    x[:, 20:] = torch.finfo(t).min
    x[1, 7] = torch.finfo(t).max  # a difference of twice the range
    tokens = torch.randint(0, 40, (rows,), generator=g, device="cuda")
    tokens[0], tokens[1], tokens[2] = vocab - 1, 30, 3
    lp, ent, top, top_tokens = V.logprobs(x, tokens, top=32, temperature=temperature, flags=SYNC)
    want = T._exact_logprobs(x, tokens, 32, temperature)
    assert torch.equal(top_tokens, want[3])
    for got, ref in ((lp, want[0]), (ent, want[1]), (top, want[2])):
        gone = ref.float() == -math.inf
        assert torch.equal(got == -math.inf, gone)
        off = (got.double() - ref).masked_fill(gone, 0).abs()
        assert bool((off <= ref.abs().masked_fill(gone, 0) * 2.0 ** -21 + 1e-4).all())
    if dtype != "f16" and temperature == 1:
        assert bool((lp[0] < -3e38) & (lp[0] > -math.inf)) and lp[1] == -math.inf
