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


# Tokens for clusters of 8, 4, 2 and 1 CTAs: they halve while the tiles of 64 tokens times the CTAs of a cluster are
# more than two to an SM.  The last tile is ragged.
CLUSTERS = {split: 64 * max(1, 2 * SMS // (2 * split) + 1) - 27 for split in (4, 2, 1)} | {8: 64 * 5 - 27}


@pytest.mark.parametrize("split", [8, 4, 2, 1])
@pytest.mark.parametrize("dtype,y_dtype", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("rank", [16, 32, 64, 128])
def test_adapters_of_every_cluster_and_rank(rank, dtype, y_dtype, split):
    """Runs of tokens of one adapter and mixed tiles; every CTA has several stages of K; the same bits again."""
    M = CLUSTERS[split]
    i = torch.arange(M, device="cuda")
    ids = torch.where(i < M // 2, i // 500 % 4 - 1, i * 7 % 5 - 1)
    c = T.Adapters(M, 100, 500 + 800 * split, rank, 4, dtype, y_dtype, ids=ids)
    got = c.run()
    c.check(got)
    for _ in range(3):
        assert torch.equal(got, c.run())


@pytest.mark.parametrize("split", [8, 4, 2, 1])
@pytest.mark.parametrize("rank,dtype,y_dtype", [(16, "bf16", "bf16"), (32, "f16", "f32"), (64, "f16", "f16"),
                                                (128, "bf16", "f32")])
def test_adapters_of_tiles_with_many_adapters(rank, dtype, y_dtype, split):
    """64 adapters in each tile, several of them for each cluster (there are 512 / tiles for a tile): the sums that the
    CTAs read of one another and the ring are used again."""
    M = max(CLUSTERS[split], 64 * 12)
    assert 512 // (M // 64) < 64
    ids = torch.arange(M, device="cuda") * 13 % 66 - 1  # two of 66 without one
    c = T.Adapters(M, 90, 900, rank, 64, dtype, y_dtype, ids=ids, ranks=[rank, rank // 2 + 1, 0, rank - 3])
    got = c.run()
    c.check(got)
    for _ in range(10):
        assert torch.equal(got, c.run())


# ------------------------------------------------------------------ log probabilities
MANY = 4 * SMS + 3  # rows of up to 4096 values that a warp each takes; the last CTA has three


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("vocab,top,temperature,masked", [
    (1, 0, 1.0, False), (1, 1, 1.0, False), (2, 1, 0.7, False), (5, 5, 0.5, False), (31, 20, 1.0, True),
    (64, 0, 1.0, True), (64, 32, 2.0, False), (257, 32, 1.0, True), (1000, 1, 0.7, False), (2048, 0, 1.0, False),
    (2048, 20, 0.9, True), (2049, 32, 1.3, False), (4095, 5, 1.0, True), (4096, 0, 1.0, True), (4096, 32, 1.0, False)])
def test_logprobs_of_many_rows(dtype, vocab, top, temperature, masked):
    """A lane adds vocab / 32 values in two sums, 64 at most, as in the tolerances of wider rows."""
    x, tokens = T._logits(T._gen(vocab + top), MANY, vocab, dtype, masked)
    got = V.logprobs(x, tokens, top=top, temperature=temperature, flags=SYNC)
    T._check_logprobs(x, tokens, top, temperature, got)
    again = V.logprobs(x, tokens, top=top, temperature=temperature, flags=SYNC)
    for a, b in zip(got, again):
        assert a is None and b is None or torch.equal(a, b)


@pytest.mark.parametrize("vocab", [40, 300, 2048, 4096])
@pytest.mark.parametrize("kind", ["constant", "rising", "falling", "steps", "block", "zeros"])
def test_logprobs_of_many_rows_equal_values_and_orders(vocab, kind):
    i = torch.arange(vocab, device="cuda").float()
    x = {"constant": 0 * i + 1.5, "rising": i / vocab * 8, "falling": -i / vocab * 8, "steps": (i % 7).floor(),
         "block": torch.where((i - vocab // 2).abs() < vocab // 8, 5 + i / vocab, -i / vocab),
         "zeros": torch.where(i % 2 == 1, 0.0, -0.0)}[kind]
    for dtype in ("f32", "f16", "bf16"):
        rows = torch.stack([x, x.flip(0), x.roll(vocab // 3)]).to(T.TYPES[dtype]).repeat(MANY // 3 + 1, 1)
        tokens = torch.arange(len(rows), device="cuda") * 31 % vocab
        got = V.logprobs(rows, tokens, top=32, flags=SYNC)
        want = T._exact_logprobs(rows[:3], tokens[:3], 32, 1.0)[3]
        assert torch.equal(got[3], want.repeat(MANY // 3 + 1, 1))
        T._check_logprobs(rows, tokens, 32, 1.0, got)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [300, 2048, 4096])
def test_logprobs_of_many_rows_worst_orders(vocab, dtype):
    """The largest values all in the places that one lane reads, and more candidates than there is room for."""
    each = 4 if dtype == "f32" else 8
    g, i = T._gen(vocab), torch.arange(vocab, device="cuda")
    for stride in (each, 2 * each, 32 * each):
        x = T._randn(g, MANY, vocab)
        x[::2, i % stride < each] += 50
        x[1::2] = torch.where(i % stride < each, 50 + i / vocab, x[1::2])
        x = x.to(T.TYPES[dtype])
        tokens = i[torch.arange(MANY, device="cuda") * 17 % vocab]
        T._check_logprobs(x, tokens, 32, 1.0, V.logprobs(x, tokens, top=32, flags=SYNC))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("vocab,extra,start", [(1, 2, 1), (9, 0, 3), (257, 0, 1), (2049, 3, 2), (4090, 1, 5)])
def test_logprobs_of_many_rows_of_any_alignment(dtype, vocab, extra, start):
    g = T._gen(vocab)
    flat = torch.full((start + MANY * (vocab + extra) + 8,), 1e4, device="cuda").to(T.TYPES[dtype])
    x = flat[start:start + MANY * (vocab + extra)].view(MANY, vocab + extra)[:, :vocab]
    x.copy_((T._randn(g, MANY, vocab) * 3).to(T.TYPES[dtype]))
    tokens = torch.randint(0, vocab, (MANY,), generator=g, device="cuda")
    top = min(20, vocab)
    T._check_logprobs(x, tokens, top, 1.0, V.logprobs(x, tokens, top=top, flags=SYNC))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("vocab", [60, 2000, 4096])
def test_logprobs_of_many_rows_closed_and_nonfinite(vocab, dtype):
    """Rows of nothing, with NaN and with infinities beside ordinary ones in the same CTA, which keep their bits."""
    x = T._randn(T._gen(vocab), MANY, vocab).to(T.TYPES[dtype])
    tokens = torch.arange(MANY, device="cuda") % vocab
    clean = V.logprobs(x, tokens, top=4, flags=SYNC)
    i = torch.arange(MANY, device="cuda")
    closed, nan, inf, one = (i % 8 == k for k in (1, 2, 4, 7))
    every = i == MANY - 1
    x[closed], x[nan, vocab // 2], x[inf, 3] = -math.inf, math.nan, math.inf
    x[one, 1:] = -math.inf
    x[every] = math.nan
    lp, ent, top, top_tokens = V.logprobs(x, tokens, top=4, flags=SYNC)
    same = ~(closed | nan | inf | one | every)
    assert bool(same[::4].any()) and all(torch.equal(a[same], b[same]) for a, b in zip((lp, ent, top, top_tokens), clean))
    closed, one = closed & ~every, one & ~every
    assert bool((lp[closed] == -math.inf).all() & (ent[closed] == 0).all() & (top[closed] == -math.inf).all())
    first = torch.arange(4, device="cuda").expand(MANY, 4)
    assert torch.equal(top_tokens[closed | one], first[closed | one])
    for k in (nan, inf, every):
        assert bool(torch.isnan(lp[k]).all() & torch.isnan(ent[k]).all() & torch.isnan(top[k]).all())
    assert bool(((top_tokens >= 0) & (top_tokens < vocab)).all())
    assert bool((ent[one] == 0).all() & (top[one][:, 0] == 0).all() & (top[one][:, 1:] == -math.inf).all())
    assert torch.equal(lp[one] == 0, tokens[one] == 0)


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
