"""GPU: heads turned by position, low-rank adapters and log probabilities against 64-bit forms.

Tolerances, derived before any run:
  rotate    norm: a sum of d squares in d/16 lanes of 16 and 12 more roundings, of 2^-24 each: below 2^-19 of
            the value; cos and sin: 2^-20.5 (the hardware's approximation over [-pi, pi]) and an angle good to
            2 * 2^-22.  So 2^-18 of |a| + |b|, and half a step of the output's type.
  adapters  products are exact in 32 bits; accumulations of at most 2^-22 of the sum of magnitudes each: K / 16
            matrix steps, 16 joins, 2 * rank / 16 + 8 in the second product; the low-rank values between
            them: 2^-17 of themselves (bf16) or 2^-22 of the token's largest (f16); half a step of the output.
  logprobs  exponents: x - m, the factor and their product round by 2^-24 of |d| each; the exponential's
            approximation 2^-22; a thread adds up to 64 + vocab / 512 terms and 20 joins follow, 2^-24 each.
            Whole numbers (the tokens) are exact.
"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("no CUDA device", allow_module_level=True)

from dac_vocoder_decode_gb300 import binding as V  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SYNC = V.VOC_FLAG_SYNC


def _half_step(ref, dtype):
    """Half a step of `dtype` at ref (64 bits): of its binade, and of the subnormals below."""
    info = torch.finfo(dtype)
    return ref.abs() * (info.eps / 2) + info.smallest_normal * info.eps / 2


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


# ------------------------------------------------------------------ rotate
def _turned(x, weight, eps, positions, rates, axis, near):
    """(y, magnitude): the heads in 64 bits, and |a| + |b| of each channel's pair."""
    x = x.double()
    if weight is not None:
        rms = (x.square().mean(2, keepdim=True) + eps).sqrt()
        x = torch.where(rms == 0, 0, x / rms) * weight.double()
    pairs = len(rates)
    positions = positions.view(-1, x.shape[0])
    at = positions.double()[axis.long() if axis is not None else torch.zeros(pairs, dtype=torch.long)].T
    angle = (at * rates)[:, None]
    cos, sin = angle.cos(), angle.sin()
    ia = torch.arange(pairs) * 2 if near else torch.arange(pairs)
    ib = ia + 1 if near else ia + pairs
    y, mag = x.clone(), x.abs()
    a, b = x[:, :, ia], x[:, :, ib]
    y[:, :, ia], y[:, :, ib] = a * cos - b * sin, a * sin + b * cos
    mag[:, :, ia] = mag[:, :, ib] = a.abs() + b.abs()
    return y, mag


def _rates(pairs, base=1e4):
    return torch.exp(-math.log(base) * torch.arange(pairs, device="cuda").double() / max(1, pairs))


def _check_turned(got, x, weight, eps, positions, rates, axis, near):
    ref, mag = _turned(x, weight, eps, positions, rates, axis, near)
    tol = mag * 2.0 ** -18 + _half_step(ref, got.dtype) * (1 + 2.0 ** -7)
    assert got.shape == x.shape and got.dtype == x.dtype
    none = torch.isnan(ref)  # an infinity in the head, turned
    assert torch.equal(torch.isnan(got), none)
    near_enough = ((got.double() - ref).abs() <= tol) | none
    assert bool(near_enough.all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,heads,kv,d,pairs,axes,near", [
    (1, 1, 1, 16, 8, 1, False), (1, 3, 1, 64, 32, 1, False), (7, 16, 4, 64, 16, 2, True),
    (300, 5, 5, 128, 64, 3, False), (33, 28, 4, 128, 64, 3, True), (3, 2, 1, 48, 16, 1, False),
    (65, 7, 1, 96, 48, 1, True), (9, 4, 2, 256, 128, 4, False), (2, 6, 3, 80, 8, 1, False),
    (1000, 8, 8, 32, 0, 1, False), (5000, 9, 3, 64, 32, 1, False), (11, 2, 2, 240, 120, 2, True)])
@pytest.mark.parametrize("norm", [True, False])
def test_rotate(dtype, tokens, heads, kv, d, pairs, axes, near, norm):
    t, g = TYPES[dtype], _gen(tokens + d)
    qkv = (_randn(g, tokens, heads + 2 * kv, d) * 2).to(t)  # views with a stride of their own
    q, k, _ = qkv.split([heads, kv, kv], 1)
    qw, kw = ((1 + 0.3 * _randn(g, d)).to(t) if norm else None for _ in range(2))
    pos = torch.randint(-1000, 100000, (axes, tokens), generator=g, device="cuda", dtype=torch.int32)
    axis = torch.randint(0, axes, (pairs,), generator=g, device="cuda", dtype=torch.int32) if axes > 1 else None
    rates = _rates(pairs)
    args = dict(axis=axis, q_weight=qw, k_weight=kw, eps=1e-5, neighbours=near)
    before = qkv.clone()
    qo, ko = V.rotate_heads(q, k, pos, V.rotation_turns(rates), flags=SYNC, **args)
    assert torch.equal(qkv, before)
    _check_turned(qo, q, qw, 1e-5, pos, rates, axis, near)
    _check_turned(ko, k, kw, 1e-5, pos, rates, axis, near)
    # in place: the same bits, values beside them untouched
    V.rotate_heads(q, k, pos, V.rotation_turns(rates), q_out=q, k_out=k, flags=SYNC, **args)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, heads + kv:], before[:, heads + kv:])


@pytest.mark.parametrize("near", [False, True])
def test_rotate_far_positions(near):
    """Angles of the farthest positions, where a 32-bit product has no digit of the angle left."""
    g = _gen(1)
    pos = torch.tensor([0, 2 ** 31 - 1, -2 ** 31, 123456789, 2 ** 30 + 1], dtype=torch.int32, device="cuda")
    q = _randn(g, 5, 2, 64).half()
    rates = _rates(32)
    q_out, k_out = V.rotate_heads(q, None, pos, V.rotation_turns(rates), neighbours=near, flags=SYNC)
    assert k_out is None
    # 2^31 times a rate of 1 keeps 2^-22 of a radian in 64 bits
    _check_turned(q_out, q, None, 0, pos, rates, None, near)


def test_rotate_by_rates_beyond_half_a_turn():
    g = _gen(2)
    rates = torch.linspace(-7, 7, 8, device="cuda").double()
    pos = torch.arange(50, device="cuda", dtype=torch.int32)
    q = _randn(g, 50, 1, 16).half()
    out, _ = V.rotate_heads(q, None, pos, V.rotation_turns(rates), flags=SYNC)
    _check_turned(out, q, None, 0, pos, rates, None, False)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 80, 256])
def test_rotate_far_magnitudes(dtype, d):
    """Squares that overflow or vanish in 32 bits, and heads of zeros, beside ordinary heads."""
    t, g = TYPES[dtype], _gen(d)
    q = _randn(g, 6, 3, d)
    big, small = (1e30, 1e-30) if dtype == "bf16" else (3e4, 1e-7)
    q[0] *= big
    q[1, 1] *= small
    q[2, 0] = 0
    q[3] = 0
    q[4, 2] = float(torch.finfo(t).max)
    q = q.to(t)
    w = torch.ones(d, device="cuda").to(t)
    pos, rates = torch.arange(6, device="cuda", dtype=torch.int32), _rates(16)
    for eps in (1e-6, 0.0):
        out, _ = V.rotate_heads(q, None, pos, V.rotation_turns(rates), q_weight=w, eps=eps, flags=SYNC)
        _check_turned(out, q, w, eps, pos, rates, None, False)


def test_rotate_nonfinite_heads_stay_alone():
    g = _gen(3)
    q, k = _randn(g, 5, 6, 64).bfloat16(), _randn(g, 5, 2, 64).bfloat16()
    w = torch.ones(64, device="cuda").bfloat16()
    pos, turns = torch.arange(5, device="cuda", dtype=torch.int32), V.rotation_turns(_rates(32))
    clean = V.rotate_heads(q, k, pos, turns, q_weight=w, k_weight=w, flags=SYNC)
    q2 = q.clone()
    q2[1, 2, 5] = math.nan
    q2[3, 0, 63] = math.inf
    got = V.rotate_heads(q2, k, pos, turns, q_weight=w, k_weight=w, flags=SYNC)
    keep = torch.ones(5, 6, dtype=torch.bool)
    keep[1, 2] = keep[3, 0] = False
    assert torch.equal(got[0][keep], clean[0][keep]) and torch.equal(got[1], clean[1])
    assert torch.isnan(got[0][1, 2]).all()
    assert torch.isnan(got[0][3, 0][[31, 63]]).all()


def test_rotate_pairs_without_an_axis_stay():
    q = _randn(_gen(4), 3, 2, 32).half()
    axis = torch.tensor([0, 1, 2, -1, 0, 7, 1, 0], dtype=torch.int32, device="cuda")
    pos = torch.tensor([[5, 6, 7], [1, 2, 3]], dtype=torch.int32, device="cuda")
    rates = _rates(8)
    out, _ = V.rotate_heads(q, None, pos, V.rotation_turns(rates), axis=axis, flags=SYNC)
    still = (axis < 0) | (axis > 1)
    assert torch.equal(out[:, :, :8][:, :, still], q[:, :, :8][:, :, still])
    _check_turned(out, q, None, 0, pos, torch.where(still, 0, rates), axis.clamp(0, 1), False)


def test_rotate_one_norm_of_two_and_odd_buffers():
    """A weight for the queries alone, outputs given as strided views, positions as rows of a larger tensor."""
    g = _gen(5)
    q, k = _randn(g, 9, 4, 64).half(), _randn(g, 9, 2, 64).half()
    buf = torch.full((9, 8, 72), 7.0, device="cuda").half()
    pos = torch.arange(60, device="cuda", dtype=torch.int32).view(3, 20)[:, 5:14]
    axis = torch.arange(32, device="cuda", dtype=torch.int32) % 3
    w, rates = (1 + 0.1 * _randn(g, 64)).half(), _rates(32)
    qo, ko = V.rotate_heads(q, k, pos, V.rotation_turns(rates), axis=axis, q_weight=w, q_out=buf[:, 1:5, :64],
                            k_out=buf[:, 6:8, 8:], flags=SYNC)
    _check_turned(qo, q, w, 1e-6, pos, rates, axis, False)
    _check_turned(ko, k, None, 1e-6, pos, rates, axis, False)
    assert bool((buf[:, 0] == 7).all()) and bool((buf[:, 5] == 7).all()) and bool((buf[:, 1:5, 64:] == 7).all())


# ------------------------------------------------------------------ adapters
class Adapters:
    """Inputs of one call; x in e4m3 with row strides of 16, pools with strides of 8."""

    def __init__(self, M, N, K, rank, pool, dtype="bf16", y_dtype=None, ids=None, ranks=None, seed=0):
        g, t = _gen(seed + M + N), TYPES[dtype]
        self.M, self.N, self.K, self.rank, self.pool = M, N, K, rank, pool
        pad = -(-K // 16) * 16
        self.x8 = torch.full((M, pad), 0x7f, dtype=torch.uint8, device="cuda")  # NaN codes behind the rows
        v = _randn(g, M, K)
        self.x_scale = v.abs().amax(1) / 448
        self.x8[:, :K] = (v / self.x_scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        self.x = self.x8.view(torch.float8_e4m3fn)[:, :K]
        self.y = _randn(g, M, N).to(TYPES[y_dtype or dtype])
        wide = -(-K // 8) * 8
        self.a = (_randn(g, pool, rank, wide) / math.sqrt(K)).to(t)
        self.a[:, :, K:] = math.nan
        self.a = self.a[:, :, :K]
        self.b = (_randn(g, pool, N, rank) / math.sqrt(rank)).to(t)
        self.scale = 0.5 + torch.rand(pool, generator=g, device="cuda")
        self.ids = ids if ids is not None else torch.randint(-1, pool, (M,), generator=g, device="cuda")
        self.ids = self.ids.to(torch.int32)
        self.ranks = None
        if ranks is not None:
            self.ranks = torch.tensor([ranks[i % len(ranks)] for i in range(pool)], dtype=torch.int32,
                                      device="cuda")
            for i, r in enumerate(self.ranks.tolist()):  # what lies behind an adapter's rank is not used
                self.a[i, max(0, r):] = math.nan
                self.b[i, :, max(0, r):] = math.nan

    def run(self, **kw):
        kw.setdefault("flags", SYNC)
        return V.adapters_fp8(kw.pop("y", self.y), self.x, self.x_scale, self.a, self.b, self.scale, self.ids,
                              ranks=self.ranks, **kw)

    def check(self, got):
        ref, tol = self.y.double(), torch.zeros(self.M, self.N, dtype=torch.float64, device="cuda")
        bf16 = self.a.dtype == torch.bfloat16
        for i in set(self.ids.tolist()):
            r = 0 if not 0 <= i < self.pool else self.rank if self.ranks is None else int(self.ranks[i])
            if r <= 0:
                continue
            rows = torch.nonzero(self.ids == i)[:, 0]
            x = self.x[rows].double() * self.x_scale[rows].double()[:, None]
            a, b, s = self.a[i, :r].double(), self.b[i, :, :r].double(), float(self.scale[i])
            ref[rows] += s * (x @ a.T) @ b.T
            mag = x.abs() @ a.abs().T
            steps = (self.K / 16 + 16 + 2 * self.rank / 16 + 8) * 2.0 ** -22
            each = mag @ b.abs().T
            if bf16:
                tol[rows] += s * (steps + 2.0 ** -17) * each
            else:
                tol[rows] += s * (steps * each + 2.0 ** -22 * mag.amax(1)[:, None] * b.abs().sum(1))
        tol = tol + _half_step(ref, self.y.dtype) * (1 + 2.0 ** -7)
        assert got.shape == self.y.shape and got.dtype == self.y.dtype
        off = (got.double() - ref).abs()
        assert bool((off <= tol).all()), float((off / tol).max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,rank,pool", [
    (1, 1, 1, 8, 1), (1, 8, 16, 8, 1), (3, 33, 65, 16, 2), (8, 1536, 1024, 16, 8), (33, 1000, 4096, 16, 64),
    (64, 96, 200, 32, 3), (65, 200, 31, 24, 5), (130, 77, 1001, 64, 4), (100, 260, 520, 128, 7),
    (257, 512, 300, 40, 300), (1000, 130, 77, 8, 2), (20, 64, 9000, 48, 1)])
def test_adapters(dtype, M, N, K, rank, pool):
    c = Adapters(M, N, K, rank, pool, dtype)
    got = c.run()
    c.check(got)
    assert torch.equal(got, c.run())  # the same bits


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_adapters_beside_a_32_bit_projection(dtype):
    c = Adapters(70, 203, 500, 32, 3, dtype, "f32")
    c.check(c.run())


@pytest.mark.parametrize("rank,ranks", [(16, [1, 16, 0, 5]), (64, [64, 3, 33, 8, 0, -2]), (128, [100, 1, 128]),
                                        (32, [7, 31, 99]), (8, [3, 8])])
def test_adapters_of_ranks_of_their_own(rank, ranks):
    c = Adapters(150, 300, 257, rank, 6, "bf16", ranks=ranks)
    if max(ranks) > rank:
        c.ranks.clamp_(max=rank)
        d = Adapters(150, 300, 257, rank, 6, "bf16")
        c.a, c.b = d.a, d.b
        c.ranks[0] = 7
        want = c.run()
        c.ranks[2] = 99  # counts as the pool's rank
        assert torch.equal(c.run(), want)
        c.ranks.clamp_(max=rank)
        c.check(want)
        return
    c.check(c.run())


@pytest.mark.parametrize("M,how", [(64, "runs"), (500, "runs"), (500, "spread"), (200, "one"), (200, "none"),
                                   (129, "each")])
def test_adapters_orders_of_tokens(M, how):
    pool = 200 if how == "each" else 6
    i = torch.arange(M, device="cuda")
    ids = {"runs": i * 5 // M, "spread": i * 7 % 6 - 1, "one": i * 0 + 3, "none": i * 0 + 17 * (i % 2) - 1,
           "each": i}[how]
    c = Adapters(M, 72, 130, 16, pool, "f16", ids=ids)
    got = c.run()
    c.check(got)
    if how == "none":
        assert torch.equal(got, c.y)
    # in another order: the same up to the order of 32-bit sums, which goes by the number of tokens that share an
    # adapter in a tile; the same bits where they are alone
    order = torch.randperm(M, generator=_gen(1), device="cuda")
    c.x, c.x_scale, c.y, c.ids = (c.x8[order].view(torch.float8_e4m3fn)[:, :c.K], c.x_scale[order], c.y[order],
                                  c.ids[order])
    if how in ("each", "none"):
        assert torch.equal(c.run(), got[order])
    c.check(c.run())


@pytest.mark.parametrize("N", [64, 61])
def test_adapters_in_place_and_strided(N):
    c = Adapters(90, N, 128, 16, 4)
    want = c.run()
    y = c.y.clone()
    assert c.run(y=y, out=y) is y and torch.equal(y, want)
    wide = torch.full((90, N + 11), 5.0, device="cuda").bfloat16()
    wide[:, 3:3 + N] = c.y
    view = wide[:, 3:3 + N]
    c.run(y=view, out=view)
    assert torch.equal(view, want)
    assert bool((wide[:, :3] == 5).all()) and bool((wide[:, 3 + N:] == 5).all())
    out = torch.full((95, N), 9.0, device="cuda").bfloat16()
    c.run(out=out[:90])
    assert torch.equal(out[:90], want) and bool((out[90:] == 9).all())


def test_adapters_nonfinite_tokens_stay_alone():
    c = Adapters(40, 100, 96, 16, 2, "f16", ids=torch.arange(40, device="cuda") % 3 - 1)
    want = c.run()
    c.x8[4, 50] = 0x7f
    c.x_scale[9] = math.inf
    c.ids[4] = c.ids[9] = 1
    got = c.run()
    keep = [i for i in range(40) if i not in (4, 9)]
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[4]).all() and not torch.isfinite(got[9]).any()


def test_adapters_of_large_and_small_values():
    """Low-rank values beyond the range of 16 bits keep their bits."""
    c = Adapters(20, 64, 512, 16, 2, "f16", "f32")
    c.a.mul_(1000)  # about 448 * 1000 * sqrt(512) / sqrt(512)
    c.check(c.run())
    c.a.mul_(2.0 ** -20)
    c.x_scale.mul_(2.0 ** -60)
    c.y.zero_()
    got = c.run()
    assert float(got.abs().max()) > 0
    c.check(got)


# ------------------------------------------------------------------ log probabilities
def _exact_logprobs(x, tokens, top, temperature):
    """(logprob, entropy, top, top_tokens, spread): in 64 bits, on the CPU for the order of equal values."""
    z = x.double() / temperature
    m = z.amax(1, keepdim=True)
    low = torch.where(z == -math.inf, -math.inf, z - m)
    w = low.exp()
    s = w.sum(1, keepdim=True)
    lp = low - s.log()
    spread = torch.where(w > 0, w * low.abs(), 0).sum(1) / s[:, 0]
    entropy = s[:, 0].log() + spread
    order = torch.sort((x.float() + 0).cpu(), dim=1, descending=True, stable=True).indices[:, :top].cuda()
    return (lp.gather(1, tokens[:, None])[:, 0], entropy, lp.gather(1, order), order, spread)


def _check_logprobs(x, tokens, top, temperature, got):
    lp, ent, best, best_tokens, spread = _exact_logprobs(x, tokens, top, temperature)
    n = x.shape[1]
    sums = ((64 + n / 512 + 20) * 2.0 ** -24 + 2.0 ** -22 + 3 * 2.0 ** -24 * spread) * 1.5

    def near(a, ref, tol):
        assert a.dtype == torch.float32 and a.shape == ref.shape
        closed = ref == -math.inf
        assert torch.equal(a == -math.inf, closed)
        a, ref = a.double().masked_fill(closed, 0), ref.masked_fill(closed, 0)
        tol = tol + (ref.abs() + ent.view(-1, *[1] * (ref.dim() - 1)) + 1) * 2.0 ** -22
        off = (a - ref).abs()
        assert bool((off <= tol).all()), float((off / tol).max())

    near(got[0], lp, sums)
    near(got[1], ent, sums * (2 + spread))
    if top:
        assert got[3].dtype == torch.int64 and torch.equal(got[3], best_tokens)
        near(got[2], best, sums[:, None])
    else:
        assert got[2] is None and got[3] is None


def _logits(g, rows, vocab, dtype, masked=False):
    x = _randn(g, rows, vocab) * 4
    if masked:
        x.masked_fill_(torch.rand(rows, vocab, generator=g, device="cuda") < 0.3, -math.inf)
        x[:, vocab // 2] = 0.5
    return x.to(TYPES[dtype]), torch.randint(0, vocab, (rows,), generator=g, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab,top,temperature,masked", [
    (1, 1, 1, 1.0, False), (3, 5, 5, 0.5, False), (5, 31, 20, 1.0, True), (130, 64, 0, 1.0, True),
    (7, 1000, 32, 0.7, False), (300, 2048, 5, 1.3, True), (6, 4096, 20, 1.0, False), (9, 4097, 20, 1.0, True),
    (2, 10007, 32, 2.0, False), (400, 5000, 1, 1.0, False), (1, 131072, 20, 1.0, True),
    (8, 70001, 20, 0.1, True), (200, 33333, 7, 1.0, False)])
def test_logprobs(dtype, rows, vocab, top, temperature, masked):
    x, tokens = _logits(_gen(rows + vocab), rows, vocab, dtype, masked)
    got = V.logprobs(x, tokens, top=top, temperature=temperature, flags=SYNC)
    _check_logprobs(x, tokens, top, temperature, got)
    again = V.logprobs(x, tokens, top=top, temperature=temperature, flags=SYNC)
    for a, b in zip(got, again):
        assert a is None and b is None or torch.equal(a, b)


@pytest.mark.parametrize("vocab", [40, 2048, 4096, 8192, 50001])
@pytest.mark.parametrize("kind", ["constant", "rising", "falling", "steps", "block", "zeros"])
def test_logprobs_equal_values_and_orders(vocab, kind):
    """Ties go to the lowest index; orders that bring more candidates together than there is room for."""
    i = torch.arange(vocab, device="cuda").float()
    x = {"constant": 0 * i + 1.5, "rising": i / vocab * 8, "falling": -i / vocab * 8, "steps": (i % 7).floor(),
         "block": torch.where((i - vocab // 2).abs() < vocab // 8, 5 + i / vocab, -i / vocab),
         "zeros": torch.where(i % 2 == 1, 0.0, -0.0)}[kind]
    for dtype in ("f32", "f16"):
        rows = torch.stack([x, x.flip(0), x]).to(TYPES[dtype])
        tokens = torch.tensor([0, vocab - 1, vocab // 2], device="cuda")
        _check_logprobs(rows, tokens, 32, 1.0, V.logprobs(rows, tokens, top=32, flags=SYNC))


@pytest.mark.parametrize("vocab", [100, 4096, 20000])
def test_logprobs_worst_orders(vocab):
    """The largest values all in the places that one lane reads: the bound from the subsets is at its worst."""
    g = _gen(vocab)
    for stride in (8, 8 * 32, 8 * 256):
        x = _randn(g, 2, vocab)
        i = torch.arange(vocab, device="cuda")
        x[0, i % stride < 8] += 50
        x[1] = torch.where(i % stride < 8, 50 + i / vocab, x[1])
        x = x.float()
        tokens = torch.tensor([0, vocab - 1], device="cuda")
        _check_logprobs(x, tokens, 32, 1.0, V.logprobs(x, tokens, top=32, flags=SYNC))


@pytest.mark.parametrize("vocab", [50, 3000, 9001])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_logprobs_ends_of_the_range(vocab, dtype):
    """Rows of the type's lowest value (equal weights), of its largest, of both, and of far apart values."""
    t = TYPES[dtype]
    lo, hi = torch.finfo(t).min, torch.finfo(t).max
    x = torch.zeros(5, vocab, device="cuda").to(t)
    x[0], x[1], x[2] = lo, hi, lo
    x[2, vocab // 3], x[3, ::2] = hi, lo
    x[4] = (torch.arange(vocab, device="cuda") - vocab / 2) * (hi / vocab / 2)
    tokens = torch.tensor([vocab - 1, 0, vocab // 3, 1, vocab - 1], device="cuda")
    got = V.logprobs(x, tokens, top=9, flags=SYNC)
    want = _exact_logprobs(x, tokens, 9, 1.0)
    assert torch.equal(got[3], want[3])
    for a, b in zip(got[:2], want[:2]):
        assert torch.allclose(a.double(), b, rtol=2e-6, atol=2e-6)
    # differences beyond 32 bits are -infinity there
    far = want[2] < -3e38
    assert torch.allclose(got[2].double().masked_fill(far, 0), want[2].masked_fill(far, 0), rtol=2e-6, atol=2e-6)


@pytest.mark.parametrize("vocab", [60, 2000, 12000])
def test_logprobs_closed_and_nonfinite_rows(vocab):
    x = _randn(_gen(vocab), 6, vocab)
    clean = V.logprobs(x, torch.zeros(6, dtype=torch.int64, device="cuda"), top=4, flags=SYNC)
    x[1] = -math.inf
    x[2, vocab // 2] = math.nan
    x[4, 3] = math.inf
    x[5, 1:] = -math.inf
    tokens = torch.tensor([0, 0, 0, 0, 0, 1], device="cuda")
    lp, ent, top, top_tokens = V.logprobs(x, tokens, top=4, flags=SYNC)
    for i in (0, 3):
        assert all(torch.equal(a[i], b[i]) for a, b in zip((lp, ent, top, top_tokens), clean))
    assert lp[1] == -math.inf and ent[1] == 0 and (top[1] == -math.inf).all()
    assert top_tokens[1].tolist() == [0, 1, 2, 3]
    for i in (2, 4):
        assert torch.isnan(lp[i]) and torch.isnan(ent[i]) and torch.isnan(top[i]).all()
        assert ((top_tokens[i] >= 0) & (top_tokens[i] < vocab)).all()
    assert lp[5] == -math.inf and ent[5] == 0 and top[5].tolist() == [0.0] + [-math.inf] * 3
    assert top_tokens[5].tolist() == [0, 1, 2, 3]
    every = torch.full((1, vocab), math.nan, device="cuda")
    got = V.logprobs(every, torch.zeros(1, dtype=torch.int64, device="cuda"), top=4, flags=SYNC)
    assert torch.isnan(got[0]) and sorted(got[3][0].tolist()) == sorted(set(got[3][0].tolist()))
    assert ((got[3] >= 0) & (got[3] < vocab)).all()


def test_logprobs_tokens_outside_and_parts_not_wanted():
    x = _randn(_gen(6), 4, 500).half()
    tokens = torch.tensor([-1, 500, 2 ** 40, 3], device="cuda")
    lp, ent, top, top_tokens = V.logprobs(x, tokens, entropy=False, flags=SYNC)
    assert ent is None and top is None and top_tokens is None
    assert (lp[:3] == -math.inf).all() and bool(torch.isfinite(lp[3]))
    lp, ent, top, _ = V.logprobs(x, top=3, flags=SYNC)
    assert lp is None and ent.shape == (4,) and top.shape == (4, 3)
    assert V.logprobs(x, entropy=False) == (None, None, None, None)
    empty = V.logprobs(x[:0], tokens[:0], top=2, flags=SYNC)
    assert [tuple(t.shape) for t in empty] == [(0,), (0,), (0, 2), (0, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("vocab,extra,start", [(257, 0, 1), (2049, 3, 2), (9000, 1, 5), (50001, 0, 7)])
def test_logprobs_rows_of_any_alignment(dtype, vocab, extra, start):
    """Rows that start and end anywhere; what lies between them is not read as a logit."""
    g = _gen(vocab)
    flat = torch.full((start + 5 * (vocab + extra) + 8,), 1e4, device="cuda").to(TYPES[dtype])
    x = flat[start:start + 5 * (vocab + extra)].view(5, vocab + extra)[:, :vocab]
    x.copy_((_randn(g, 5, vocab) * 3).to(TYPES[dtype]))
    tokens = torch.randint(0, vocab, (5,), generator=g, device="cuda")
    _check_logprobs(x, tokens, 20, 1.0, V.logprobs(x, tokens, top=20, flags=SYNC))
