"""Measured cases of three operators that a token model runs beside the 8-bit ones.

  rotate     queries and keys between the product that makes them and the cache: RMS norm of each head
             and rotation by position in one pass, pairs of channels turning with one of several
             position axes
  adapters   low-rank adapters of many requests at once beside a shared projection: every token adds
             the product with its own request's two thin matrices to the projection's output
  logprobs   log probabilities of given tokens, the entropy and the top alternatives of rows of logits

`run` takes the plain form (elementary torch operations in 32 bits) or, with `own`, the calls that
a user makes.  `exact` restates each operator in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one frame of 8 streamed speech sequences: the smallest call
        dict(name="rotate frame 8", op="rotate", tokens=8, heads=16, kv_heads=4, d=64, turned=64,
             axes=1, near=False, norm=True, far=250, dtype="bf16"),
        # the whole prompt of a 180 s song
        dict(name="rotate song 15504", op="rotate", tokens=15504, heads=16, kv_heads=4, d=128,
             turned=128, axes=1, near=False, norm=True, far=15504, dtype="bf16"),
        # an odd number of tokens at places of three axes, far along the first
        dict(name="rotate three axes 4001", op="rotate", tokens=4001, heads=28, kv_heads=4, d=128,
             turned=128, axes=3, near=False, norm=True, far=2000000, dtype="f16"),
        # one window's frames, half of each head turned, neighbouring channels, no norm
        dict(name="rotate half 689", op="rotate", tokens=689, heads=16, kv_heads=16, d=64, turned=32,
             axes=1, near=True, norm=False, far=689, dtype="f16"),
        # one frame of 8 sequences, each with a voice of its own: latency
        dict(name="adapters frame 8x1024x1536", op="adapters", seqs="1," * 7 + "1", k=1024, n=1536,
             rank=16, pool=8, mixed=False, dtype="bf16"),
        # an odd batch of single tokens beside a wide layer: the adapters' bytes count
        dict(name="adapters step 33x4096x12288", op="adapters", seqs="1," * 32 + "1", k=4096, n=12288,
             rank=16, pool=64, mixed=False, dtype="bf16"),
        # prompts of several lengths, adapters of ranks of their own, at a ragged width
        dict(name="adapters prompts 1001x1540", op="adapters", seqs="8192,4001,1,2400,129,700",
             k=1001, n=1540, rank=32, pool=16, mixed=True, dtype="f16"),
        # a song's prompt beside a square layer
        dict(name="adapters song 15504x4096x4096", op="adapters", seqs="15504", k=4096, n=4096,
             rank=64, pool=4, mixed=False, dtype="bf16"),
        # one frame of 8 sequences, 16 codebooks of 2048 entries each, candidates for sampling
        dict(name="logprobs frame 128x2048", op="logprobs", rows=128, vocab=2048, top=20,
             temperature=0.9, masked=False, dtype="bf16"),
        # the codes of a song scored, one codebook
        dict(name="logprobs song 15504x2048", op="logprobs", rows=15504, vocab=2048, top=0,
             temperature=1.0, masked=False, dtype="bf16"),
        # single tokens over a large vocabulary, part of it forbidden
        dict(name="logprobs step 8x131072", op="logprobs", rows=8, vocab=131072, top=20,
             temperature=0.7, masked=True, dtype="f32"),
        # an odd number of rows of an odd width
        dict(name="logprobs text 4001x50001", op="logprobs", rows=4001, vocab=50001, top=5,
             temperature=1.0, masked=True, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rotate", "adapters", "logprobs"])
    if op == "rotate":
        kv = rng.choice([1, 2, 4, 8, 16])
        heads = kv * rng.choice([1, 2, 4, 7])
        d = rng.choice([64, 64, 96, 128, 128, 256])
        turned = rng.choice([d, d, d // 2])
        tokens = max(1, min(_log(rng, 1, 16384), 39_000_000 // ((heads + kv) * d)))
        return dict(op=op, tokens=tokens, heads=heads, kv_heads=kv, d=d, turned=turned,
                    axes=rng.choice([1, 1, 2, 3]), near=rng.random() < 0.4, norm=rng.random() < 0.7,
                    far=_log(rng, 100, 1_000_000), dtype=rng.choice(["bf16", "f16"]))
    if op == "adapters":
        k, n = _log(rng, 64, 8192), _log(rng, 64, 12288)
        rank = rng.choice([8, 16, 16, 32, 64, 128])
        m = max(1, min(_log(rng, 1, 16384), 120_000_000 // (k + 2 * n), 8_000_000_000 // ((k + n) * rank)))
        if m <= 256 and rng.random() < 0.7:
            seqs = [1] * m
        else:
            seqs = []
            while sum(seqs) < m and len(seqs) < 200:
                seqs.append(_log(rng, 1, m - sum(seqs)))
        return dict(op=op, seqs=",".join(map(str, seqs)), k=k, n=n,
                    rank=rank, pool=_log(rng, 1, 64), mixed=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "f16"]))
    vocab = _log(rng, 64, 200000)
    dtype = rng.choice(["bf16", "f16", "f32"])
    rows = max(1, min(_log(rng, 1, 16384), (100 if dtype == "f32" else 200) * 1_000_000 // vocab))
    return dict(op=op, rows=rows, vocab=vocab, top=rng.choice([0, 1, 5, 20]),
                temperature=rng.choice([1.0, 0.7, 1.3]), masked=rng.random() < 0.4, dtype=dtype)


def _ints(text):
    return [int(v) for v in text.split(",")]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return globals()["_prepare_" + case["op"]](case, g)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _prepare_rotate(c, g):
    t = TYPES[c["dtype"]]
    tokens, d, pairs = c["tokens"], c["d"], c["turned"] // 2
    # q | k | v side by side, as one product makes them
    qkv = (_normal(g, tokens, c["heads"] + 2 * c["kv_heads"], d) * 1.3).to(t)
    q, k, _ = qkv.split([c["heads"], c["kv_heads"], c["kv_heads"]], 1)
    s = dict(case=c, q=q, k=k, q_weight=None, k_weight=None)
    if c["norm"]:
        s["q_weight"] = (1 + 0.2 * _normal(g, d)).to(t)
        s["k_weight"] = (1 + 0.2 * _normal(g, d)).to(t)
    # radians for each position: 1 down to about 1e-4
    rates = torch.exp(-math.log(1e4) / pairs * torch.arange(pairs, device="cuda").double())
    s["rates"] = rates
    # the same as a program keeps them: 2^-64 of a turn (less than half a turn each)
    s["turns"] = (rates / (2 * math.pi) * 2.0 ** 64).to(torch.int64)
    s["axis"] = None
    if c["axes"] > 1:
        s["axis"] = (torch.arange(pairs, device="cuda") * c["axes"] // pairs).to(torch.int32)
    first = torch.randint(0, c["far"], (c["axes"], 1), generator=g, device="cuda")
    step = torch.arange(tokens, device="cuda")
    place = [first[0] + step] + [first[a] % 97 + step // 7 ** a % 50 for a in range(1, c["axes"])]
    s["positions"] = torch.stack(place).to(torch.int32)
    return s


def _codes(g, rows, k):
    """Random e4m3 rows as a quantiser leaves them (largest value at 448), rows padded to 16."""
    pad = -(-k // 16) * 16
    v = _normal(g, rows, k)
    scale = v.abs().amax(1) / E4M3_MAX
    buf = torch.zeros(rows, pad, dtype=torch.uint8, device="cuda")
    buf[:, :k] = (v / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return buf.view(torch.float8_e4m3fn)[:, :k], scale


def _prepare_adapters(c, g):
    t = TYPES[c["dtype"]]
    lens, k, n, r, pool = _ints(c["seqs"]), c["k"], c["n"], c["rank"], c["pool"]
    m = sum(lens)
    s = dict(case=c)
    s["x"], s["x_scale"] = _codes(g, m, k)
    s["y"] = _normal(g, m, n).to(t)
    pad = -(-k // 8) * 8
    s["a"] = (_normal(g, pool, r, pad) / math.sqrt(k)).to(t)[:, :, :k]
    s["b"] = (_normal(g, pool, n, r) / math.sqrt(r)).to(t)
    s["scale"] = 0.5 + torch.rand(pool, generator=g, device="cuda")
    s["ranks"] = None
    if c["mixed"]:
        s["ranks"] = torch.randint(max(1, r // 4), r + 1, (pool,), generator=g, device="cuda").to(torch.int32)
    # one request in ten runs without an adapter
    of = torch.randint(0, pool, (len(lens),), generator=g, device="cuda")
    bare = torch.rand(len(lens), generator=g, device="cuda") < 0.1
    of = torch.where(bare, -1, of)
    if len(lens) == 1:
        of = of.clamp(min=0)
    times = torch.tensor(lens, device="cuda")
    s["ids"] = of.repeat_interleave(times, output_size=m).to(torch.int32)
    return s


def _prepare_logprobs(c, g):
    rows, vocab = c["rows"], c["vocab"]
    x = _normal(g, rows, vocab) * 3
    loud = torch.randint(0, vocab, (rows, 3), generator=g, device="cuda")
    x.scatter_(1, loud, 9 + 3 * _normal(g, rows, 3))
    if c["masked"]:  # the same part of the vocabulary is closed to every row
        x.masked_fill_(torch.rand(1, vocab, generator=g, device="cuda") < 0.2, -math.inf)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    tokens = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.7, loud[:, 0], tokens)
    return dict(case=c, logits=x.to(TYPES[c["dtype"]]), tokens=tokens)


# ------------------------------------------------------------------ one pass
def run(s):
    return globals()[("_own_" if own else "_plain_") + s["case"]["op"]](s)


def _own_rotate(s):
    from dac_vocoder_decode_gb300 import binding as V
    q, k = V.rotate_heads(s["q"], s["k"], s["positions"], s["turns"], axis=s["axis"],
                          q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                          neighbours=s["case"]["near"])
    return {"q": q, "k": k}


def _own_adapters(s):
    from dac_vocoder_decode_gb300 import binding as V
    return V.adapters_fp8(s["y"], s["x"], s["x_scale"], s["a"], s["b"], s["scale"], s["ids"],
                          ranks=s["ranks"])


def _own_logprobs(s):
    from dac_vocoder_decode_gb300 import binding as V
    c = s["case"]
    logprob, entropy, top, top_tokens = V.logprobs(s["logits"], s["tokens"], top=c["top"],
                                                   temperature=c["temperature"])
    return {"logprob": logprob, "entropy": entropy, "top": top, "top_tokens": top_tokens}


def _plain_rotate(s):
    c = s["case"]
    pairs = c["turned"] // 2
    at = s["positions"].double().T  # [tokens, axes]
    at = at[:, s["axis"].long()] if s["axis"] is not None else at.expand(-1, pairs)
    angle = at * s["rates"]  # far positions lose their angle in 32 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    return {"q": _turn(s["q"].float(), s["q_weight"], cos, sin, c["near"]).to(s["q"].dtype),
            "k": _turn(s["k"].float(), s["k_weight"], cos, sin, c["near"]).to(s["k"].dtype)}


def _turn(x, weight, cos, sin, near):
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * weight.to(x.dtype)
    pairs = cos.shape[2]
    a, b = _pairs(x, pairs, near)
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], 3).flatten(2) if near else torch.cat([a, b], 2)
    return torch.cat([turned, x[:, :, 2 * pairs:]], 2)


def _pairs(x, pairs, near):
    if near:
        return x[:, :, 0:2 * pairs:2], x[:, :, 1:2 * pairs:2]
    return x[:, :, :pairs], x[:, :, pairs:2 * pairs]


def _plain_adapters(s):
    c, pool, r = s["case"], s["case"]["pool"], s["case"]["rank"]
    m = len(s["ids"])
    x = s["x"].float() * s["x_scale"][:, None]
    v = (x @ s["a"].float().reshape(pool * r, -1).T).view(m, pool, r)
    use = (s["ids"][:, None] == torch.arange(pool, device="cuda")) * s["scale"]  # [m, pool]
    v = v * use[:, :, None]
    if s["ranks"] is not None:
        v = v * (torch.arange(r, device="cuda") < s["ranks"][:, None])
    b = s["b"].float().permute(0, 2, 1).reshape(pool * r, c["n"])
    return (s["y"].float() + v.view(m, pool * r) @ b).to(s["y"].dtype)


def _plain_logprobs(s):
    c, x = s["case"], s["logits"].float() / s["case"]["temperature"]
    low = x - x.amax(1, keepdim=True)
    e = torch.exp(low)
    total = e.sum(1)
    lse = torch.log(total)
    logprob = low.gather(1, s["tokens"][:, None])[:, 0] - lse
    entropy = lse - torch.where(e > 0, e * low, torch.zeros_like(e)).sum(1) / total
    del e
    if not c["top"]:
        return {"logprob": logprob, "entropy": entropy, "top": None, "top_tokens": None}
    order = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices[:, :c["top"]]
    return {"logprob": logprob, "entropy": entropy, "top": low.gather(1, order) - lse[:, None],
            "top_tokens": order}


# ------------------------------------------------------------------ what a pass has to move
def work(case):
    c = case
    if c["op"] == "rotate":
        n = c["tokens"] * (c["heads"] + c["kv_heads"]) * c["d"]
        return dict(bytes=4 * n + 4 * c["axes"] * c["tokens"] + 4 * c["turned"],
                    flops=n * (4 if c["norm"] else 0) + 3 * n * c["turned"] // c["d"])
    if c["op"] == "adapters":
        lens, k, n, r = _ints(c["seqs"]), c["k"], c["n"], c["rank"]
        m, used = sum(lens), min(len(lens), c["pool"])
        return dict(bytes=m * k + 4 * m * n + 8 * m + 2 * used * r * (k + n),
                    flops=2 * m * r * (k + n))
    n = c["rows"] * c["vocab"]
    return dict(bytes=n * (4 if c["dtype"] == "f32" else 2) + c["rows"] * (16 + 12 * c["top"]),
                flops=6 * n)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    return globals()["_exact_" + case["op"]](prepare(case, seed))


def _exact_rotate(s):
    c, out = s["case"], {}
    pairs = c["turned"] // 2
    axis = s["axis"].long() if s["axis"] is not None else torch.zeros(pairs, dtype=torch.long,
                                                                      device="cuda")
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                       s["positions"].double()[axis].T * s["rates"])  # complex [tokens, pairs]
    for name in ("q", "k"):
        x = s[name].double()
        if s[name + "_weight"] is not None:
            x = x / (x.pow(2).sum(2, keepdim=True) / c["d"] + EPS).sqrt() * s[name + "_weight"].double()
        a, b = _pairs(x, pairs, c["near"])
        z = torch.complex(a, b) * turn[:, None]
        y = x.clone()
        a, b = _pairs(y, pairs, c["near"])
        a.copy_(z.real)
        b.copy_(z.imag)
        out[name] = y
    return out


def _exact_adapters(s):
    out = s["y"].double()
    for a in range(s["case"]["pool"]):
        rows = torch.nonzero(s["ids"] == a)[:, 0]
        if not len(rows):
            continue
        r = int(s["ranks"][a]) if s["ranks"] is not None else s["case"]["rank"]
        x = s["x"][rows].double() * s["x_scale"][rows].double()[:, None]
        low = x @ s["a"][a, :r].double().T
        out[rows] += float(s["scale"][a]) * (low @ s["b"][a, :, :r].double().T)
    return out


def _exact_logprobs(s):
    c = s["case"]
    k = c["top"]
    got = [[] for _ in range(4)]
    step = max(1, 40_000_000 // c["vocab"])
    for i in range(0, c["rows"], step):
        x = s["logits"][i:i + step].double()
        z = x / c["temperature"]
        lp = z - torch.logsumexp(z, 1, keepdim=True)
        p = lp.exp()
        got[0].append(lp.gather(1, s["tokens"][i:i + step, None])[:, 0])
        got[1].append(-(p * lp.clamp(min=-1e300)).sum(1))
        if k:
            # the k-th largest value; of those equal to it the first ones
            border = x.topk(k, 1).values[:, -1:]
            above = x > border
            tie = x == border
            keep = above | (tie & (tie.cumsum(1) <= k - above.sum(1, keepdim=True)))
            at = torch.nonzero(keep)[:, 1].view(-1, k)  # ascending places
            at = at.gather(1, torch.sort(x.gather(1, at), dim=1, descending=True, stable=True).indices)
            got[2].append(lp.gather(1, at))
            got[3].append(at)
    return {"logprob": torch.cat(got[0]), "entropy": torch.cat(got[1]),
            "top": torch.cat(got[2]) if k else None, "top_tokens": torch.cat(got[3]) if k else None}
