"""Measured cases of the 8-bit operators that a token model runs in front of the decoder.

The latents that the decoder turns into audio come from a transformer that runs frame by frame
(streamed speech) or over a whole prompt (music).  Its layer is four operators over e4m3 values:

  rows       normalise rows (optionally after adding the residual), or take a gated product or
             the rows as they are, and store them as e4m3 with one 32-bit scale per row
  linear     product of e4m3 rows with e4m3 weights, scales per row and per output channel
  append     store keys and values of new tokens in a paged cache: e4m3, one power-of-two scale
             for each block of 64 tokens and head
  attention  softmax attention of the newest tokens over that cache (shared heads, causal,
             optional sliding window), lengths of their own for every sequence

`run` takes the plain form (elementary torch operations in 32 bits) or, with `own`, the calls that
a user makes.  `exact` restates each operator in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 64          # tokens of one cache block (one scale for each block and head)
E4M3_MAX = 448.0
MIN_EXP = -96       # block and row scales stay at or above 2^-96 (rows: over 448)
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one frame of 8 streamed speech sequences, 1024 channels: the smallest call
        dict(name="rows frame 8x1024", op="rows", mode="rms", rows=8, d=1024, dtype="bf16",
             residual=True),
        # the whole prompt of a 180 s song, 1536 channels, residual stream in bf16
        dict(name="rows song 15504x1536", op="rows", mode="rms", rows=15504, d=1536,
             dtype="bf16", residual=True),
        # gated activations of a feed-forward layer at a ragged width, fp16
        dict(name="rows gated 4001x4100", op="rows", mode="gated", rows=4001, d=4100,
             dtype="f16", residual=False),
        # one frame of 8 sequences through a 1024 -> 1536 projection: latency
        dict(name="linear frame 8x1024x1536", op="linear", m=8, k=1024, n=1536, out="bf16",
             bias=True),
        # odd batch of single tokens through a wide layer: the weights' bytes count
        dict(name="linear step 33x4096x12288", op="linear", m=33, k=4096, n=12288, out="bf16",
             bias=False),
        # a song's prompt through a square layer: the tensor cores count
        dict(name="linear song 15504x4096x4096", op="linear", m=15504, k=4096, n=4096,
             out="bf16", bias=False),
        # the newest token of 8 sequences into the cache
        dict(name="append frame 8", op="append", lens="250,249,64,1,2000,65,777,128",
             new="1,1,1,1,1,1,1,1", kv_heads=8, d=128, dtype="bf16"),
        # prompts of several lengths at once
        dict(name="append prompts", op="append", lens="8192,4001,1,2500,130,777",
             new="8192,4001,1,2400,129,700", kv_heads=8, d=128, dtype="bf16"),
        # one speech sequence of 20 s (250 frames), newest frame only: latency
        dict(name="attention frame 250", op="attention", lens="250", new="1", heads=16,
             kv_heads=16, d=64, window=0, dtype="bf16"),
        # 8 songs at their last frame, shared heads: the cache's bytes count
        dict(name="attention step 8x15504", op="attention",
             lens="15504,15504,15504,15504,15504,15504,15504,15504",
             new="1,1,1,1,1,1,1,1", heads=32, kv_heads=8, d=128, window=0, dtype="bf16"),
        # chunks of odd lengths over caches of odd lengths, sliding window
        dict(name="attention chunks", op="attention", lens="2000,689,37,1,1300,250,4001,100",
             new="37,200,37,1,129,16,77,3", heads=16, kv_heads=4, d=64, window=250,
             dtype="f16"),
        # a whole song as one prompt
        dict(name="attention song 15504", op="attention", lens="15504", new="15504", heads=16,
             kv_heads=4, d=128, window=0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _not_3072(v):
    return v + 16 if v == 3072 else v


def draw(rng):
    op = rng.choice(["rows", "linear", "append", "attention", "attention"])
    if op == "rows":
        d = _not_3072(_log(rng, 64, 8192))
        rows = _not_3072(max(1, min(_log(rng, 1, 16384), 32_000_000 // d)))
        mode = rng.choice(["rms", "rms", "gated", "none"])
        return dict(op=op, mode=mode, rows=rows, d=d, dtype=rng.choice(["bf16", "f16", "f32"]),
                    residual=mode != "gated" and rng.random() < 0.7)
    if op == "linear":
        k = _not_3072(16 * _log(rng, 4, 512) - rng.choice([0, 0, 0, 5]))
        n = _not_3072(_log(rng, 64, 12288))
        m = _not_3072(max(1, min(_log(rng, 1, 16384), 250_000_000_000 // (k * n))))
        return dict(op=op, m=m, k=k, n=n, out=rng.choice(["bf16", "f16"]),
                    bias=rng.random() < 0.5)
    kv_heads = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "f16"])
    if op == "append":
        b = _log(rng, 1, 16)
        lens = [_not_3072(_log(rng, 1, 4000)) for _ in range(b)]
        new = [1] * b if rng.random() < 0.4 else _part(rng, lens)
        return dict(op=op, lens=_text(lens), new=_text(new), kv_heads=kv_heads, d=d, dtype=dtype)
    heads = kv_heads * rng.choice([1, 2, 4, 7])
    window = rng.choice([0, 0, 72, 1000])
    if rng.random() < 0.6:  # single tokens
        b = _log(rng, 1, 16)
        lens = [_not_3072(_log(rng, 1, 16000)) for _ in range(b)]
        new = [1] * b
    else:
        b = _log(rng, 1, 6)
        lens = [_not_3072(_log(rng, 1, 6000)) for _ in range(b)]
        new = _part(rng, lens)
    return dict(op=op, lens=_text(lens), new=_text(new), heads=heads, kv_heads=kv_heads, d=d,
                window=window, dtype=dtype)


def _part(rng, lens):
    """A number of new tokens for each length."""
    new = [_log(rng, 1, n) for n in lens]
    return [n - 1 if n == 3072 else n for n in new]


def _text(values):
    return ",".join(str(v) for v in values)


def _ints(text):
    return [int(v) for v in text.split(",")]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return globals()["_prepare_" + case["op"]](case, g)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _prepare_rows(c, g):
    t = TYPES[c["dtype"]]
    width = 2 * c["d"] if c["mode"] == "gated" else c["d"]
    # a residual stream has channels far larger than the rest
    loud = 1 + 7 * (torch.rand(width, generator=g, device="cuda") < 0.02)
    s = dict(case=c, x=(_normal(g, c["rows"], width) * loud).to(t), residual=None, weight=None)
    if c["residual"]:
        s["residual"] = (_normal(g, c["rows"], width) * loud).to(t)
    if c["mode"] == "rms":
        s["weight"] = (1 + 0.2 * _normal(g, width)).to(t)
    return s


def _codes(g, rows, k):
    """Random e4m3 rows as a quantiser leaves them (largest value at 448), rows padded to 16."""
    pad = -(-k // 16) * 16
    v = _normal(g, rows, k)
    scale = v.abs().amax(1) / E4M3_MAX
    buf = torch.zeros(rows, pad, dtype=torch.uint8, device="cuda")
    buf[:, :k] = (v / scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return buf.view(torch.float8_e4m3fn)[:, :k], scale


def _prepare_linear(c, g):
    s = dict(case=c)
    s["x"], s["x_scale"] = _codes(g, c["m"], c["k"])
    s["w"], s["w_scale"] = _codes(g, c["n"], c["k"])
    s["w_scale"] = s["w_scale"] / math.sqrt(c["k"])
    s["bias"] = _normal(g, c["n"]) if c["bias"] else None
    return s


def _pages(c, g):
    """Blocks of every sequence, in a shuffled pool."""
    lens = _ints(c["lens"])
    blocks = [-(-n // BLOCK) for n in lens]
    pool = sum(blocks) + 1
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(blocks)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    new = _ints(c["new"])
    cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32,
                      device="cuda")
    return dict(case=c, page_table=table, pool=pool, max_q=max(new), max_kv=max(lens),
                kv_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                cu_q=None if all(n == 1 for n in new) else cu, total=sum(new))


def _cache(c, g, pool):
    """A pool of blocks as the cache keeps it: K [page][head][token][d], V [page][head][d][token]."""
    heads, d = c["kv_heads"], c["d"]
    loud = 1 + 5 * (torch.rand(heads, 1, d, generator=g, device="cuda") < 0.03)
    k = _normal(g, pool, heads, BLOCK, d) * loud
    v = _normal(g, pool, heads, d, BLOCK)
    out = []
    for t in (k, v):
        e = _exponent(t.abs().amax((2, 3)))
        out.append((torch.ldexp(t, -e[..., None, None])).to(torch.float8_e4m3fn))
        out.append(torch.ldexp(torch.ones_like(e, dtype=torch.float32), e))
    return dict(k=out[0], k_scale=out[1], v=out[2], v_scale=out[3])


def _exponent(amax):
    """Smallest e >= MIN_EXP with amax <= 448 * 2^e."""
    f, x = torch.frexp(amax)
    e = torch.where(f <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)


def _prepare_append(c, g):
    s = _pages(c, g)
    s.update(_cache(c, g, s["pool"]))
    t = TYPES[c["dtype"]]
    shape = (s["total"], c["kv_heads"], c["d"])
    s["new_k"] = (_normal(g, *shape) * 1.5).to(t)
    s["new_v"] = _normal(g, *shape).to(t)
    return s


def _prepare_attention(c, g):
    s = _pages(c, g)
    s.update(_cache(c, g, s["pool"]))
    s["q"] = (_normal(g, s["total"], c["heads"], c["d"]) * 1.2).to(TYPES[c["dtype"]])
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return globals()[("_own_" if own else "_plain_") + s["case"]["op"]](s)


def _own_rows(s):
    from dac_vocoder_decode_gb300 import binding as V
    mode = {"rms": V.VOC_LM_RMS, "none": V.VOC_LM_NONE, "gated": V.VOC_LM_GATED}
    q, scale, total = V.rows_fp8(s["x"], mode[s["case"]["mode"]], weight=s["weight"],
                                 residual=s["residual"], eps=1e-6)
    return {"q": q, "scale": scale, "sum": total}


def _own_linear(s):
    from dac_vocoder_decode_gb300 import binding as V
    return V.linear_fp8(s["x"], s["x_scale"], s["w"], s["w_scale"], bias=s["bias"],
                        out_dtype=TYPES[s["case"]["out"]])


def _own_append(s):
    from dac_vocoder_decode_gb300 import binding as V
    cache = V.KVCacheFP8(s["k"], s["v"], s["k_scale"], s["v_scale"])
    V.kv_append_fp8(cache, s["new_k"], s["new_v"], s["page_table"], s["kv_lens"],
                    cu_q=s["cu_q"], max_q=s["max_q"])
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _own_attention(s):
    from dac_vocoder_decode_gb300 import binding as V
    cache = V.KVCacheFP8(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return V.attention_fp8(s["q"], cache, s["page_table"], s["kv_lens"], cu_q=s["cu_q"],
                           max_q=s["max_q"], max_kv=s["max_kv"], window=s["case"]["window"])


def _plain_rows(s):
    c, x = s["case"], s["x"].float()
    total = None
    if s["residual"] is not None:
        x = x + s["residual"].float()
        total = x.to(s["x"].dtype)
    if c["mode"] == "rms":
        x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-6) * s["weight"].float()
    elif c["mode"] == "gated":
        gate, up = x[:, :c["d"]], x[:, c["d"]:]
        x = gate / (1 + torch.exp(-gate)) * up
    scale = x.abs().amax(1).clamp(min=2.0 ** MIN_EXP) / E4M3_MAX
    return {"q": (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn),
            "scale": scale, "sum": total}


def _plain_linear(s):
    y = s["x"].float() @ s["w"].float().T
    y = y * s["x_scale"][:, None] * s["w_scale"][None, :]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(TYPES[s["case"]["out"]])


def _token_places(s):
    """Sequence and position of every new token."""
    n = s["total"]
    if s["cu_q"] is None:
        b = torch.arange(n, device="cuda")
        return b, s["kv_lens"].long() - 1
    i = torch.arange(n, device="cuda")
    b = torch.searchsorted(s["cu_q"].long(), i, right=True) - 1
    new = s["cu_q"][1:].long() - s["cu_q"][:-1].long()
    return b, (s["kv_lens"].long() - new)[b] + i - s["cu_q"].long()[b]


def _plain_append(s):
    c = s["case"]
    heads, d, pool = c["kv_heads"], c["d"], s["pool"]
    b, pos = _token_places(s)
    page = s["page_table"][b, pos // BLOCK].long()
    slot = pos % BLOCK
    fresh = torch.zeros(pool, dtype=torch.bool, device="cuda")
    fresh[page[slot == 0]] = True
    taken = torch.zeros(pool, BLOCK, dtype=torch.bool, device="cuda")
    taken[page, slot] = True
    written = torch.zeros(pool, dtype=torch.bool, device="cuda")
    written[page] = True
    for name, token_axis in (("k", 2), ("v", 3)):
        new = s["new_" + name].float()
        old_scale = s[name + "_scale"]
        need = torch.zeros(pool, heads, device="cuda")
        need.scatter_reduce_(0, page[:, None].expand(-1, heads), new.abs().amax(2), "amax")
        e = _exponent(need)
        scale = torch.ldexp(torch.ones_like(need), e)
        scale = torch.where(fresh[:, None], scale, torch.maximum(scale, old_scale))
        # earlier codes move to the new scale; the free slots of a fresh block hold zeros
        codes = s[name].float() * (old_scale / scale)[:, :, None, None]
        codes = torch.where(fresh[:, None, None, None], torch.zeros_like(codes), codes)
        if token_axis == 3:
            codes = codes.transpose(2, 3).contiguous()
        codes[page, :, slot] = new / scale[page][:, :, None]
        if token_axis == 3:
            codes = codes.transpose(2, 3)
        codes = codes.to(torch.float8_e4m3fn).view(torch.uint8)
        s[name].view(torch.uint8).copy_(
            torch.where(written[:, None, None, None], codes, s[name].view(torch.uint8)))
        old_scale.copy_(torch.where(written[:, None], scale, old_scale))
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _dense(s, dtype):
    """The caches as [B, heads, tokens, d] in `dtype`."""
    c = s["case"]
    pages = s["page_table"].long().clamp(min=0)
    at = pages.flatten()
    n = (len(pages), pages.shape[1], c["kv_heads"])
    k = s["k"].view(torch.uint8)[at].view(torch.float8_e4m3fn).to(dtype)
    v = s["v"].view(torch.uint8)[at].view(torch.float8_e4m3fn).to(dtype)
    k = (k * s["k_scale"][at].to(dtype)[:, :, None, None]).view(*n, BLOCK, c["d"])
    v = (v * s["v_scale"][at].to(dtype)[:, :, None, None]).view(*n, c["d"], BLOCK)
    k = k.permute(0, 2, 1, 3, 4).reshape(n[0], n[2], -1, c["d"])
    v = v.permute(0, 2, 1, 4, 3).reshape(n[0], n[2], -1, c["d"])
    return k, v


def _plain_attention(s):
    c = s["case"]
    heads, kv_heads, d = c["heads"], c["kv_heads"], c["d"]
    group = heads // kv_heads
    k, v = _dense(s, torch.float32)
    b, pos = _token_places(s)
    nb, tokens, mq = len(s["kv_lens"]), k.shape[2], s["max_q"]
    first = s["cu_q"].long()[b] if s["cu_q"] is not None else torch.arange(len(b), device="cuda")
    i = torch.arange(len(b), device="cuda") - first
    q = torch.zeros(nb, mq, heads, d, device="cuda")
    q[b, i] = s["q"].float()
    where = torch.full((nb, mq), -1, dtype=torch.long, device="cuda")  # position of each query
    where[b, i] = pos
    q = q.view(nb, mq, kv_heads, group, d).permute(0, 2, 3, 1, 4).reshape(nb, kv_heads, -1, d)
    sc = (q @ k.transpose(2, 3)).view(nb, kv_heads, group, mq, tokens)
    sc *= 1 / math.sqrt(d)
    key = torch.arange(tokens, device="cuda")
    hidden = key[None, None, :] > where[:, :, None]
    if c["window"]:
        hidden |= key[None, None, :] <= where[:, :, None] - c["window"]
    sc.masked_fill_(hidden[:, None, None], -math.inf)
    top = sc.amax(4, keepdim=True)
    sc -= torch.where(top == -math.inf, torch.zeros_like(top), top)
    sc.exp_()
    total = sc.sum(4, keepdim=True)
    o = (sc.view(nb, kv_heads, group * mq, tokens) @ v).view(nb, kv_heads, group, mq, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(nb, mq, heads, d)
    return o[b, i].to(s["q"].dtype)


# ------------------------------------------------------------------ what a pass has to move
def work(case):
    c = case
    if c["op"] == "rows":
        e = 4 if c["dtype"] == "f32" else 2
        n = c["rows"] * c["d"]
        moved = n * e * (2 if c["mode"] == "gated" else 1) + n + 4 * c["rows"]
        moved += 2 * n * e if c["residual"] else 0
        return dict(bytes=moved + (c["d"] * e if c["mode"] == "rms" else 0), flops=8 * n)
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        return dict(bytes=m * k + n * k + 2 * m * n + 4 * (m + n) + (4 * n if c["bias"] else 0),
                    flops=2 * m * n * k)
    lens, new = _ints(c["lens"]), _ints(c["new"])
    row = c["kv_heads"] * c["d"]
    if c["op"] == "append":
        # the new tokens once in 16 bits and once as codes, and the codes that share their
        # first block read for its scale
        return dict(bytes=2 * row * 3 * sum(new), flops=2 * row * 2 * sum(new))
    seen, pairs = 0, 0
    for n, m in zip(lens, new):
        w = c["window"] or n
        seen += min(n, m - 1 + w)
        for p in (n - m, n - 1):  # the number of visible keys is linear in between, or w
            pairs += min(p + 1, w) * m / 2
        if n - m + 1 < w < n:     # it saturates on the way
            rise = w - (n - m + 1)
            pairs += (w - (n - m + 1)) * (m - rise) / 2
    return dict(bytes=2 * row * seen + 4 * c["heads"] * c["d"] * sum(new),
                flops=4 * c["heads"] * c["d"] * pairs)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    return globals()["_exact_" + case["op"]](prepare(case, seed))


def _exact_rows(s):
    c = s["case"]
    x = s["x"].double()
    total = None
    if s["residual"] is not None:
        total = x = x + s["residual"].double()
    if c["mode"] == "rms":
        rms = (x.pow(2).sum(1) / c["d"] + 1e-6).sqrt()
        x = x / rms[:, None] * s["weight"].double()
    elif c["mode"] == "gated":
        x = x[:, :c["d"]] * torch.sigmoid(x[:, :c["d"]]) * x[:, c["d"]:]
    scale = x.abs().max(1).values.clamp(min=2.0 ** MIN_EXP) / E4M3_MAX
    return {"q": x / scale[:, None], "scale": scale, "sum": total}


def _exact_linear(s):
    m, n, k = (s["case"][w] for w in "mnk")
    w = s["w"].double() * s["w_scale"].double()[:, None]
    y = torch.empty(m, n, dtype=torch.float64, device="cuda")
    for a in range(0, m, 4096):
        x = s["x"][a:a + 4096].double() * s["x_scale"][a:a + 4096].double()[:, None]
        y[a:a + 4096] = x @ w.T
    return y if s["bias"] is None else y + s["bias"].double()


def _exact_append(s):
    c = s["case"]
    table, lens, new = s["page_table"].tolist(), _ints(c["lens"]), _ints(c["new"])
    out = {n: s[n].double() for n in ("k", "v", "k_scale", "v_scale")}
    at = 0
    for b in range(len(lens)):
        pos = lens[b] - new[b]
        while pos < lens[b]:
            end = min(lens[b], (pos // BLOCK + 1) * BLOCK)
            page, lo, hi = table[b][pos // BLOCK], pos % BLOCK, pos % BLOCK + end - pos
            for n in ("k", "v"):
                t = s["new_" + n][at:at + end - pos].double().transpose(0, 1)  # [head][token][d]
                amax = t.abs().amax((1, 2))
                # 16-bit inputs: the ratio is a power of two or at least 2^-11 away from one, so
                # the margin only keeps the logarithm's own rounding from counting
                scale = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX) - 1e-6))
                scale = scale.clamp(min=2.0 ** MIN_EXP)
                block = out[n][page] if n == "k" else out[n][page].transpose(1, 2)
                if lo == 0:
                    block.zero_()
                else:
                    scale = torch.maximum(scale, out[n + "_scale"][page])
                    block *= (out[n + "_scale"][page] / scale)[:, None, None]
                block[:, lo:hi] = t / scale[:, None, None]
                out[n + "_scale"][page] = scale
            at += end - pos
            pos = end
    return out


def _exact_attention(s):
    c = s["case"]
    lens, new = _ints(c["lens"]), _ints(c["new"])
    heads, d = c["heads"], c["d"]
    group = heads // c["kv_heads"]
    k, v = _dense(s, torch.float64)
    out = torch.empty(s["total"], heads, d, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        step = max(1, min(m, 300_000_000 // n))
        for h in range(heads):
            kh, vh = k[b, h // group, :n], v[b, h // group, :n]
            for a in range(0, m, step):
                z = min(m, a + step)
                q = s["q"][at + a:at + z, h].double()
                sc = q @ kh.T / math.sqrt(d)
                p = torch.arange(n - m + a, n - m + z, device="cuda")[:, None]
                key = torch.arange(n, device="cuda")[None, :]
                seen = key <= p
                if c["window"]:
                    seen &= key > p - c["window"]
                w = torch.softmax(sc.masked_fill(~seen, -math.inf), 1)
                out[at + a:at + z, h] = w @ vh
        at += m
    return out
