"""GPU: the stack in front of the decoder as a token model: heads turned by position, a low-rank adapter for
each sequence, log probabilities of codes, together.

Bounds, set beforehand, as for the plain stack: streaming and one prompt take the same sums in other orders
and differ by a code's step now and then, below one rounding of everything, 2^-4; against the same stack in
64 bits without any rounding, two layers of four rounded operands of 2.6 % each stay below 20 %.  Log
probabilities of given logits: 32-bit sums, 1e-5."""
from __future__ import annotations

import dataclasses
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("no CUDA device", allow_module_level=True)

from dac_vocoder_decode_gb300 import binding as V  # noqa: E402
from dac_vocoder_decode_gb300.front import Front, FrontArch  # noqa: E402

PLAIN = FrontArch(latent=64, dim=192, layers=2, heads=6, kv_heads=2, head_dim=64, hidden=160,
                  window=40, books=4, entries=64)
TOKEN = dataclasses.replace(PLAIN, rotary=True, voices=3, rank=8, head=True)


def _codes(B, n, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, PLAIN.entries, (B, n, PLAIN.books), generator=g, device="cuda")


def _off(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def _plain(front, codes, last):
    """The stack in 64 bits, the weights as the codes stand for them; `last`: its last product."""
    a, (B, n, _) = front.arch, codes.shape
    w = lambda p: p[0].double() * p[1].double()[:, None]  # noqa: E731
    norm = lambda x, g: x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * g.double()  # noqa: E731

    def product(p, name, x):
        y = x @ w(p[name]).T
        if a.voices:
            down, up, scale = p[name + "_voice"]
            for b, i in enumerate(front.voice.tolist()):
                if i >= 0:
                    y[b] += float(scale[i]) * (x[b] @ down[i].double().T) @ up[i].double().T
        return y

    at = torch.arange(n, device="cuda")
    x = front.embed.double()[torch.arange(a.books, device="cuda"), codes].sum(2)
    if not a.rotary:
        turn = at[:, None] * front.rates.double()
        x = x + torch.cat([turn.sin(), turn.cos()], 1)
    seen = (at[None] <= at[:, None]) & (at[None] > at[:, None] - a.window)
    half = a.head_dim // 2
    angle = at[:, None] * torch.exp(-math.log(1e4) * torch.arange(half, device="cuda").double() / half)

    def turned(x, g):
        x = norm(x, g)
        u, v = x[..., :half], x[..., half:]
        return torch.cat([u * angle.cos() - v * angle.sin(), u * angle.sin() + v * angle.cos()], -1)

    for p in front.layers:
        qkv = product(p, "qkv", norm(x, p["norm1"])).view(B, n, -1, a.head_dim).transpose(1, 2)
        q, k, v = qkv.split([a.heads, a.kv_heads, a.kv_heads], 1)
        if a.rotary:
            q, k = turned(q, p["q_norm"]), turned(k, p["k_norm"])
        k, v = (t.repeat_interleave(a.heads // a.kv_heads, 1) for t in (k, v))
        s = (q @ k.transpose(2, 3) / math.sqrt(a.head_dim)).masked_fill(~seen, -math.inf)
        x = x + product(p, "out", (s.softmax(-1) @ v).transpose(1, 2).reshape(B, n, -1))
        g, u = (norm(x, p["norm2"]) @ w(p["up"]).T).chunk(2, -1)
        x = x + (torch.nn.functional.silu(g) * u) @ w(p["down"]).T
    return norm(x, front.last_norm) @ w(last).T


def _voices(front, *voice):
    front.voice.copy_(torch.tensor(voice, dtype=torch.int32))


def test_options_leave_the_plain_stack_as_it_is():
    codes = _codes(2, 30)
    a, b = Front(PLAIN, 2, 30), Front(dataclasses.replace(PLAIN, voices=3, rank=8, head=True), 2, 30)
    assert torch.equal(a.prompt(codes), b.prompt(codes))  # no sequence has a voice


@pytest.mark.parametrize("rotary,voices", [(True, 0), (False, 3), (True, 3)])
def test_prompt_against_64_bits(rotary, voices):
    codes = _codes(3, 130)
    front = Front(dataclasses.replace(TOKEN, rotary=rotary, voices=voices), 3, 130)
    if voices:
        _voices(front, 2, -1, 0)
    y = front.prompt(codes)
    assert _off(y, _plain(front, codes, front.last).transpose(1, 2)) < 0.2
    if voices:  # a voice makes a difference, to its own sequence
        front.reset()
        _voices(front, 1, -1, 0)
        z = front.prompt(codes)
        assert _off(z[0], y[0]) > 0.01 and torch.equal(z[1:], y[1:])


@pytest.mark.parametrize("prompt", [1, 63, 70])
def test_streamed_frames_match_one_prompt(prompt):
    codes = _codes(2, 100, seed=prompt)
    front = Front(TOKEN, 2, 100)
    _voices(front, 1, 2)
    whole = front.prompt(codes).clone()
    front.reset()
    got = [front.prompt(codes[:, :prompt])]
    got += [front.step(codes[:, i]).clone() for i in range(prompt, 100)]
    assert _off(torch.cat(got, 2), whole) < 2 ** -4


def test_captured_steps_follow_the_voices():
    """The graph of a step reads the voices of the moment, not those of its capture."""
    codes = _codes(2, 40, seed=3)
    front, again = Front(TOKEN, 2, 40), Front(TOKEN, 2, 40)
    for f, late in ((front, False), (again, True)):
        _voices(f, *((0, 0) if late else (2, -1)))
        if late:
            f.step(codes[:, 0])  # captured with other voices
            f.reset()
            _voices(f, 2, -1)
    a = torch.cat([front.step(codes[:, i]).clone() for i in range(40)], 2)
    b = torch.cat([again.step(codes[:, i]).clone() for i in range(40)], 2)
    assert torch.equal(a, b)


@pytest.mark.parametrize("top,temperature", [(0, 1.0), (5, 0.8)])
def test_score(top, temperature):
    codes = _codes(2, 50, seed=5)
    front = Front(TOKEN, 2, 100)
    _voices(front, -1, 1)
    logprob, entropy, best, best_codes = front.score(codes, top=top, temperature=temperature)
    assert logprob.shape == (2, 49, 4) and entropy.shape == (2, 50, 4)
    # the logits, once more
    front.reset()
    front.lens += 50
    h, hs = front._hidden(codes, 50, 50)
    logits = V.linear_fp8(h, hs, *front.codes_head, out_dtype=torch.float32).view(2, 50, 4, 64)
    lp = torch.log_softmax(logits.double() / temperature, -1)
    want = lp[:, :-1].gather(3, codes[:, 1:, :, None])[..., 0]
    assert float((logprob - want).abs().max()) < 1e-5 * float(want.abs().max())
    assert float((entropy + (lp.exp() * lp).sum(-1)).abs().max()) < 1e-4
    if top:
        values, at = lp.topk(top, -1)
        assert best.shape == (2, 50, 4, top) and torch.equal(best_codes, at)
        assert float((best - values).abs().max()) < 1e-4
    else:
        assert best is None and best_codes is None
    ref = _plain(front, codes, front.codes_head).view(2, 50, 4, 64)
    assert _off(logits, ref) < 0.2


def test_score_goes_on_with_the_sequence():
    """Scored in two parts, the second sees the first; the likeliest codes can be fed back."""
    codes = _codes(2, 60, seed=6)
    front = Front(TOKEN, 2, 61)
    whole = front.score(codes)[0]
    front.reset()
    a, b = front.score(codes[:, :33])[0], front.score(codes[:, 33:], top=1)
    assert float((torch.cat([a, whole[:, 32:33], b[0]], 1) - whole).abs().mean()) < 0.1
    front.step(b[3][:, -1, :, 0])
    with pytest.raises(V.VocoderError) as e:
        front.score(codes[:, :1])
    assert e.value.status == V.VOC_INVALID_ARG


def test_score_needs_a_head():
    front = Front(PLAIN, 1, 5)
    with pytest.raises(V.VocoderError) as e:
        front.score(_codes(1, 5))
    assert e.value.status == V.VOC_INVALID_ARG and front.frames == 0
