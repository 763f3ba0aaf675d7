"""GPU: the 8-bit operators together, as the stack in front of the decoder uses them.

Bounds, set beforehand: one e4m3 rounding is off by at most 2^-4 of a value, 2.6% in the mean square.
  - Streaming frame by frame and one prompt take the same sums in other orders, which moves a code by
    a step now and then and nothing else: far below one rounding of everything, 2^-4.
  - Against the same stack in 64 bits without any rounding, each layer adds four rounded operands
    (2.6% each of a branch): two layers of them and the last product stay below 20%.
"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, never run there
    pytest.skip("no CUDA device", allow_module_level=True)

from dac_vocoder_decode_gb300 import binding as V  # noqa: E402
from dac_vocoder_decode_gb300 import workloads as W  # noqa: E402
from dac_vocoder_decode_gb300.front import Front, FrontArch  # noqa: E402

ARCH = FrontArch(latent=64, dim=192, layers=2, heads=6, kv_heads=2, head_dim=64, hidden=160,
                 window=40, books=4, entries=64)


def _codes(B, n, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, ARCH.entries, (B, n, ARCH.books), generator=g, device="cuda")


def _off(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def _plain(front, codes):
    """The stack in 64 bits, the weights as the codes stand for them."""
    a, (B, n, _) = front.arch, codes.shape
    w = lambda p: p[0].double() * p[1].double()[:, None]  # noqa: E731
    norm = lambda x, g: x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * g.double()  # noqa: E731
    at = torch.arange(n, device="cuda")
    turn = at[:, None] * front.rates.double()
    x = front.embed.double()[torch.arange(a.books, device="cuda"), codes].sum(2)
    x = x + torch.cat([turn.sin(), turn.cos()], 1)
    seen = (at[None] <= at[:, None]) & (at[None] > at[:, None] - a.window)
    for p in front.layers:
        qkv = (norm(x, p["norm1"]) @ w(p["qkv"]).T).view(B, n, -1, a.head_dim).transpose(1, 2)
        q, k, v = qkv.split([a.heads, a.kv_heads, a.kv_heads], 1)
        k, v = (t.repeat_interleave(a.heads // a.kv_heads, 1) for t in (k, v))
        s = (q @ k.transpose(2, 3) / math.sqrt(a.head_dim)).masked_fill(~seen, -math.inf)
        o = (s.softmax(-1) @ v).transpose(1, 2).reshape(B, n, -1)
        x = x + o @ w(p["out"]).T
        g, u = (norm(x, p["norm2"]) @ w(p["up"]).T).chunk(2, -1)
        x = x + (torch.nn.functional.silu(g) * u) @ w(p["down"]).T
    return (norm(x, front.last_norm) @ w(front.last).T).transpose(1, 2)


def test_prompt_against_64_bits():
    codes = _codes(3, 130)
    front = Front(ARCH, 3, 130)
    y = front.prompt(codes)
    assert y.shape == (3, ARCH.latent, 130) and y.dtype == torch.float32
    assert _off(y, _plain(front, codes)) < 0.2


@pytest.mark.parametrize("prompt", [1, 63, 70])
def test_streamed_frames_match_one_prompt(prompt):
    codes = _codes(2, 100, seed=prompt)
    front = Front(ARCH, 2, 100)
    whole = front.prompt(codes).clone()
    front.reset()
    got = [front.prompt(codes[:, :prompt])]
    got += [front.step(codes[:, i]).clone() for i in range(prompt, 100)]
    got = torch.cat(got, 2)
    assert _off(got, whole) < 2 ** -4


def test_more_frames_than_room_are_refused():
    front = Front(ARCH, 1, 3)
    front.prompt(_codes(1, 3))
    with pytest.raises(V.VocoderError) as e:
        front.step(_codes(1, 1)[:, 0])
    assert e.value.status == V.VOC_INVALID_ARG


def test_latents_stream_into_the_decoder():
    """Latents of the stack, streamed through a causal decoder, equal one decode of all of them."""
    arch = W.Arch(latent_channels=64, channels0=128, strides=(8, 5, 4, 4, 3),
                  widths=(96, 64, 48, 32, 16), padding=V.VOC_PAD_CAUSAL)
    wl = W.make_custom(arch, B=2, T=20, seed=5)
    voc = V.Vocoder(arch, V.fold_params(wl.params))
    stream = V.VocoderStream(voc, 2, 10)
    front = Front(ARCH, 2, 20)
    codes = _codes(2, 20, seed=9)
    latents = [front.prompt(codes[:, :10]).clone()]
    audio = [stream.decode(latents[0])]
    for i in range(10, 20):
        latents.append(front.step(codes[:, i]).clone())
        audio.append(stream.decode(latents[-1]))
    whole = voc.decode(torch.cat(latents, 2).contiguous(), flags=V.VOC_FLAG_SYNC)
    assert torch.equal(torch.cat(audio, 2), whole)
    stream.close()
    voc.close()
