"""A small transformer in front of the decoder, on the library's 8-bit operators.

The published pipelines decode latents that a transformer makes: for a whole prompt at once, or
frame by frame beside the streamed decode (qwentts.cpp Architecture, "Streaming decode (stateful
path)").  ``Front`` is such a stack with random weights: codes of a residual quantiser are looked up
and summed, each layer is

    rows (RMS norm, residual added)  -> product -> q | k | v
    cache append, attention          -> rows (as they are) -> product
    rows (RMS norm, residual added)  -> product -> rows (gated) -> product

and the last norm's product gives fp32 latents for ``Vocoder.decode`` or ``VocoderStream.decode``.

    python -m dac_vocoder_decode_gb300.front        # a prompt, then streamed frames to audio
"""
from __future__ import annotations

import dataclasses
import math

from . import binding as V


@dataclasses.dataclass
class FrontArch:
    """Sizes of the stack: `latent` channels out, `books` codebooks of `entries` codes in."""
    latent: int = 1024
    dim: int = 1024
    layers: int = 4
    heads: int = 16
    kv_heads: int = 4
    head_dim: int = 64
    hidden: int = 2048
    window: int = 250  # keys that a query sees at most (0: all)
    books: int = 16
    entries: int = 2048


class Front:
    """The stack for B sequences of up to `max_frames` frames on the current CUDA device."""

    def __init__(self, arch: FrontArch, B: int, max_frames: int, seed: int = 0):
        import torch
        self.arch, self.B, self.max_frames = arch, B, max_frames
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            """Random [n, k] weights in e4m3, a scale for each output channel."""
            w = torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k)
            return V.rows_fp8(w, V.VOC_LM_NONE)[:2]

        def norm(n):
            return (1 + 0.1 * torch.randn(n, generator=g, device="cuda")).bfloat16()

        a = arch
        self.embed = torch.randn((a.books, a.entries, a.dim), generator=g, device="cuda") \
            / math.sqrt(a.books)
        self.layers = [dict(norm1=norm(a.dim), norm2=norm(a.dim),
                            qkv=weight((a.heads + 2 * a.kv_heads) * a.head_dim, a.dim),
                            out=weight(a.dim, a.heads * a.head_dim),
                            up=weight(2 * a.hidden, a.dim), down=weight(a.dim, a.hidden))
                       for _ in range(a.layers)]
        self.last_norm, self.last = norm(a.dim), weight(a.latent, a.dim)
        blocks = (max_frames + V.VOC_LM_BLOCK - 1) // V.VOC_LM_BLOCK
        self.cache = [V.KVCacheFP8.empty(B * blocks, a.kv_heads, a.head_dim)
                      for _ in range(a.layers)]
        self.page_table = torch.arange(B * blocks, dtype=torch.int32, device="cuda").view(B, blocks)
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.frames = 0  # of every sequence, on the host
        half = torch.arange(a.dim // 2, device="cuda") / (a.dim // 2)
        self.rates = torch.exp(-math.log(1e4) * half)
        self._graph = None

    def reset(self):
        """Forget all frames."""
        self.lens.zero_()
        self.frames = 0

    def _run(self, codes, new: int, max_kv: int):
        """codes [B, new, books] -> latents [B, latent, new] fp32; the lengths on the device count
        the new frames already."""
        import torch
        a = self.arch
        at = self.lens[:, None] - new + torch.arange(new, device="cuda")  # positions
        turn = at[:, :, None] * self.rates
        x = self.embed[torch.arange(a.books, device="cuda"), codes].sum(2)
        x = (x + torch.cat([turn.sin(), turn.cos()], 2)).view(-1, a.dim).bfloat16()
        delta = None
        for p, cache in zip(self.layers, self.cache):
            h, hs, total = V.rows_fp8(x, V.VOC_LM_RMS, weight=p["norm1"], residual=delta)
            x = x if total is None else total
            qkv = V.linear_fp8(h, hs, *p["qkv"]).view(-1, a.heads + 2 * a.kv_heads, a.head_dim)
            q, k, v = qkv.split([a.heads, a.kv_heads, a.kv_heads], 1)
            V.kv_append_fp8(cache, k, v, self.page_table, self.lens, max_q=new)
            o = V.attention_fp8(q, cache, self.page_table, self.lens, max_q=new, max_kv=max_kv,
                                window=a.window)
            h, hs, _ = V.rows_fp8(o.view(-1, a.heads * a.head_dim), V.VOC_LM_NONE)
            delta = V.linear_fp8(h, hs, *p["out"])
            h, hs, x = V.rows_fp8(x, V.VOC_LM_RMS, weight=p["norm2"], residual=delta)
            h, hs, _ = V.rows_fp8(V.linear_fp8(h, hs, *p["up"]), V.VOC_LM_GATED)
            delta = V.linear_fp8(h, hs, *p["down"])
        h, hs, _ = V.rows_fp8(x, V.VOC_LM_RMS, weight=self.last_norm, residual=delta)
        y = V.linear_fp8(h, hs, *self.last, out_dtype=torch.float32)
        return y.view(self.B, new, a.latent).transpose(1, 2).contiguous()

    def _room(self, new: int):
        if self.frames + new > self.max_frames:
            raise V.VocoderError(V.VOC_INVALID_ARG, f"beyond max_frames = {self.max_frames}")
        self.frames += new

    def prompt(self, codes):
        """The next codes [B, new, books] (int64, on the device) of every sequence at once ->
        latents [B, latent, new]."""
        self._room(codes.shape[1])
        self.lens += codes.shape[1]
        return self._run(codes, codes.shape[1], self.frames)

    def step(self, codes):
        """One frame of codes [B, books] of every sequence -> latents [B, latent, 1].  The launches
        are captured into a CUDA graph with the first call and replayed from then on; the result is
        overwritten by the next call."""
        import torch
        self._room(1)
        if self._graph is None:
            self._codes = codes.clone().view(self.B, 1, -1)
            self.lens += 1
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):  # lookups and limits are set up outside of the capture
                self._run(self._codes, 1, self.max_frames)
            torch.cuda.current_stream().wait_stream(side)
            self.lens -= 1
            self._graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self._graph):
                self.lens += 1
                self._latent = self._run(self._codes, 1, self.max_frames)
        self._codes.copy_(codes.view(self.B, 1, -1))
        self._graph.replay()
        return self._latent


def main(frames: int = 50, prompt: int = 100):
    """A prompt of codes, then frame by frame to audio with the 24 kHz speech decoder."""
    import torch

    from . import workloads as W
    B = 8
    wl = W.make_workload("speech", T=4, B=1)
    voc = V.Vocoder(wl.arch, V.fold_params(wl.params))
    stream = V.VocoderStream(voc, B, max(prompt, 1))
    front = Front(FrontArch(latent=wl.arch.latent_channels), B, prompt + frames)
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, front.arch.entries, (B, prompt + frames, front.arch.books),
                          generator=g, device="cuda")
    audio = [stream.decode(front.prompt(codes[:, :prompt]))]
    audio.append(stream.decode(front.step(codes[:, prompt])))  # set-up of the graphs
    torch.cuda.synchronize()
    marks = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    ms = [0.0, 0.0]
    for i in range(prompt + 1, prompt + frames):
        marks[0].record()
        latent = front.step(codes[:, i])
        marks[1].record()
        audio.append(stream.decode(latent))
        marks[2].record()
        torch.cuda.synchronize()
        ms[0] += marks[0].elapsed_time(marks[1])
        ms[1] += marks[1].elapsed_time(marks[2])
    audio = torch.cat(audio, 2)
    assert bool(torch.isfinite(audio).all())
    n = max(1, frames - 1)
    print(f"{B} sequences, {prompt} prompt frames and {frames} streamed ones -> "
          f"{tuple(audio.shape)} samples; a streamed frame takes {ms[0] / n:.3f} ms in front of "
          f"the decoder and {ms[1] / n:.3f} ms in it")
    stream.close()
    voc.close()


if __name__ == "__main__":
    main()
