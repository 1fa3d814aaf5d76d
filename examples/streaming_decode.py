"""Codes to audio, frame by frame: a one-layer model writes one code a step for each of B streams,
and a streaming transposed convolution turns every frame into samples at once.

A step runs ``PagedAttention.forward`` (the new token's attention over the paged cache, which puts
its key and value there and accumulates every slot's attention weight), ``Sampler`` (the next code
from the logits and given random numbers) and a streaming ``Plan`` (the frame's samples).  When a
stream's cache has grown to its limit, ``PagedAttention.evict`` keeps the heaviest slots and moves
them to the cache's other half.  The weights are random: the example shows the calls, not a model.

    python examples/streaming_decode.py
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import transposed_convolution_gb300 as ctr  # noqa: E402


class StreamingDecoder:
    """B streams; codes of a ``vocab``-entry codebook; heads of D columns; a cache of at most
    ``limit`` slots a stream, of which an eviction keeps ``budget``."""

    def __init__(self, B=2, vocab=1024, H_q=8, H_kv=2, D=64, page=16, limit=64, budget=48, sinks=2,
                 recent=16, channels=64, samples=8, dtype=torch.bfloat16, seed=0):
        self.B, self.vocab, self.H_q, self.H_kv, self.D = B, vocab, H_q, H_kv, D
        self.limit, self.budget, self.sinks, self.recent = limit, budget, sinks, recent
        self.channels = channels
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            w = torch.randn(shape, generator=g, device="cuda") / shape[0] ** 0.5
            return w.to(dtype)

        width = H_q * D
        self.embed = torch.randn(vocab, width, generator=g, device="cuda").to(dtype)
        self.w_qkv = weight(width, (H_q + 2 * H_kv) * D)
        self.w_out, self.w_logits = weight(width, width), weight(width, vocab)
        self.frames = torch.randn(vocab, channels, generator=g, device="cuda")

        # The cache: each stream has as many pages as its limit needs, twice: an eviction moves the
        # kept slots from one half to the other.
        pages = -(-limit // page)
        self.attention = ctr.PagedAttention(B, H_q, H_kv, D, page, pages, num_pages=2 * B * pages,
                                            dtype=dtype, weights=True)
        halves = torch.arange(2 * B * pages, dtype=torch.int32, device="cuda").view(2, B, pages)
        self.tables, self.spare = halves[0].contiguous(), halves[1].contiguous()
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.weights = torch.zeros(B, H_kv, self.attention.capacity, device="cuda")
        self.length = 0                        # the streams of this example run in step

        self.sampler = ctr.Sampler(B, vocab, dtype=dtype)
        self.temperature = torch.full((B,), 0.9, device="cuda")
        self.top_k = torch.full((B,), 250, dtype=torch.int32, device="cuda")
        self.top_p = torch.full((B,), 0.95, device="cuda")
        self.min_p = torch.full((B,), 0.01, device="cuda")

        # One frame a step in, `samples` samples out.
        self.upsampler = ctr.Plan(B, channels, 1, (1,), (2 * samples,), samples, streaming=True,
                                  path=ctr.CTR_PATH_POLYPHASE)
        self.w_up = torch.randn(channels, 1, 2 * samples, generator=g, device="cuda") / channels ** 0.5
        self.upsampler.prepack(self.w_up)

    def evict(self):
        """Keep ``budget`` slots of every stream and head, in the cache's other half."""
        kept = torch.zeros_like(self.weights)
        slots, self.lens, self.weights = self.attention.evict(
            self.tables, self.lens, self.weights, self.spare, self.budget, self.sinks, self.recent,
            weights_out=kept)
        self.tables, self.spare = self.spare, self.tables
        self.length = min(self.length, self.budget)
        return slots

    def step(self, codes, noise):
        """codes [B] and Exp(1) numbers [B, vocab] to the next codes [B] and this frame's samples
        [B, 1, samples]."""
        if self.length == self.limit:
            self.evict()
        x = self.embed[codes]
        qkv = (x @ self.w_qkv).view(self.B, self.H_q + 2 * self.H_kv, self.D)
        q, k, v = qkv.split([self.H_q, self.H_kv, self.H_kv], dim=1)
        seen = self.attention.forward(q, self.tables, self.lens, k, v, weights=self.weights)
        self.lens += 1
        self.length += 1
        logits = (x + seen.view(self.B, -1) @ self.w_out) @ self.w_logits
        codes = self.sampler.forward(logits, noise, self.temperature, self.top_k, self.top_p,
                                     self.min_p)
        audio = self.upsampler.forward(self.frames[codes].view(self.B, self.channels, 1))
        return codes, audio

    def run(self, steps, seed=1):
        """Codes [B, steps] and audio [B, 1, steps * samples] of ``steps`` frames from code 0."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        codes = torch.zeros(self.B, dtype=torch.int64, device="cuda")
        all_codes, audio = [], []
        for _ in range(steps):
            noise = torch.empty(self.B, self.vocab, device="cuda").exponential_(generator=g)
            codes, samples = self.step(codes, noise)
            all_codes.append(codes)
            audio.append(samples)
        self.attention.check()
        self.upsampler.check()
        return torch.stack(all_codes, 1), torch.cat(audio, 2)


if __name__ == "__main__":
    decoder = StreamingDecoder()
    codes, audio = decoder.run(200)
    print("codes", tuple(codes.shape), codes[0, :10].tolist())
    print("audio", tuple(audio.shape), "rms %.3f" % audio.square().mean().sqrt().item())
    print(decoder.attention.describe())
    print(decoder.sampler.describe())
    print(decoder.upsampler.describe())
