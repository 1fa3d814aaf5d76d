"""Prompts, drafted codes and single steps on one paged cache, with rotary positions.

B streams of different lengths: ``PagePool.reserve`` takes pages for the new tokens of all of them and
says where each goes; ``PagedAttention.put`` turns the keys by their positions (``Rotary``) on
their way there, and the queries beside them; ``PagedAttention.forward_chunk`` attends, prompts of any lengths
at once, and ``PagedAttention.forward`` does for one token a stream.  A step may be taken back
(``PagePool.release``), as drafted codes are that turn out wrong.  Streams that the pool refuses, or that are
idle, stay as they are beside the others (``rows_as_asked``).  The weights are random: the example shows
the calls, not a model.

    python examples/prompt_decode.py
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import transposed_convolution_gb300 as ctr  # noqa: E402


def rows_as_asked(counts, granted, first, slots, positions):
    """Starts [B + 1], slots and positions of rows that lie as ``counts`` asked for them, from what
    ``PagePool.reserve`` says of the rows that it granted, which follow one another without those that it
    refused.  Refused rows get slot -1 and position 0.  On the GPU, as only it knows who was refused."""
    T = len(slots)
    ends = counts.clamp(min=0).cumsum(0).clamp(max=T)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    row = torch.arange(T, device=slots.device)
    stream = torch.searchsorted(ends, row, right=True).clamp(max=len(counts) - 1)
    has = (granted[stream] > 0) & (row < ends[-1])
    at = (first[stream] + row - starts[stream]).clamp(0, max(T - 1, 0))
    return starts.to(torch.int32), torch.where(has, slots[at], -1), torch.where(has, positions[at], 0)


class PromptDecoder:
    """B streams; codes of a ``vocab``-entry codebook; heads of D columns; room for ``limit`` tokens a
    stream in pages of ``page``, ``num_pages`` of them for all streams."""

    def __init__(self, B=3, vocab=1024, H_q=8, H_kv=2, D=64, page=16, limit=512, num_pages=64,
                 dtype=torch.bfloat16, seed=0):
        self.B, self.vocab, self.H_q, self.H_kv, self.D = B, vocab, H_q, H_kv, D
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            w = torch.randn(shape, generator=g, device="cuda") / shape[0] ** 0.5
            return w.to(dtype)

        width = H_q * D
        self.embed = torch.randn(vocab, width, generator=g, device="cuda").to(dtype)
        self.w_qkv = weight(width, (H_q + 2 * H_kv) * D)
        self.w_out, self.w_logits = weight(width, width), weight(width, vocab)
        pages = -(-limit // page)
        self.attention = ctr.PagedAttention(B, H_q, H_kv, D, page, pages, num_pages=num_pages, dtype=dtype,
                                            chunks=True)
        self.rotary = ctr.Rotary(D, dtype=dtype)
        self.pool = ctr.PagePool(B, page, pages, num_pages)
        self.tables = torch.full((B, pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.granted = None                 # of the last call

    def qkv(self, codes):
        x = self.embed[codes]
        qkv = (x @ self.w_qkv).view(len(codes), self.H_q + 2 * self.H_kv, self.D)
        return (x,) + qkv.split([self.H_q, self.H_kv, self.H_kv], dim=1)

    def logits(self, x, seen):
        return (x + seen.reshape(len(x), -1) @ self.w_out) @ self.w_logits

    def extend(self, codes, counts):
        """codes [T] (int64), of which each stream has the next ``counts`` [B] (int32), to the logits
        [T, vocab] after each of them, and the counts that were granted: all of a stream's, or 0 where the pool
        has no room or the stream is idle.  A refused stream is as it was; its rows are codes that saw nothing."""
        T = len(codes)
        granted, first, slots, positions, lens = self.pool.reserve(self.tables, self.lens, counts, T)
        starts, slots, positions = rows_as_asked(counts, granted, first, slots, positions)
        x, q, k, v = self.qkv(codes)
        q = self.attention.put(k, v, slots, q=q, positions=positions, rotary=self.rotary)
        seen = self.attention.forward_chunk(q, self.tables, torch.where(granted == counts, self.lens, -1),
                                            starts)
        self.lens, self.granted = lens, granted
        return self.logits(x, seen), granted

    def step(self, codes):
        """codes [B], one more for each stream, to the logits [B, vocab], by the decode step's attention.
        ``granted`` [B] then says 0 for a stream that is idle or was refused, as ``extend`` does."""
        ones = torch.ones_like(self.lens)
        granted, first, slots, positions, lens = self.pool.reserve(self.tables, self.lens, ones, self.B)
        _, slots, positions = rows_as_asked(ones, granted, first, slots, positions)
        x, q, k, v = self.qkv(codes)
        q = self.attention.put(k, v, slots, q=q, positions=positions, rotary=self.rotary)
        seen = self.attention.forward(q, self.tables, torch.where(granted > 0, lens, -1))
        self.lens, self.granted = lens, granted
        return self.logits(x, seen)

    def take_back(self, counts):
        """Forget each stream's last ``counts`` [B] tokens."""
        self.lens = self.pool.release(self.tables, self.lens, self.lens - counts)

    def check(self):
        self.attention.check()
        self.pool.check()


if __name__ == "__main__":
    decoder = PromptDecoder()
    counts = torch.tensor([200, 1, 77], dtype=torch.int32, device="cuda")
    codes = torch.randint(0, decoder.vocab, (278,), device="cuda")
    logits, granted = decoder.extend(codes, counts)
    print("prompts", granted.tolist(), "logits", tuple(logits.shape))
    last = logits[counts.cumsum(0) - 1].argmax(-1)
    for _ in range(20):
        last = decoder.step(last).argmax(-1)
    drafted = torch.full((decoder.B,), 4, dtype=torch.int32, device="cuda")
    decoder.extend(torch.randint(0, decoder.vocab, (12,), device="cuda"), drafted)
    decoder.take_back(drafted - 1)
    decoder.check()
    print("lengths", decoder.lens.tolist(), "free pages", decoder.pool.count.item())
    for plan in (decoder.attention, decoder.rotary, decoder.pool):
        print(plan.describe())
