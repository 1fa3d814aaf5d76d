"""The example of prompts, drafts and steps where the pool refuses a stream that others follow, and where a stream
is idle: the other streams' logits are those of a 64-bit replay, and nothing of the refused one is kept."""
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import oracle  # noqa: E402
import test_gpu_prompt_decode as base  # noqa: E402
import transposed_convolution_gb300 as ctr  # noqa: E402


class Streams:
    """The example in fp32 and each stream's codes as a list; logits within 1e-4 of their size."""

    def __init__(self, num_pages, limit=160):
        self.d = base.example().PromptDecoder(B=3, vocab=200, page=8, limit=limit, num_pages=num_pages,
                                              dtype=torch.float32)
        self.codes, self.rng = [[], [], []], random.Random(5)

    def new(self, counts):
        return [[self.rng.randrange(200) for _ in range(n)] for n in counts]

    def compare(self, got, new, granted):
        at = 0
        for b, a in enumerate(new):
            if granted[b]:
                self.codes[b] += a
                want = base.replay(self.d, self.codes[b])[-len(a):]
                assert oracle.rel_l2(got[at:at + len(a)].cpu().numpy(), want) <= 1e-4
            at += len(a)

    def extend(self, counts, granted):
        new = self.new(counts)
        codes = torch.tensor(sum(new, []), dtype=torch.int64, device="cuda")
        got, g = self.d.extend(codes, torch.tensor(counts, dtype=torch.int32, device="cuda"))
        assert g.tolist() == granted and got.shape[0] == sum(counts)
        self.compare(got, new, granted)

    def step(self, granted):
        new = self.new([1, 1, 1])
        got = self.d.step(torch.tensor(sum(new, []), device="cuda"))
        self.compare(got, new, granted)
        assert self.d.granted.tolist() == granted

    def idle(self, b):
        """Give back all of a stream."""
        keep = self.d.lens.clone()
        keep[b] = -1
        self.d.lens = self.d.pool.release(self.d.tables, self.d.lens, keep)
        self.codes[b] = []
        assert self.d.lens[b] == -1


def test_the_first_stream_is_refused_a_chunk():
    s = Streams(num_pages=6)
    s.extend([16, 5, 5], [16, 5, 5])
    s.extend([30, 1, 2], [0, 1, 2])
    s.extend([1, 40, 1], [1, 0, 1])
    s.extend([2, 0, 900], [2, 0, 0])            # more than a stream's table holds: the pool reports it
    with pytest.raises(ctr.CtrError):
        s.d.pool.check()
    s.extend([1, 1, 1], [1, 1, 1])
    assert s.d.lens.tolist() == [len(c) for c in s.codes]
    s.d.check()


def test_the_first_stream_is_refused_a_step():
    s = Streams(num_pages=4)
    s.extend([16, 5, 5], [16, 5, 5])
    for _ in range(2):
        s.step([0, 1, 1])
    assert s.d.lens.tolist() == [16, 7, 7]
    s.idle(1)
    s.step([1, 0, 1])
    s.step([1, 0, 0])                           # 2 has filled its page
    s.extend([2, 3, 0], [2, 0, 0])
    assert s.d.lens.tolist() == [20, -1, 8]
    s.d.check()


def test_an_idle_stream_between_others():
    s = Streams(num_pages=40)
    s.extend([20, 30, 10], [20, 30, 10])
    s.idle(1)
    s.extend([5, 200, 9], [5, 0, 9])            # more rows than the stream could have
    for _ in range(3):
        s.step([1, 0, 1])
    s.idle(0)
    s.extend([4, 4, 4], [0, 0, 4])
    s.step([0, 0, 1])
    s.d.check()
