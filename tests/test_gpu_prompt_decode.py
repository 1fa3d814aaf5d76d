"""The example that runs page reservation, rotary positions, chunk attention and the decode step together,
against a 64-bit replay: each stream as a list of codes, all of them attended to anew."""
import importlib.util
import os
import random

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import chunk_reference as ref  # noqa: E402
import oracle  # noqa: E402

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "prompt_decode.py")


def example():
    spec = importlib.util.spec_from_file_location("prompt_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def replay(d, codes):
    """The logits after every one of a stream's codes, in 64 bits."""
    embed, w_qkv, w_out, w_logits = (t.double().cpu().numpy() for t in (d.embed, d.w_qkv, d.w_out, d.w_logits))
    x = embed[codes]
    n, G = len(codes), d.H_q // d.H_kv
    qkv = (x @ w_qkv).reshape(n, -1, d.D)
    f = ref.frequencies(d.D)
    q, _ = ref.rotary(qkv[:, :d.H_q], np.arange(n), f)
    k, _ = ref.rotary(qkv[:, d.H_q:d.H_q + d.H_kv], np.arange(n), f)
    v = qkv[:, d.H_q + d.H_kv:]
    seen = np.zeros((n, d.H_q, d.D))
    hidden = np.triu(np.full((n, n), -np.inf), 1)
    for h in range(d.H_q):
        s = q[:, h] @ k[:, h // G].T / np.sqrt(d.D) + hidden
        p = np.exp(s - s.max(1, keepdims=True))
        seen[:, h] = p @ v[:, h // G] / p.sum(1, keepdims=True)
    return (x + seen.reshape(n, -1) @ w_out) @ w_logits


def test_prompts_drafts_and_steps_follow_the_replay():
    """fp32: logits within 1e-4 of their size (products of 512 columns leave 1e-5 at most)."""
    rng = random.Random(3)
    d = example().PromptDecoder(B=3, vocab=200, page=8, limit=160, num_pages=40, dtype=torch.float32)
    streams = [[] for _ in range(3)]

    def counts(c):
        return torch.tensor(c, dtype=torch.int32, device="cuda")

    def extend(c, granted=None):
        new = [[rng.randrange(200) for _ in range(n)] for n in c]
        codes = torch.tensor(sum((a for a, n in zip(new, c)), []), dtype=torch.int64, device="cuda")
        got, g = d.extend(codes, counts(c))
        assert g.tolist() == (granted or c)
        at = 0
        for b, a in enumerate(new):
            if g[b] == 0:
                continue
            streams[b] += a
            want = replay(d, streams[b])[-len(a):]
            assert oracle.rel_l2(got[at:at + len(a)].cpu().numpy(), want) <= 1e-4
            at += len(a)

    extend([70, 1, 9])                 # prompts
    extend([3, 40, 0])                 # pieces and drafts
    for _ in range(9):
        new = [rng.randrange(200) for _ in range(3)]
        got = d.step(torch.tensor(new, device="cuda")).cpu().numpy()
        for b in range(3):
            streams[b].append(new[b])
            assert oracle.rel_l2(got[b], replay(d, streams[b])[-1]) <= 1e-4
    extend([4, 4, 4])                  # four drafted codes, of which three are taken back
    d.take_back(counts([3, 3, 3]))
    streams = [s[:-3] for s in streams]
    assert d.lens.tolist() == [len(s) for s in streams]
    extend([30, 100, 30], granted=[30, 100, 0])    # the pool has no pages left for the last
    extend([1, 1, 1])
    d.check()
    held = sum(-(-len(s) // 8) for s in streams)
    assert d.pool.count.item() == 40 - held
    d.take_back(d.lens)
    assert d.pool.count.item() == 40 and (d.tables == -1).all() and d.lens.tolist() == [0, 0, 0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_runs_in_16_bits_and_repeats(dtype):
    def run():
        d = example().PromptDecoder(dtype=dtype)
        c = torch.tensor([200, 1, 77], dtype=torch.int32, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(1)
        logits, _ = d.extend(torch.randint(0, 1024, (278,), generator=g, device="cuda"), c)
        out = [logits]
        last = logits[c.cumsum(0) - 1].argmax(-1)
        for _ in range(10):
            out.append(d.step(last))
            last = out[-1].argmax(-1)
        d.check()
        return torch.cat(out)
    a, b = run(), run()
    assert torch.equal(a, b) and a.isfinite().all()


def test_two_captured_graphs_of_one_plan():
    """A prompt's chunk and a piece's, captured with the same plan and workspace, replayed in turn: each
    replay is the call's own result."""
    import transposed_convolution_gb300 as ctr
    k = torch.randn(40, 2, 16, 64, device="cuda").bfloat16()
    plan = ctr.PagedAttention(1, 8, 2, 64, 16, 40, k_pages=k, v_pages=torch.randn_like(k), chunks=True)
    tables = torch.randperm(40, device="cuda").to(torch.int32)[None]
    calls = []
    for n, m in ((0, 500), (500, 3)):
        q = torch.randn(m, 8, 64, device="cuda").bfloat16()
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        starts = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        want = plan.forward_chunk(q, tables, lens, starts)
        graph, out = torch.cuda.CUDAGraph(), torch.zeros_like(want)
        with torch.cuda.graph(graph):
            plan.forward_chunk(q, tables, lens, starts, out=out)
        calls.append((graph, out, want, q, lens, starts))
    for _ in range(3):
        for graph, *_ in calls:
            graph.replay()
        torch.cuda.synchronize()
        for _, out, want, *_ in calls:
            assert torch.equal(out, want)
            out.zero_()
