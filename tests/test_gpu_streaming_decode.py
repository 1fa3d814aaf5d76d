"""The example that runs attention, eviction, sampling and the streaming upsampler together, against
a 64-bit replay of its steps: the cache as lists of rows, evictions by the replay's own weights."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import decode_reference as ref  # noqa: E402
import oracle  # noqa: E402

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "streaming_decode.py")


def example():
    spec = importlib.util.spec_from_file_location("streaming_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_steps_follow_the_replay():
    """150 steps with evictions at every 64 slots, in fp32: codes, evicted slots and audio."""
    d = example().StreamingDecoder(B=2, vocab=300, limit=64, budget=40, dtype=torch.float32)
    evicted = []
    keep = d.evict
    d.evict = lambda: evicted.append(keep().cpu().numpy())
    codes, audio = d.run(150)
    codes, audio = codes.cpu().numpy(), audio.cpu().numpy()
    assert len(evicted) == 4

    def f64(t):
        return t.double().cpu().numpy()
    embed, w_qkv, w_out, w_logits = (f64(t) for t in (d.embed, d.w_qkv, d.w_out, d.w_logits))
    G = d.H_q // d.H_kv
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = [[dict(k=[], v=[], w=[]) for _ in range(d.H_kv)] for _ in range(d.B)]
    last, rounds = np.zeros(d.B, int), 0
    for step in range(150):
        noise = torch.empty(d.B, d.vocab, device="cuda").exponential_(generator=g).cpu().numpy()
        if len(cache[0][0]["w"]) == d.limit:
            for b in range(d.B):
                for h in range(d.H_kv):
                    c = cache[b][h]
                    slots = ref.evict(np.asarray(c["w"]), d.limit, d.budget, d.sinks, d.recent)
                    assert evicted[rounds][b, h].tolist() == slots
                    for a in c:
                        c[a] = [c[a][j] for j in slots]
            rounds += 1
        for b in range(d.B):
            x = embed[last[b]]
            qkv = (x @ w_qkv).reshape(-1, d.D)
            seen = np.zeros((d.H_q, d.D))
            for h in range(d.H_kv):
                c = cache[b][h]
                c["k"].append(qkv[d.H_q + h])
                c["v"].append(qkv[d.H_q + d.H_kv + h])
                c["w"].append(0.0)
                s = qkv[h * G:(h + 1) * G] @ np.stack(c["k"]).T / np.sqrt(d.D)
                p = np.exp(s - s.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                seen[h * G:(h + 1) * G] = p @ np.stack(c["v"])
                c["w"] = list(np.asarray(c["w"]) + p.sum(0))
            logits = (x + seen.reshape(-1) @ w_out) @ w_logits
            # fp32 products over 512 columns leave relative errors of 1e-5 at most.
            want = ref.sample(logits, noise[b], 0.9, 250, 0.95, 0.01, slack=1e-3)
            assert codes[b, step] in want
        last = codes[:, step]
    # The audio is the unpadded transposed convolution of all frames, cut to the samples emitted.
    x = d.frames.cpu().numpy()[codes].transpose(0, 2, 1)
    stride = d.w_up.shape[2] // 2
    want = oracle.conv_transpose(x, d.w_up.cpu().numpy(), None, stride, 0, 0)[:, :, :150 * stride]
    assert oracle.rel_l2(audio, want) <= 1e-5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_runs_in_16_bits_and_repeats(dtype):
    module = example()
    a = module.StreamingDecoder(dtype=dtype).run(100)
    b = module.StreamingDecoder(dtype=dtype).run(100)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert a[0].min() >= 0 and a[0].max() < 1024 and torch.isfinite(a[1]).all()
