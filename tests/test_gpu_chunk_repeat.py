"""GPU test of PagedAttention.forward_chunk over random batches that mix units of one and of two tiles of rows,
masked and whole tiles, parts and whole units: each is within its bound of the formula, and repeats are the
same bits."""
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import test_gpu_chunk as chunk  # noqa: E402


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    rng = random.Random(seed)
    dtype = rng.choice(["bf16", "f16", "bf16", "f16", "f32"])
    Hkv, G = rng.choice([1, 2, 3]), rng.choice([1, 2, 3, 4, 8])
    D = rng.choice([64, 80, 128, 256, 16 * rng.randint(1, 16)])
    B = rng.choice([1, 2, 5, 40])
    most = rng.choice([3, 70, 400]) if B > 5 else rng.choice([5, 200, 1500])
    lens = [rng.choice([0, rng.randint(0, most), rng.randint(0, 2 * most), -1]) for _ in range(B)]
    counts = [rng.choice([0, 1, rng.randint(1, 40), rng.randint(1, max(1, most // 4))]) for _ in range(B)]
    window = rng.choice([0, 0, 0, rng.randint(1, most)])
    s = chunk.make(Hkv * G, Hkv, D, rng.choice([1, 8, 16, 20, 64]), lens, counts, dtype,
                   rng.choice(["head", "token"]), seed=seed, peaked=rng.choice([1.0, 4.0]), window=window,
                   before=rng.choice([0, 2]), behind=rng.choice([0, 3]))
    if s["q"].shape[0] == 0:
        return
    out = chunk.run(s)
    chunk.check(s, out)
    for _ in range(30):
        assert torch.equal(chunk.run(s), out)
    s["plan"].check()
