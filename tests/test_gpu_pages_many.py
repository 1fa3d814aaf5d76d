"""GPU tests of PagePool where both kernels have many blocks: as many as 147 of them reserve, 8 of them give
back, and the last to finish writes the list's count."""
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import test_gpu_pages as pages  # noqa: E402


@pytest.mark.parametrize("B,page,max_pages,num_pages", [
    (1024, 4, 64, 60000), (300, 1, 200, 50000), (2, 16, 20000, 40000), (64, 3, 400, 17000)])
def test_random_steps(B, page, max_pages, num_pages):
    rng = random.Random(num_pages)
    s = pages.Both(B, page, max_pages, num_pages)
    share = page * max_pages * 6 // 10
    most = 0
    for step in range(3):
        counts = [rng.choice([share, rng.randint(0, share)]) if n < share else rng.randint(0, page)
                  for n in s.lens]
        s.reserve(counts, min(sum(counts) + 3, 200000))
        before = len(s.sim.free)
        # Every other time all of them, idle sequences starting anew.
        s.release([-1 if step % 2 else rng.choice([-1, 0, n // 2, n]) for n in s.lens])
        most = max(most, len(s.sim.free) - before)
        s.lens = [max(n, 0) for n in s.lens]
    assert most > 8192
