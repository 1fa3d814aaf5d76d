"""rows_as_asked of the prompt example against lists: rows laid out by the counts asked for, some refused."""
import importlib.util
import os
import random

import pytest

torch = pytest.importorskip("torch")

import chunk_reference as ref  # noqa: E402

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "prompt_decode.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("prompt_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("seed", range(40))
def test_rows_as_asked(example, seed):
    rng = random.Random(seed)
    B, page = rng.randint(1, 6), rng.choice([1, 4, 16])
    pool = ref.Pool(B, page, 6, rng.randint(1, 4 * B))
    lens = [rng.choice([0, -1, 0]) for _ in range(B)]
    for _ in range(5):
        counts = [rng.choice([0, 1, -2, rng.randint(0, 3 * page)]) for _ in range(B)]
        T = sum(max(c, 0) for c in counts) + rng.choice([0, 3])
        granted, first, slots, positions, after, _ = pool.reserve(lens, counts, T)
        i32 = dict(dtype=torch.int32)
        got = example.rows_as_asked(torch.tensor(counts, **i32), torch.tensor(granted, **i32),
                                    torch.tensor(first, **i32), torch.tensor(slots, dtype=torch.int64),
                                    torch.tensor(positions, **i32))
        starts, want_slots, want_positions = [0], [], []
        for b in range(B):
            n = max(counts[b], 0)
            have = granted[b] > 0
            mine = slice(first[b], first[b] + n)
            want_slots += slots[mine] if have else [-1] * n
            want_positions += positions[mine] if have else [0] * n
            starts.append(len(want_slots))
        rest = T - len(want_slots)
        assert got[0].tolist() == starts and got[0].dtype == torch.int32
        assert got[1].tolist() == want_slots + [-1] * rest and got[1].dtype == torch.int64
        assert got[2].tolist() == want_positions + [0] * rest and got[2].dtype == torch.int32
        lens = after
