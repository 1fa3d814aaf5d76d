"""GPU tests of Sampler rows that several blocks share, call after call without a pause: blocks of a
cluster that start at different times and end at different times.  The tokens are compared with
the 64-bit form, as in test_gpu_sampler.py."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import decode_reference as ref  # noqa: E402
import transposed_convolution_gb300 as ctr  # noqa: E402

SHAPES = [(1, 150001), (19, 70001), (40, 20001), (152, 9000)]     # clusters of 8, 8, 4 and 2 blocks
CALLS = 40


def columns(filters):
    kinds = (torch.float32, torch.int32, torch.float32, torch.float32)
    return [torch.tensor(c, dtype=d, device="cuda") for c, d in zip(zip(*filters), kinds)]


def run(rows, V, some, seed):
    """CALLS calls in a row on inputs of their own; every token has to be the formula's."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    filters = [some[i % len(some)] for i in range(rows)]
    logits = torch.randn(rows, V, generator=g, device="cuda") * 3
    noise = torch.empty(rows, V, device="cuda").exponential_(generator=g)
    # Four inputs of the same numbers in other places: other tokens for each.
    inputs = [(logits.roll(a, 1), noise.roll(a, 1)) for a in (0, 7919, 4001, 63)]
    f = columns(filters)
    plan = ctr.Sampler(rows, V)
    torch.cuda.synchronize()
    got = [plan.forward(*inputs[i % 4], *f) for i in range(CALLS)]
    got = torch.stack(got).cpu().numpy()
    for j, (x, e) in enumerate(inputs):
        x, e = x.cpu().numpy(), e.cpu().numpy()
        for r, (T, k, p, min_p) in enumerate(filters):
            want = ref.sample(x[r], e[r], float(np.float32(T)), k, float(np.float32(p)),
                              float(np.float32(min_p)))
            assert {int(v) for v in got[j::4, r]} <= want, (j, r, filters[r])
        assert (got[j::4] == got[j]).all()


@pytest.mark.parametrize("rows,V", SHAPES)
def test_unfiltered_and_greedy(rows, V):
    """Each block passes its maximum to its peers as soon as it has it, and its best token to the first."""
    run(rows, V, [(1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (0.7, 0, 1.0, 0.0), (1.0, 1, 0.5, 0.0)], V)


@pytest.mark.parametrize("rows,V", SHAPES)
def test_listed_rows(rows, V):
    """The first block has the list and decides alone, with little to do (min-p alone, small top-k)
    while its peers still read its totals; rows that all blocks search lie in between."""
    run(rows, V, [(1.0, 0, 1.0, 0.3), (0.7, 50, 0.95, 0.02), (0.5, 5, 1.0, 0.0), (1.3, 0, 0.95, 0.0),
                  (0.6, 0, 0.5, 0.5), (1.0, 0, 0.9, 0.05)], V + 1)
