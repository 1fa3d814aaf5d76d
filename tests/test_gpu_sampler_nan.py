"""GPU tests of Sampler with filters that are no number or infinite: by the formula's comparisons a NaN
top-p or min-p filters nothing, and a NaN temperature takes the first token."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import decode_reference as ref  # noqa: E402
import transposed_convolution_gb300 as ctr  # noqa: E402

NAN, INF = float("nan"), float("inf")
# What is given, and what it is the same as.
SAME = [
    ((1.0, 0, 1.0, NAN), (1.0, 0, 1.0, 0.0)), ((1.0, 0, 0.9, NAN), (1.0, 0, 0.9, 0.0)),
    ((0.7, 20, 1.0, NAN), (0.7, 20, 1.0, 0.0)), ((1.0, 0, NAN, 0.0), (1.0, 0, 1.0, 0.0)),
    ((1.0, 30, NAN, 0.05), (1.0, 30, 1.0, 0.05)), ((0.8, 5, NAN, NAN), (0.8, 5, 1.0, 0.0)),
    ((NAN, 0, 0.9, NAN), (0.0, 0, 0.9, 0.0)), ((NAN, 7, NAN, 0.1), (0.0, 7, 1.0, 0.1)),
    ((1.0, 0, INF, -INF), (1.0, 0, 1.0, 0.0)), ((1.0, 0, -INF, 0.0), (0.0, 0, 1.0, 0.0)),
    ((1.0, 9, 0.9, INF), (0.0, 0, 1.0, 0.0)), ((-INF, 0, 1.0, NAN), (0.0, 0, 1.0, 0.0)),
    ((INF, 0, 1.0, 0.0), (1e30, 0, 1.0, 0.0)), ((INF, 100, 0.5, 0.0), (1e30, 100, 0.5, 0.0)),
    ((INF, 100, 0.9, NAN), (1e30, 100, 0.9, 0.0)), ((INF, 0, 0.5, 0.1), (1e30, 0, 0.5, 0.0)),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 3, 1000, 9001, 70001])
def test_filters_that_are_no_number(V, dtype):
    g = torch.Generator(device="cuda").manual_seed(V)
    rows = len(SAME)
    x = (torch.randn(rows, V, generator=g, device="cuda") * 3).to(dtype)
    x[:, V // 2:V // 2 + V // 8] = -INF
    noise = torch.empty(rows, V, device="cuda").exponential_(generator=g)
    kinds = (torch.float32, torch.int32, torch.float32, torch.float32)
    columns = [torch.tensor(c, dtype=d, device="cuda") for c, d in zip(zip(*(a for a, _ in SAME)), kinds)]
    got = ctr.Sampler(rows, V, dtype=dtype).forward(x, noise, *columns).tolist()
    l, e = x.float().cpu().numpy(), noise.cpu().numpy()
    for i, (given, (T, k, p, min_p)) in enumerate(SAME):
        want = ref.sample(l[i], e[i], float(np.float32(T)), k, float(np.float32(p)), float(np.float32(min_p)))
        assert got[i] in want, (i, given, got[i], want)
