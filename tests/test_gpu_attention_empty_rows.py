"""GPU test of PagedAttention.forward: a head whose scores are all -inf gives 0, infinities and NaN in V included, by
one block and where several share the sequence."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import test_gpu_chunk as chunk  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("G", [1, 4, 12])
@pytest.mark.parametrize("n,slots", [(8, [2]), (203, [10]), (200, [10, 199]), (6001, [10, 3000, 6000])])
def test_scores_of_minus_infinity_beside_values_without_a_number(n, slots, G, bad, dtype):
    s = chunk.make(2 * G, 2, 64, 16, [n], [1], dtype)
    s["q"].zero_()
    s["q"][:, G:, 0] = -1.0                        # the first KV head's scores stay 0 or NaN
    s["k"].zero_()
    s["k"][:, 1, :, 0] = float("inf")
    for j in slots:
        s["v"][s["tables"][0, j // 16].item(), 1, j % 16, 3] = bad
    out = s["plan"].forward(s["q"], s["tables"], s["lens"] + 1)
    assert (out[:, G:] == 0).all() and out[:, :G].isfinite().all()
    s["plan"].check()
