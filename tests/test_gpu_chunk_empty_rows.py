"""GPU tests of PagedAttention.forward_chunk for rows that weigh nothing: every score -inf beside values that are
no numbers, in units of one block and in units that several share."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import test_gpu_chunk as chunk  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("n,m,slots", [(5, 3, [2]),              # a tile that rows attend to in part,
                                       (200, 3, [10]),           # one that all attend to in whole,
                                       (200, 3, [10, 201]),      # both;
                                       (6000, 1, [10, 3000]),    # parts of one unit
                                       (6000, 300, [10, 6000])])
def test_scores_of_minus_infinity_beside_values_without_a_number(n, m, slots, bad, dtype):
    s = chunk.make(1, 1, 64, 16, [n], [m], dtype)
    s["q"].zero_()
    s["q"][..., 0] = -1.0
    s["k"].zero_()
    s["k"][..., 0] = float("inf")
    for j in slots:
        s["v"][s["tables"][0, j // 16].item(), 0, j % 16, 3] = bad
    assert (chunk.run(s) == 0).all()
    s["plan"].check()
