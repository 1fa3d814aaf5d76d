"""GPU test of PagedAttention.forward_chunk: an idle sequence may have any number of rows."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import test_gpu_chunk as chunk  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("idle", [-1, -2 ** 31])
def test_an_idle_sequence_of_more_rows_than_the_cache_has_slots(idle, dtype):
    """160 rows, 80 slots: the rows give 0 and nothing is reported, as no slot is asked for."""
    s = chunk.make(4, 2, 64, 16, [0, 50], [60, 20], dtype, max_pages=5, before=100)
    s["starts"][0] = 0
    s["lens"][0] = idle
    out = chunk.run(s)
    chunk.check(s, out)
    assert (out[:160] == 0).all()
    s["plan"].check()
