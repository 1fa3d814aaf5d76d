"""GPU test of Rotary with frequencies below zero: as exact at far positions as those above."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import transposed_convolution_gb300 as ctr  # noqa: E402


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_small_frequencies_at_far_positions(sign):
    """Frequencies of about 2^-32 and 2^-40 turn whose last bit is at 2^-54: one less them has no bit there.
    The vector (1, 0) becomes (cos a, sin a).  The angle is off by 2^-32 turn and the rounding of its fp32
    value, 2^-26 turn, together 2^-23.3 radians; sine and cosine by 2^-23, the product by 2^-24."""
    turns = [2.0 ** -32 + 2.0 ** -54, 2.0 ** -33 + 3 * 2.0 ** -54, 2.0 ** -40 + 2.0 ** -54,
             2.0 ** -40 + 5 * 2.0 ** -54]
    f = [sign * 2 * np.pi * t for t in turns]
    pos = np.array([2 ** 31 - 1, -(2 ** 31), 2 ** 31 - 12345, 1 << 30, 7, 0])
    x = torch.zeros(len(pos), 1, 8, device="cuda")
    x[..., :4] = 1.0
    rope = ctr.Rotary(8, frequencies=f, dtype=torch.float32)
    got, _ = rope.forward(x, None, torch.from_numpy(pos.astype(np.int32)).cuda())
    a = pos[:, None] * np.array(f)
    want = np.concatenate([np.cos(a), np.sin(a)], 1)
    off = np.abs(got[:, 0].double().cpu().numpy() - want)
    assert off.max() <= 2 * np.pi * (2.0 ** -32 + 2.0 ** -26) + 2.0 ** -23 + 2.0 ** -24
