"""GPU test of two pools that share one free list, of different numbers of sequences, pages of one size."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import transposed_convolution_gb300 as ctr  # noqa: E402


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_two_pools_take_from_one_list():
    a = ctr.PagePool(2, 4, 8, 10)
    b = ctr.PagePool(3, 4, 5, free=a.free, count=a.count)
    assert b.count.item() == 10                       # not filled anew
    ta, tb = i32([[-1] * 8] * 2), i32([[-1] * 5] * 3)
    assert a.reserve(ta, i32([0, 0]), i32([9, 4]), 20)[0].tolist() == [9, 4]
    assert b.reserve(tb, i32([0, 0, 0]), i32([4, 17, 5]), 30)[0].tolist() == [4, 17, 0]
    assert a.count is b.count and a.count.item() == 0
    held = [p for t in (ta, tb) for row in t.tolist() for p in row if p >= 0]
    assert sorted(held) == list(range(10))
    assert a.release(ta, i32([9, 4]), i32([-1, 1])).tolist() == [-1, 1]
    assert b.count.item() == 3
    assert b.reserve(tb, i32([4, 17, 0]), i32([0, 0, 5]), 30)[0].tolist() == [0, 0, 5]
    a.check()
    b.check()
    # The list on the host and back: a third pool goes on from it.
    c = ctr.PagePool(1, 4, 3, free=a.free.cpu().cuda(), count=a.count.cpu().cuda())
    assert c.reserve(i32([[-1] * 3]), i32([0]), i32([8]), 8)[0].tolist() == [0]
    assert c.reserve(i32([[-1] * 3]), i32([0]), i32([4]), 8)[0].tolist() == [4] and c.count.item() == 0
    c.check()
