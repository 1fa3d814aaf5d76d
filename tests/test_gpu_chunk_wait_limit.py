"""The bounded waits of the 16-bit chunk kernel.  A limit of 0 ns makes them give up on a healthy run: the block
waits for its copies and products in flight, frees its TMEM and returns; ctr_attn_check reports it once, and the
next call is the one that an undisturbed plan makes, to the bit."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import test_gpu_chunk as chunk  # noqa: E402
import transposed_convolution_gb300 as ctr  # noqa: E402

NORMAL = 10_000_000_000

CASES = [  # (D, lens, counts): units of one and two tiles of rows; units cut (the join runs), and whole ones
    (64, [0, 30], [200, 40]), (64, [4000, 7], [300, 90]), (128, [100], [120]), (128, [9000, 500], [300, 40]),
    (256, [0, 30], [200, 40]), (256, [4000, 7], [300, 90])]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,lens,counts", CASES)
def test_waits_that_give_up_are_reported_and_the_next_call_is_right(D, lens, counts, dtype):
    s = chunk.make(8, 2, D, 16, lens, counts, dtype, seed=D)
    want = chunk.run(s)
    chunk.check(s, want)
    s["plan"].check()
    for _ in range(3):
        s["plan"].set_wait_limit_ns(0)
        chunk.run(s)
        with pytest.raises(ctr.CtrError) as e:
            s["plan"].check()
        assert e.value.status == ctr.CTR_ERR_DEVICE_TIMEOUT
        s["plan"].check()
        s["plan"].set_wait_limit_ns(NORMAL)
        assert torch.equal(chunk.run(s), want)
        s["plan"].check()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_waits_that_give_up_at_any_time(D):
    """Limits around the time of a tile, a segment and the call: a call that reports nothing is right, and the
    one after a report too."""
    s = chunk.make(8, 2, D, 16, [9000, 500, 40], [300, 40, 3], "bf16", seed=D)
    want = chunk.run(s)
    for limit in (500, 1000, 2000, 3000, 5000, 8000, 20000, 60000) * 2:
        s["plan"].set_wait_limit_ns(limit)
        got = chunk.run(s)
        try:
            s["plan"].check()
        except ctr.CtrError as e:
            assert e.status == ctr.CTR_ERR_DEVICE_TIMEOUT
        else:
            assert torch.equal(got, want)
        s["plan"].set_wait_limit_ns(NORMAL)
        assert torch.equal(chunk.run(s), want)
        s["plan"].check()
