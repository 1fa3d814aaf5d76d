"""GPU tests of the decode step's classes on a stream other than the current one: what a call makes for
itself has to be in order on that stream."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import transposed_convolution_gb300 as ctr  # noqa: E402


def test_evict_default_outputs_on_another_stream():
    """The current stream is busy when the call is made, and the side stream is not: the call's own
    weights_out must not be cleared after the kernels have filled it."""
    k = torch.randn(8, 2, 16, 64, device="cuda")
    plan = ctr.PagedAttention(1, 4, 2, 64, 16, 4, k_pages=k, v_pages=k.clone())
    tables = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    to = tables + 4
    lens = torch.tensor([60], dtype=torch.int32, device="cuda")
    w = torch.rand(1, 2, 64, device="cuda") + 1.0
    want = plan.evict(tables, lens, w, to, 32)
    torch.cuda._sleep(1000)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)            # about 30 ms of the current stream
    got = plan.evict(tables, lens, w, to, 32, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # Where fewer slots than the budget are kept, the rest of weights_out is 0.
    lens[0] = 10
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    _, n, kept = plan.evict(tables, lens, w, to, 32, stream=side)
    torch.cuda.synchronize()
    assert n.tolist() == [10]
    assert torch.equal(kept[:, :, :10], w[:, :, :10]) and not kept[:, :, 10:].any()
