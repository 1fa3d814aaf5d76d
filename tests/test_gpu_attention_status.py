"""GPU tests of what PagedAttention.check reports: a length past the capacity, wherever in the batch
it is."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import transposed_convolution_gb300 as ctr  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new", [True, False])
@pytest.mark.parametrize("B,at,max_pages", [(2, 1, 3), (3, 1, 3), (130, 129, 3), (300, 150, 3), (1000, 999, 3),
                                            (5, 3, 40)])
def test_a_length_past_the_capacity_anywhere(B, at, max_pages, new, dtype):
    """Sequence ``at`` alone is full (or, without a new row, longer than its table)."""
    page, cap = 16, 16 * max_pages
    g = torch.Generator(device="cuda").manual_seed(B)
    k, v = (torch.randn(max_pages + B, 1, page, 64, generator=g, device="cuda").to(dtype) for _ in range(2))
    plan = ctr.PagedAttention(B, 2, 1, 64, page, max_pages, k_pages=k, v_pages=v)
    tables = torch.full((B, max_pages), 2 ** 30, dtype=torch.int32, device="cuda")
    tables[:, 0] = torch.arange(max_pages, max_pages + B, dtype=torch.int32, device="cuda")
    tables[at] = torch.arange(max_pages, dtype=torch.int32, device="cuda")
    q = torch.randn(B, 2, 64, generator=g, device="cuda").to(dtype)
    fresh = [torch.randn(B, 1, 64, generator=g, device="cuda").to(dtype) for _ in range(2)] if new else []
    lens = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    plan.forward(q, tables, lens, *fresh)
    plan.check()                                # nothing to report
    lens[at] = cap - 1 if new else cap
    plan.forward(q, tables, lens, *fresh)
    plan.check()                                # just room enough
    before = k[:max_pages].clone()
    for n in (cap if new else cap + 1, 2 ** 31 - 1):
        lens[at] = n
        plan.forward(q, tables, lens, *fresh)
        with pytest.raises(ctr.CtrError) as e:
            plan.check()
        assert e.value.status == ctr.CTR_ERR_INVALID_ARG
        plan.check()                            # cleared
    assert torch.equal(k[:max_pages], before)   # no row was put in the full sequence
