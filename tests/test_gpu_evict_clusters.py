"""GPU tests of PagedAttention.evict where several blocks share a (sequence, head) and nothing is
to be chosen: every slot stays, the sinks and recent slots fill the budget, or the row is idle.  The
blocks then pass their counts to one another as soon as they start."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import decode_reference as ref  # noqa: E402
import transposed_convolution_gb300 as ctr  # noqa: E402

# Tables of 8192 and of 16384 slots and up give clusters of 2 and of 4 blocks to few heads.
@pytest.mark.parametrize("Hkv,max_pages", [(1, 32), (1, 128), (9, 64), (24, 32)])
@pytest.mark.parametrize("lens,budget,sinks,recent", [
    ([8191, 3], 8191, 0, 0),          # both under the budget
    ([5000, -1], 300, 100, 200),      # nothing beside the sinks and the recent slots; idle
    ([0, 7000], 6999, 1, 1),          # empty, and one slot to give up
])
def test_nothing_to_choose(Hkv, max_pages, lens, budget, sinks, recent):
    page, D, B = 256, 16, 2
    g = torch.Generator(device="cuda").manual_seed(Hkv + budget)
    most, to_pages = -(-max(lens) // page), -(-budget // page)
    total = B * (most + to_pages)
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    tables = torch.full((B, max_pages), 2 ** 30, dtype=torch.int32, device="cuda")
    tables[:, :most] = perm[:B * most].view(B, most)
    to = perm[B * most:].view(B, to_pages).contiguous()
    k, v = (torch.randn(total, Hkv, page, D, generator=g, device="cuda") for _ in range(2))
    plan = ctr.PagedAttention(B, Hkv, Hkv, D, page, max_pages, k_pages=k, v_pages=v)
    w = torch.rand(B, Hkv, plan.capacity, generator=g, device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    got = [plan.evict(tables, n, w, to, budget, sinks, recent) for _ in range(30)]
    plan.check()
    for slots, lens_out, w_out in got:
        assert lens_out.tolist() == [min(x, budget) for x in lens]
        assert torch.equal(slots, got[0][0]) and torch.equal(w_out, got[0][2])
    slots = got[0][0]
    for b in range(B):
        for h in range(Hkv):
            keep = ref.evict(w[b, h].cpu().numpy(), max(lens[b], 0), budget, sinks, recent)
            assert slots[b, h, :len(keep)].tolist() == keep
            assert (slots[b, h, len(keep):] == -1).all()
            j = torch.tensor(keep, dtype=torch.int64, device="cuda")
            i = torch.arange(len(keep), device="cuda")
            src, dst = tables[b].long()[j // page], to[b].long()[i // page]
            for x in (k, v):
                assert torch.equal(x[dst, h, i % page], x[src, h, j % page])
