"""GPU tests of PagedAttention.evict: the kept slots, lengths, weights and rows have to equal the
formula's exactly."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import decode_reference as ref  # noqa: E402
import transposed_convolution_gb300 as ctr  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def run(lens, Hkv, D, page, budget, sinks=0, recent=0, dtype="bf16", layout="head", w=None, seed=0,
        spare=0):
    """Evict on a random cache and compare everything with the formula."""
    B = len(lens)
    g = torch.Generator().manual_seed(seed)
    most = max(1, -(-max(max(lens), 1) // page)) + spare
    to_pages = -(-budget // page) + spare
    total = B * (most + to_pages)
    perm = torch.randperm(total, generator=g).to(torch.int32)
    tables, to = perm[:B * most].view(B, most), perm[B * most:].view(B, to_pages)
    shape = (total, Hkv, page, D) if layout == "head" else (total, page, Hkv, D)
    k, v = (torch.randn(shape, generator=g).to(DT[dtype]).cuda() for _ in range(2))
    if w is None:
        w = torch.empty(B, Hkv, most * page).exponential_(generator=g) ** 2
    k0, v0 = k.clone(), v.clone()
    plan = ctr.PagedAttention(B, Hkv, Hkv, D, page, most, k_pages=k, v_pages=v, layout=layout)
    w_out = torch.full((B, Hkv, budget + 3), 9.0, device="cuda")
    slots, n, got_w = plan.evict(tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                 w.cuda(), to.cuda(), budget, sinks, recent, weights_out=w_out)
    plan.check()
    assert got_w is w_out
    assert n.tolist() == [x if x < 0 else min(x, budget) for x in lens]
    slots, w_out = slots.cpu().numpy(), w_out.cpu().numpy()
    for b in range(B):
        for h in range(Hkv):
            keep = ref.evict(w[b, h].numpy(), max(lens[b], 0), budget, sinks, recent)
            m = len(keep)
            assert slots[b, h, :m].tolist() == keep
            assert (slots[b, h, m:] == -1).all()
            np.testing.assert_array_equal(w_out[b, h, :m], w[b, h].numpy()[keep])
            assert (w_out[b, h, m:] == 9.0).all()
            j, i = np.asarray(keep, int), np.arange(m)
            src, dst = tables[b].numpy()[j // page], to[b].numpy()[i // page]
            for x, x0 in ((k, k0), (v, v0)):
                if layout == "head":
                    x0[dst, h, i % page] = x0[src, h, j % page]
                else:
                    x0[dst, i % page, h] = x0[src, j % page, h]
    # All that was to be copied has been, and nothing else has changed.
    assert torch.equal(k, k0) and torch.equal(v, v0)


@pytest.mark.parametrize("dtype,layout", [("bf16", "head"), ("f16", "token"), ("f32", "token")])
@pytest.mark.parametrize("lens,Hkv,D,page,budget,sinks,recent", [
    ([100], 2, 64, 16, 32, 4, 8),
    ([0, 1, 31, 32, 33, -1], 1, 16, 16, 32, 0, 0),           # at, under and over the budget; idle
    ([500, 77, 1200], 4, 80, 24, 300, 4, 100),
    ([5000, 4999], 2, 128, 64, 4096, 0, 256),
    ([40], 3, 64, 8, 1, 0, 0),                               # a budget of one
    ([40], 1, 64, 8, 1, 1, 0),
    ([50, 20], 2, 64, 8, 10, 4, 6),                          # sinks and recent fill the budget
    ([33000], 2, 32, 128, 1000, 8, 128),                     # long, few kept
    ([2049, 1025], 2, 256, 1, 1024, 3, 5),                   # pages of one row
])
def test_random_weights(lens, Hkv, D, page, budget, sinks, recent, dtype, layout):
    run(lens, Hkv, D, page, budget, sinks, recent, dtype, layout, seed=budget)


@pytest.mark.parametrize("kind", ["equal", "few values", "nan", "inf", "negative", "denormal",
                                  "ascending", "descending"])
def test_ties_and_odd_weights(kind):
    g = torch.Generator().manual_seed(2)
    n, cap = 1500, 1504
    w = torch.rand(1, 2, cap, generator=g)
    if kind == "equal":
        w[:] = 0.25
    elif kind == "few values":
        w = torch.randint(0, 4, (1, 2, cap), generator=g).float() - 1
        w[w == 0] = -0.0
        w[0, 0, ::7] = 0.0              # -0 and +0 are equal
    elif kind == "nan":
        w[w < 0.5] = float("nan")
        w[0, 1, 10:20] = -float("inf")  # still above NaN
    elif kind == "inf":
        w[w > 0.9] = float("inf")
    elif kind == "negative":
        w = -w
    elif kind == "denormal":
        w = w * 1e-42
    elif kind == "ascending":
        w = torch.arange(cap).float().expand(1, 2, cap).contiguous()
    elif kind == "descending":
        w = -torch.arange(cap).float().expand(1, 2, cap).contiguous()
    for budget, sinks, recent in ((700, 0, 0), (1400, 10, 300), (20, 4, 8)):
        run([n], 2, 16, 16, budget, sinks, recent, "f16", "head", w=w.clone())


@pytest.mark.parametrize("kind", ["random", "equal", "few values", "heavy end"])
@pytest.mark.parametrize("lens,cap_pages", [([20000], 0), ([8192, 100], 0), ([16385, -1], 40),
                                            ([50000], 0), ([170000], 0)])
def test_few_long_sequences(lens, cap_pages, kind):
    """Several blocks a head, whose parts the ties cross, and parts that do not fit shared memory."""
    g = torch.Generator().manual_seed(7)
    page = 256
    cap = (-(-max(lens) // page) + cap_pages) * page
    w = torch.rand(len(lens), 1, cap, generator=g)
    if kind == "equal":
        w[:] = 1.0
    elif kind == "few values":
        w = torch.randint(0, 3, w.shape, generator=g).float()
    elif kind == "heavy end":
        w[:, :, max(lens) // 2:] += 1.0
    for budget, sinks, recent in ((3000, 5, 70), (7, 0, 0)):
        run(lens, 1, 16, page, budget, sinks, recent, "f16", "head", w=w, spare=cap_pages)


def test_wider_tables_and_default_outputs():
    run([300, 200], 2, 64, 16, 100, 2, 20, spare=3)
    k = torch.randn(8, 2, 16, 64).cuda()
    plan = ctr.PagedAttention(1, 4, 2, 64, 16, 4, k_pages=k, v_pages=k.clone())
    tables = torch.arange(4, dtype=torch.int32).cuda()[None]
    lens = torch.tensor([60], dtype=torch.int32).cuda()
    w = torch.rand(1, 2, 64).cuda()
    slots, n, w_out = plan.evict(tables, lens, w, tables + 4, 32)
    assert slots.shape == (1, 2, 32) and n.tolist() == [32] and w_out.shape == (1, 2, 32)
    assert torch.equal(w_out, w.gather(2, slots.long()))


def test_bad_pages_are_reported():
    k = torch.randn(8, 2, 16, 64).cuda()
    plan = ctr.PagedAttention(1, 4, 2, 64, 16, 4, k_pages=k, v_pages=k.clone())
    tables = torch.arange(4, dtype=torch.int32).cuda()[None]
    lens = torch.tensor([60], dtype=torch.int32).cuda()
    w = torch.rand(1, 2, 64).cuda()
    before = k.clone()
    for bad in (8, -1, 2 ** 31 - 1):
        to = torch.tensor([[5, bad]], dtype=torch.int32).cuda()
        plan.evict(tables, lens, w, to, 32)
        with pytest.raises(ctr.CtrError):
            plan.check()
        keep = [i for i in range(8) if i != 5]
        assert torch.equal(k[keep], before[keep])
    src = tables.clone()
    src[0, 2] = 77
    plan.evict(src, lens, w, tables + 4, 60)
    with pytest.raises(ctr.CtrError):
        plan.check()
    assert torch.equal(k[4], before[0]) and torch.equal(k[6], before[6])
    plan.evict(tables, torch.tensor([1000], dtype=torch.int32).cuda(), w, tables + 4, 64)
    with pytest.raises(ctr.CtrError):
        plan.check()                  # cut to the table's 64 slots
    assert torch.equal(k[4:], before[:4])


def test_refusals():
    k = torch.randn(8, 2, 16, 64).cuda()
    plan = ctr.PagedAttention(1, 4, 2, 64, 16, 4, k_pages=k, v_pages=k.clone())
    tables = torch.arange(4, dtype=torch.int32).cuda()[None]
    lens = torch.tensor([60], dtype=torch.int32).cuda()
    w = torch.rand(1, 2, 64).cuda()
    for budget, sinks, recent in ((0, 0, 0), (10, 11, 0), (10, 6, 5), (10, -1, 0), (10, 0, -1),
                                  (65, 0, 0)):
        with pytest.raises(ctr.CtrError) as e:
            plan.evict(tables, lens, w, tables + 4, budget, sinks, recent)
        assert e.value.status == ctr.CTR_ERR_INVALID_ARG
    with pytest.raises(ctr.CtrError):
        plan.evict(tables, lens, w, tables + 4, 32, lens_out=lens)
    with pytest.raises(ValueError):
        plan.evict(tables, lens, w[:, :, :63], tables + 4, 32)
    with pytest.raises(TypeError):
        plan.evict(tables.long(), lens, w, tables + 4, 32)
    with pytest.raises(ValueError):
        plan.evict(tables, lens, w, (tables + 4)[0], 32)


def test_attention_after_eviction():
    """The evicted cache attends as the kept rows do."""
    g = torch.Generator().manual_seed(5)
    n, budget, page, D = 100, 40, 16, 64
    k, v = (torch.randn(16, 1, page, D, generator=g).cuda() for _ in range(2))
    q = torch.randn(1, 2, D, generator=g).cuda()
    plan = ctr.PagedAttention(1, 2, 1, D, page, 8, k_pages=k, v_pages=v, weights=True)
    tables = torch.arange(8, dtype=torch.int32).cuda()[None]
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    w = torch.zeros(1, 1, plan.capacity).cuda()
    plan.forward(q, tables, lens, weights=w)
    to = torch.full((1, 8), 2 ** 30, dtype=torch.int32).cuda()
    to[0, :3] = torch.tensor([8, 10, 12])
    w2 = torch.zeros_like(w)
    slots, lens2, _ = plan.evict(tables, lens, w, to, budget, 2, 10, weights_out=w2)
    out = plan.forward(q, to, lens2, weights=w2)
    plan.check()
    j = slots[0, 0].long()
    kk, vv = (x[j // page, 0, j % page].double() for x in (k, v))
    p = torch.softmax(q[0].double() @ kk.T / D ** 0.5, -1)
    assert (out[0].double() - p @ vv).abs().max().item() < 1e-5
    assert ((w2[0, 0, :budget] - w[0, 0, j]).double() - p.sum(0)).abs().max().item() < 1e-5
