"""GPU tests of PagedAttention.forward against the 64-bit form of its formula, with an error
bound derived per output (decode_reference.attention_bound)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import decode_reference as ref  # noqa: E402
import transposed_convolution_gb300 as ctr  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def make(B, Hq, Hkv, D, page, lens, dtype="bf16", layout="head", new=True, extra=0, seed=0,
         stale=float("nan"), peaked=1.0, max_pages=None):
    """A cache whose unused rows hold ``stale``, with pages dealt out in a random order, and the
    step's inputs as slices of one fused projection."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    need = [max(1, -(-(max(n, 0) + (1 if new else 0)) // page)) for n in lens]
    most = max(need) if max_pages is None else max_pages
    total = sum(need) + extra
    perm = torch.randperm(total, generator=g).tolist()
    tables = torch.full((B, most), 2 ** 30, dtype=torch.int32)     # past the end: never read
    at = 0
    for b in range(B):
        tables[b, :need[b]] = torch.tensor(perm[at:at + need[b]], dtype=torch.int32)
        at += need[b]
    shape = (total, Hkv, page, D) if layout == "head" else (total, page, Hkv, D)
    k, v = (torch.full(shape, stale).to(dt) for _ in range(2))
    for b in range(B):
        for j in range(max(lens[b], 0)):
            at = (tables[b, j // page].item(), slice(None), j % page) if layout == "head" else \
                (tables[b, j // page].item(), j % page)
            k[at] = torch.randn(Hkv, D, generator=g).to(dt)
            v[at] = torch.randn(Hkv, D, generator=g).to(dt)
    qkv = torch.randn(B, Hq + 2 * Hkv, D, generator=g)
    qkv[:, :Hq] *= peaked
    qkv = qkv.to(dt).cuda()
    s = dict(q=qkv[:, :Hq], tables=tables.cuda(),
             lens=torch.tensor(lens, dtype=torch.int32).cuda(), k=k.cuda(), v=v.cuda(),
             k_new=qkv[:, Hq:Hq + Hkv] if new else None,
             v_new=qkv[:, Hq + Hkv:] if new else None)
    return s


def check(s, out, page, layout, dtype, window=0, scale=None, weights=None, hidden=()):
    """Compare with the reference on the cache as it was; returns the probabilities."""
    lens = s["lens"].cpu().numpy()
    args = [f64(x) for x in (s["q"], s["k"], s["v"])]
    new = [None if s[a] is None else f64(s[a]) for a in ("k_new", "v_new")]
    want, probs, ds, mass = ref.attention(*args, s["tables"].cpu().numpy(), lens, page, layout,
                                          *new, window=window, scale=scale, hidden=hidden)
    bound = ref.attention_bound(want, ds, mass, int(lens.max()) + 1, dtype)
    err = np.abs(f64(out) - want)
    assert np.isfinite(err).all()
    assert (err <= bound).all(), "worst error %.3g of its bound" % (err / bound).max()
    return probs, ds


SHAPES = [  # (B, Hq, Hkv, D, page, lens, layout, window)
    (1, 1, 1, 64, 16, [0], "head", 0),                       # the first token of all
    (1, 16, 16, 64, 16, [125], "head", 0),
    (3, 8, 2, 128, 16, [1, 63, 64], "head", 0),              # around a tile of 64
    (4, 8, 8, 80, 20, [15, 16, 17, 300], "token", 0),        # a head size of no power of two
    (2, 32, 8, 128, 64, [1000, 7], "head", 0),
    (2, 6, 2, 96, 24, [129, 511], "token", 100),             # group of three, window, odd page
    (5, 16, 1, 128, 8, [0, 5, 77, 256, 1025], "head", 0),    # one KV head for all
    (1, 40, 2, 64, 32, [333], "head", 0),                    # group of 20: more than 16 rows
    (2, 4, 4, 256, 16, [50, 200], "token", 7),
    (3, 2, 1, 16, 1, [3, 40, 65], "head", 0),                # pages of one row, smallest head
    (2, 8, 4, 128, 1000, [1500, 999], "head", 1),            # window of the new token alone
    (70, 4, 2, 64, 16, list(range(70)), "head", 0),
    (1, 8, 2, 128, 64, [20000], "token", 0),                 # split over the length
    (3, 12, 4, 48, 16, [700, 2, 5000], "head", 3000),
    (2, 9, 9, 144, 48, [100, 333], "head", 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "B%d-q%d-kv%d-D%d-p%d-n%d-%s-w%d" % (
    s[:5] + (max(s[5]),) + s[6:]))
def test_with_new_token(shape, dtype):
    B, Hq, Hkv, D, page, lens, layout, window = shape
    s = make(B, Hq, Hkv, D, page, lens, dtype, layout, seed=len(lens) + D, peaked=2.0)
    before = s["k"].clone(), s["v"].clone()
    plan = ctr.PagedAttention(B, Hq, Hkv, D, page, s["tables"].shape[1], k_pages=s["k"],
                              v_pages=s["v"], layout=layout, window=window)
    out = plan.forward(s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"])
    plan.check()
    s["k"], s["v"] = before
    check(s, out, page, layout, dtype, window)
    # The new rows are in place, and nothing else of the cache has changed.
    for b, n in enumerate(lens):
        pg = s["tables"][b, n // page].item()
        at = (pg, slice(None), n % page) if layout == "head" else (pg, n % page)
        before[0][at], before[1][at] = s["k_new"][b], s["v_new"][b]
    assert torch.equal(plan.k_pages.view(torch.uint8), before[0].view(torch.uint8))
    assert torch.equal(plan.v_pages.view(torch.uint8), before[1].view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_new_token_empty_and_idle_rows(dtype):
    lens = [0, -1, 33, 128, -2147483648, 1]
    s = make(6, 8, 2, 64, 16, lens, dtype, new=False, seed=3)
    plan = ctr.PagedAttention(6, 8, 2, 64, 16, s["tables"].shape[1], k_pages=s["k"],
                              v_pages=s["v"])
    out = torch.full((6, 8, 64), float("nan"), dtype=DT[dtype], device="cuda")
    assert plan.forward(s["q"], s["tables"], s["lens"], out=out) is out
    plan.check()
    check(s, out, 16, "head", dtype)
    assert not out[[0, 1, 4]].any()


def test_idle_rows_leave_the_cache_alone():
    s = make(3, 4, 4, 64, 16, [-1, 20, -5], "f16", seed=4)
    before = s["k"].clone()
    plan = ctr.PagedAttention(3, 4, 4, 64, 16, s["tables"].shape[1], k_pages=s["k"],
                              v_pages=s["v"])
    out = plan.forward(s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"])
    assert not out[[0, 2]].any() and out[1].any()
    changed = (s["k"].view(torch.int16) != before.view(torch.int16)).any(-1).nonzero()
    assert {tuple(r[[0, 2]].tolist()) for r in changed} == {(s["tables"][1, 1].item(), 4)}


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [SHAPES[i] for i in (0, 3, 5, 6, 7, 12, 13)],
                         ids=lambda s: "kv%d-D%d-n%d-w%d" % (s[2], s[3], max(s[5]), s[7]))
def test_weights(shape, dtype):
    B, Hq, Hkv, D, page, lens, layout, window = shape
    s = make(B, Hq, Hkv, D, page, lens, dtype, layout, seed=9, peaked=2.0)
    cap = page * s["tables"].shape[1]
    before = s["k"].clone(), s["v"].clone()
    plan = ctr.PagedAttention(B, Hq, Hkv, D, page, s["tables"].shape[1], k_pages=s["k"],
                              v_pages=s["v"], layout=layout, window=window, weights=True)
    w = torch.rand(B, Hkv, cap, generator=torch.Generator().manual_seed(1)).cuda()
    w[:, :, -1] = float("nan")
    for b, n in enumerate(lens):
        w[b, :, n:] = float("nan")          # nothing from the new slot on is read
    w_out = torch.full_like(w, 7.0)
    out = plan.forward(s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"], weights=w,
                       weights_out=w_out)
    s["k"], s["v"] = before
    probs, ds = check(s, out, page, layout, dtype, window)
    G = Hq // Hkv
    for b, n in enumerate(lens):
        step = probs[b].reshape(Hkv, G, n + 1).sum(1)
        want = step.copy()
        want[:, :n] += f64(w[b, :, :n])
        got = f64(w_out[b])
        rel = (2 * ds[b].max() + (n / 16 + 64) * 2.0 ** -24) * 1.01
        assert (np.abs(got[:, :n + 1] - want) <= rel * step + 4 * 2.0 ** -24 * want + 1e-30).all()
        assert (got[:, n + 1:] == 7.0).all()
    # In place, and from nothing.
    again = torch.nan_to_num(w, nan=0.0).clone()
    plan.forward(s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"], weights=again)
    for b, n in enumerate(lens):
        assert torch.equal(again[b, :, :n + 1], w_out[b, :, :n + 1])
    zero = torch.full_like(w, 5.0)
    plan.forward(s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"], weights_out=zero)
    assert abs(zero[0, 0, :lens[0] + 1].sum().item() - G) < 1e-4 * G


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 96, 112, 128, 256])
def test_many_sequences_and_units_split_anywhere(D, dtype):
    """Hundreds of units whose tiles are cut at every place, with empty and idle rows between."""
    lens = [(i * 37) % 200 if i % 9 else -1 for i in range(300)] + [3000, 0]
    s = make(len(lens), 2, 1, D, 16, lens, dtype, seed=D)
    before = s["k"].clone(), s["v"].clone()
    plan = ctr.PagedAttention(len(lens), 2, 1, D, 16, s["tables"].shape[1], k_pages=s["k"],
                              v_pages=s["v"])
    out = plan.forward(s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"])
    plan.check()
    s["k"], s["v"] = before
    check(s, out, 16, "head", dtype)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_short_caches_are_cut_into_whole_units(dtype):
    """More units than blocks, in caches of at most 256 slots a sequence."""
    lens = [(i * 29) % 255 if i % 7 else 0 for i in range(200)]
    s = make(200, 6, 3, 64, 16, lens, dtype, seed=2, max_pages=16)
    before = s["k"].clone(), s["v"].clone()
    plan = ctr.PagedAttention(200, 6, 3, 64, 16, 16, k_pages=s["k"], v_pages=s["v"], weights=True)
    w = torch.zeros(200, 3, plan.capacity, device="cuda")
    out = plan.forward(s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"], weights=w)
    plan.check()
    s["k"], s["v"] = before
    probs, ds = check(s, out, 16, "head", dtype)
    for b, n in enumerate(lens):
        want = probs[b].reshape(3, 2, n + 1).sum(1)
        rel = (2 * ds[b].max() + (n / 16 + 64) * 2.0 ** -24) * 1.01 + 4 * 2.0 ** -24
        assert (np.abs(f64(w[b, :, :n + 1]) - want) <= rel * want + 1e-30).all()


def test_scale_and_huge_scores():
    """Scores of +-1e4: the running maximum keeps the exponentials in range; a scale of zero
    averages."""
    s = make(2, 4, 2, 64, 16, [200, 37], "f32", seed=5, peaked=1e4)
    plan = ctr.PagedAttention(2, 4, 2, 64, 16, s["tables"].shape[1], k_pages=s["k"],
                              v_pages=s["v"])
    out = plan.forward(s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"])
    check(s, out, 16, "head", "f32")
    plan = ctr.PagedAttention(2, 4, 2, 64, 16, s["tables"].shape[1], k_pages=s["k"],
                              v_pages=s["v"], scale=0.0)
    out = plan.forward(s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"])
    check(s, out, 16, "head", "f32", scale=0.0)


def test_same_result_every_time():
    s = make(3, 16, 2, 128, 16, [4000, 100, 9], "bf16", seed=6)
    plan = ctr.PagedAttention(3, 16, 2, 128, 16, s["tables"].shape[1], k_pages=s["k"],
                              v_pages=s["v"], weights=True)
    w = torch.zeros(3, 2, plan.capacity, device="cuda")
    outs = []
    for _ in range(20):
        o = torch.zeros_like(w)
        outs.append((plan.forward(s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"],
                                  weights=w, weights_out=o), o))
    for a, o in outs[1:]:
        assert torch.equal(a, outs[0][0]) and torch.equal(o, outs[0][1])


def test_shared_prefix_pages():
    """Two sequences read the same first pages and append to pages of their own."""
    s = make(2, 4, 2, 64, 16, [40, 40], "bf16", seed=7)
    s["tables"][1, :2] = s["tables"][0, :2]
    plan = ctr.PagedAttention(2, 4, 2, 64, 16, 3, k_pages=s["k"], v_pages=s["v"])
    before = s["k"].clone(), s["v"].clone()
    out = plan.forward(s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"])
    s["k"], s["v"] = before
    check(s, out, 16, "head", "bf16")


def test_bad_pages_and_lengths_are_reported():
    s = make(2, 4, 2, 64, 16, [40, 31], "f32", seed=8, stale=0.0)
    s["tables"][0, 1] = 1000          # slots 16..31 of sequence 0
    plan = ctr.PagedAttention(2, 4, 2, 64, 16, 3, k_pages=s["k"], v_pages=s["v"])
    before = s["k"].clone(), s["v"].clone()
    out = plan.forward(s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"])
    with pytest.raises(ctr.CtrError) as e:
        plan.check()
    assert e.value.status == ctr.CTR_ERR_INVALID_ARG
    plan.check()                      # cleared
    after = s["k"].clone()
    s["k"], s["v"] = before
    s["tables"][0, 1] = 0             # the reference reads something there and hides it
    check(s, out, 16, "head", "f32", hidden=[(0, j) for j in range(16, 32)])
    # A full sequence: no room for the new row, which is not put; the others are attended to.
    s["k"].copy_(after)
    s["tables"][0] = torch.tensor([0, 1, 2])
    full = torch.tensor([48, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    s["tables"][1] = torch.tensor([2, 1, 0])
    plan = ctr.PagedAttention(2, 4, 2, 64, 16, 3, k_pages=s["k"], v_pages=s["v"])
    before = s["k"].clone()
    out = plan.forward(s["q"], s["tables"], full, s["k_new"], s["v_new"])
    with pytest.raises(ctr.CtrError):
        plan.check()
    assert torch.equal(s["k"], before)
    cut = dict(s, lens=torch.tensor([48, 48], dtype=torch.int32), k_new=None, v_new=None)
    check(cut, out, 16, "head", "f32")


def test_cache_beyond_32_bit_offsets():
    """Pages past 2^31 elements (and 2^32 bytes) into the cache."""
    Hkv, page, D = 8, 64, 128
    total = 2 ** 31 // (Hkv * page * D) + 40
    k = torch.empty(total, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    s = make(1, 16, Hkv, D, page, [300], "bf16", seed=10)
    need = s["tables"].shape[1]
    high = torch.arange(total - need, total, dtype=torch.int32)
    k[total - need:] = s["k"][s["tables"][0].long()]
    v[total - need:] = s["v"][s["tables"][0].long()]
    plan = ctr.PagedAttention(1, 16, Hkv, D, page, need, k_pages=k, v_pages=v)
    out = plan.forward(s["q"], high.cuda()[None], s["lens"], s["k_new"], s["v_new"])
    check(s, out, page, "head", "bf16")
    assert torch.equal(k[total - need + 300 // page, :, 300 % page], s["k_new"][0])
    # Eviction to and from there.
    w = torch.rand(1, Hkv, need * page, device="cuda")
    to = torch.arange(total - need - 1, total - need, dtype=torch.int32, device="cuda")[None]
    slots, n, _ = plan.evict(high.cuda()[None], s["lens"], w, to, 50)
    assert n.item() == 50
    for h in (0, Hkv - 1):
        j = slots[0, h].long()
        rows = k[(total - need) + j // page, h, j % page]
        assert torch.equal(k[total - need - 1, h, :50], rows)


def test_other_stream_and_graph():
    s = make(2, 8, 2, 128, 16, [500, 90], "bf16", seed=11)
    plan = ctr.PagedAttention(2, 8, 2, 128, 16, s["tables"].shape[1], k_pages=s["k"],
                              v_pages=s["v"], weights=True)
    w = torch.zeros(2, 2, plan.capacity, device="cuda")
    args = (s["q"], s["tables"], s["lens"], s["k_new"], s["v_new"])
    want = plan.forward(*args, weights_out=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = plan.forward(*args, weights_out=w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.forward(*args, weights_out=w, out=out)
    s["q"].mul_(-0.5)
    fresh = plan.forward(*args, weights_out=torch.zeros_like(w))
    out.zero_()
    g.replay()
    assert torch.equal(out, fresh) and not torch.equal(out, want)


def test_refusals():
    s = make(2, 8, 2, 64, 16, [30, 3], "f16", seed=12)
    plan = ctr.PagedAttention(2, 8, 2, 64, 16, s["tables"].shape[1], k_pages=s["k"],
                              v_pages=s["v"])
    ok = dict(q=s["q"], tables=s["tables"], lens=s["lens"], k_new=s["k_new"], v_new=s["v_new"])
    plan.forward(**ok)
    bad = [
        (ValueError, dict(q=s["q"][:1])),
        (ValueError, dict(q=s["q"].cpu())),
        (TypeError, dict(q=s["q"].float())),
        (ValueError, dict(q=s["q"].transpose(1, 2).contiguous().transpose(1, 2))),
        (ValueError, dict(v_new=None)),
        (TypeError, dict(lens=s["lens"].long())),
        (ValueError, dict(tables=s["tables"][:, :1])),
        (ValueError, dict(weights=torch.zeros(2, 2, plan.capacity, device="cuda"))),
        (ValueError, dict(out=torch.empty(2, 8, 32, device="cuda"))),
    ]
    for kind, change in bad:
        with pytest.raises(kind):
            plan.forward(**dict(ok, **change))
    # Rows that do not start on 16-byte boundaries.
    wide = torch.zeros(2, 8 * 64 + 1, dtype=torch.float16, device="cuda")
    q = torch.as_strided(wide, (2, 8, 64), (8 * 64 + 1, 64, 1))
    with pytest.raises(ctr.CtrError) as e:
        plan.forward(**dict(ok, q=q))
    assert e.value.status == ctr.CTR_ERR_MISALIGNED
    with pytest.raises(ValueError):
        ctr.PagedAttention(2, 8, 2, 64, 16, 4)
    with pytest.raises(ValueError):
        ctr.PagedAttention(2, 8, 2, 64, 16, 4, num_pages=4, layout="paged")
    for args, status in (((2, 8, 3, 64, 16, 4), ctr.CTR_ERR_INVALID_ARG),
                         ((2, 8, 2, 72, 16, 4), ctr.CTR_ERR_UNSUPPORTED),
                         ((2, 8, 2, 272, 16, 4), ctr.CTR_ERR_UNSUPPORTED)):
        with pytest.raises(ctr.CtrError) as e:
            ctr.PagedAttention(*args, num_pages=4)
        assert e.value.status == status
    with pytest.raises(ValueError):
        ctr.PagedAttention(2, 8, 2, 64, 16, 4, num_pages=4, weights=True).forward(
            s["q"].float(), s["tables"], s["lens"])
