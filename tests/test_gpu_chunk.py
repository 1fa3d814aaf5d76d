"""GPU tests of PagedAttention.forward_chunk against the 64-bit form of its formula, with an error bound
derived per output (chunk_reference.attention_bound)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import chunk_reference as ref  # noqa: E402
import transposed_convolution_gb300 as ctr  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NAN = float("nan")


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def make(Hq, Hkv, D, page, lens, counts, dtype="bf16", layout="head", seed=0, peaked=1.0, max_pages=None,
         window=0, before=0, behind=0, **kw):
    """A cache whose other rows are NaN, with pages dealt out in a random order (those behind the
    window gone), q as a slice of a fused projection, and the plan."""
    g = torch.Generator().manual_seed(seed)
    B, dt = len(lens), DT[dtype]
    total = [max(n, 0) + m for n, m in zip(lens, counts)]
    need = [max(1, -(-n // page)) for n in total]
    most = max(need) if max_pages is None else max_pages
    pages = sum(need) + 2
    perm = torch.randperm(pages, generator=g)
    tables = torch.full((B, most), 2 ** 30, dtype=torch.int32)
    shape = (pages, Hkv, page, D) if layout == "head" else (pages, page, Hkv, D)
    k, v = (torch.full(shape, NAN) for _ in range(2))
    at = 0
    for b in range(B):
        tables[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        gone = max(0, max(lens[b], 0) + 1 - window) if window else 0
        j = torch.arange(gone, total[b])
        pg, off = tables[b, j // page].long(), j % page
        for x in (k, v):
            rows = torch.randn(len(j), Hkv, D, generator=g)
            if layout == "head":
                x[pg, :, off] = rows
            else:
                x[pg, off] = rows
        tables[b, :gone // page] = -1
    T = before + sum(counts) + behind
    q = torch.randn(T, Hq + 2 * Hkv, D, generator=g)[:, :Hq] * peaked
    starts = np.concatenate([[0], np.cumsum(counts)]) + before
    s = dict(q=torch.empty(T, Hq + 2 * Hkv, D, dtype=dt, device="cuda")[:, :Hq].copy_(q),
             k=k.to(dt).cuda(), v=v.to(dt).cuda(), tables=tables.cuda(),
             lens=torch.tensor(lens, dtype=torch.int32).cuda(),
             starts=torch.tensor(starts, dtype=torch.int32).cuda(),
             page=page, layout=layout, window=window, dtype=dtype)
    s["plan"] = ctr.PagedAttention(B, Hq, Hkv, D, page, most, k_pages=s["k"], v_pages=s["v"],
                                   layout=layout, window=window, chunks=True, **kw)
    return s


def run(s):
    out = torch.full(s["q"].shape, 77.0, dtype=DT[s["dtype"]], device="cuda")
    return s["plan"].forward_chunk(s["q"], s["tables"], s["lens"], s["starts"], out=out)


def check(s, out, scale=None, hidden=()):
    tables, lens, starts = (s[a].cpu().numpy() for a in ("tables", "lens", "starts"))
    want, ds, mass = ref.attention(f64(s["q"]), f64(s["k"]), f64(s["v"]), tables, lens, starts, s["page"],
                                   s["layout"], s["window"], scale, hidden=hidden)
    longest = int(np.max(lens) + np.max(np.diff(starts)))
    got = f64(out)
    free = np.isnan(want[:, 0, 0])
    assert (got[free] == 77.0).all(), "a row of no sequence was written"
    got, want, ds, mass = got[~free], want[~free], ds[~free], mass[~free]
    bound = ref.attention_bound(want, ds, mass, longest, s["dtype"])
    err = np.abs(got - want)
    assert np.isfinite(err).all()
    if err.size:
        assert (err <= bound).all(), "worst error %.3g of its bound" % (err / bound).max()
    return want


SHAPES = [  # (Hq, Hkv, D, page, lens, counts, window)
    (1, 1, 64, 16, [0], [1], 0),                              # the first token of all
    (4, 4, 64, 16, [125], [4], 0),
    (8, 2, 128, 64, [0], [300], 0),                           # a prompt: several tiles of rows
    (8, 2, 128, 16, [37, 0, 500, 63, 64], [1, 130, 70, 65, 64], 0),
    (6, 2, 80, 20, [3, 701, 90], [100, 33, 1], 0),            # three heads to a KV head
    (3, 3, 96, 24, [255, 256, 257], [1, 1, 1], 0),
    (16, 2, 128, 8, [1000], [17], 0),
    (5, 1, 256, 16, [200, 0], [130, 259], 0),
    (32, 1, 48, 7, [11], [9], 0),                             # odd pages, many heads
    (2, 2, 16, 1, [5, 0], [40, 3], 0),                        # pages of one row
    (2, 1, 112, 33, [130], [200], 0),
    (4, 2, 240, 128, [100], [100], 0),
    (4, 1, 160, 48, [0, 5], [77, 200], 0),
    (4, 2, 64, 16, [0, 300, 90, 5], [200, 40, 170, 1], 100),  # a window
    (4, 2, 128, 16, [700], [300], 1),                         # each token sees itself
    (2, 2, 80, 20, [1000, 10], [300, 300], 257),
    (8, 8, 64, 64, [2000, 0, 0, 9], [3, 0, 1, 0], 0),         # sequences without new tokens
    (4, 2, 64, 16, [-1, 50, -1], [5, 20, 1], 0),              # idle ones
    (128, 1, 64, 16, [60], [3], 0),
]


@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_formula(shape, dtype, layout):
    Hq, Hkv, D, page, lens, counts, window = shape
    s = make(Hq, Hkv, D, page, lens, counts, dtype, layout, seed=D + page, window=window, peaked=2.0)
    check(s, run(s))
    s["plan"].check()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_long_caches_are_shared_out(dtype):
    """Few rows on a long cache: every block has a part of it.  Twice: the same bits."""
    s = make(8, 2, 128, 16, [9000, 300], [5, 2], dtype, peaked=3.0)
    out = run(s)
    check(s, out)
    assert torch.equal(out, run(s))
    s = make(4, 1, 64, 64, [5000], [700], dtype, peaked=3.0)
    out = run(s)
    check(s, out)
    assert torch.equal(out, run(s))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_around_the_sequences_are_left_alone(dtype):
    s = make(4, 2, 64, 16, [40, 7], [33, 150], dtype, before=3, behind=9)
    check(s, run(s))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_short_sequences(dtype):
    rng = np.random.default_rng(5)
    lens, counts = rng.integers(0, 60, 300).tolist(), rng.integers(0, 5, 300).tolist()
    s = make(4, 2, 64, 8, lens, counts, dtype)
    check(s, run(s))
    s = make(2, 1, 32, 8, [3] * 1024, [1] * 1024, dtype)
    check(s, run(s))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_weights_far_below_the_largest(dtype):
    """One slot far above the others, whose sum still counts: 2^-13 each, 3000 of them."""
    s = make(1, 1, 64, 16, [3000], [1], dtype)
    q = torch.zeros_like(s["q"])
    q[..., 0] = 8.0
    s["q"].copy_(q)
    s["k"][:] = 0
    s["k"].view(-1, 64)[:, 0] = 0.0
    first = s["tables"][0, 0].item()
    s["k"][first, 0, 0, 0] = 9.0                              # score 9 against 0: e^-9 = 1.2e-4
    s["v"][:] = 1.0
    s["v"][first, 0, 0] = 0.0
    want = check(s, run(s))
    assert 0.2 < want[0, 0, 0] < 0.3


def test_fp16_weights_below_its_smallest_number():
    """Scores 14 under one slot's: e^-14 = 2^-20, and 30000 slots of it, 2.4% of the sum; half a step of
    fp16 itself is 2^-25, which would be 3% of each."""
    s = make(1, 1, 64, 64, [30000], [1], "f16")
    s["q"].zero_()
    s["q"][..., 0] = 8.0
    s["k"].zero_()
    first = s["tables"][0, 0].item()
    s["k"][first, 0, 0, 0] = 14.0
    s["v"][:] = 1.0
    s["v"][first, 0, 0] = 0.0
    check(s, run(s))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), NAN])
def test_what_is_masked_never_arrives(dtype, bad):
    """A token's V that is no number reaches that token and those after it, and nothing else; outside a
    window it reaches nobody."""
    s = make(4, 2, 64, 16, [150], [100], dtype)
    clean = run(s)
    pg, off = s["tables"][0, 190 // 16].item(), 190 % 16
    s["v"][pg, 1, off, 7] = bad
    got = run(s)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[40:, 2:, 7] = True
    assert torch.equal(got[~hit], clean[~hit])
    assert (got[hit].isnan() if bad != bad else got[hit] == bad).all()
    # K that is no number: the same tokens, all columns.
    s = make(4, 2, 64, 16, [150], [100], dtype)
    s["k"][pg, 1, off, 7] = NAN
    got = run(s)
    hit[40:, 2:, :] = True
    assert torch.equal(got[~hit], clean[~hit]) and got[hit].isnan().all()
    # With a window of 20 the tokens from 60 on do not see slot 190 any more.
    s = make(4, 2, 64, 16, [150], [100], dtype, window=20)
    clean = run(s)
    s["v"][pg, 1, off, 7] = bad
    got = run(s)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[40:60, 2:, 7] = True
    assert torch.equal(got[~hit], clean[~hit])
    assert (got[hit].isnan() if bad != bad else got[hit] == bad).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_opposite_infinities(dtype):
    s = make(2, 1, 64, 16, [300], [10], dtype)
    pg = s["tables"][0].tolist()
    s["v"][pg[0], 0, 0, 3] = float("inf")
    s["v"][pg[305 // 16], 0, 305 % 16, 3] = -float("inf")
    got = run(s)
    assert (got[:5, :, 3] == float("inf")).all() and got[5:, :, 3].isnan().all()
    rest = torch.ones(64, dtype=torch.bool)
    rest[3] = False
    assert got[:, :, rest].isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_values_in_shared_units(dtype):
    """The part of a unit that holds the infinity has a far smaller maximum than another part."""
    s = make(1, 1, 64, 16, [6000], [1], dtype)
    pg = s["tables"][0].tolist()
    s["q"].zero_()
    s["q"][..., 0] = 8.0
    s["k"][pg[0], 0, 0, 0] = 60.0
    s["v"][pg[350], 0, 3, 5] = float("inf")
    got = run(s)
    assert got[0, 0, 5] == float("inf")
    got[0, 0, 5] = 0
    assert got.isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_scores_without_a_number(dtype):
    s = make(2, 2, 64, 16, [40], [30], dtype)
    s["q"][3, 1] = float("inf")                               # +inf and -inf scores, or NaN
    got = run(s)
    assert got[3, 1].isnan().all()
    keep = torch.ones(30, 2, dtype=torch.bool)
    keep[3, 1] = False
    assert got[keep].isfinite().all()
    # Every score -inf: nothing is attended to.
    s = make(1, 1, 16, 16, [5], [3], dtype)
    s["k"][:] = 0
    s["k"][..., 0] = float("inf")
    s["q"].zero_()
    s["q"][..., 0] = -1.0
    # 0 times the infinities of the other columns' q is not in play: K has one infinite column.
    assert (run(s) == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_bad_pages_hide_their_slots(dtype):
    s = make(4, 2, 64, 16, [100, 30], [20, 3], dtype)
    s["tables"][0, 2] = 10 ** 6
    s["tables"][1, 0] = -3
    hidden = [(0, j) for j in range(32, 48)] + [(1, j) for j in range(16)]
    s["tables"] = s["tables"].contiguous()
    out = run(s)
    tables = s["tables"].clone()
    s["tables"][0, 2] = s["tables"][1, 0] = 0
    check(s, out, hidden=hidden)
    with pytest.raises(ctr.CtrError) as e:
        s["plan"].check()
    assert e.value.status == ctr.CTR_ERR_INVALID_ARG
    s["plan"].check()
    # A sequence of nothing but bad pages.
    s["tables"].copy_(tables)
    s["tables"][1] = -1
    assert (run(s)[20:] == 0).all()
    with pytest.raises(ctr.CtrError):
        s["plan"].check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_starts_and_lengths_out_of_range(dtype):
    s = make(4, 2, 64, 16, [30, 20, 10], [20, 5, 3], dtype)
    good = run(s)
    s["starts"].copy_(torch.tensor([0, 20, 19, 22], dtype=torch.int32))      # the second is empty
    out = run(s)
    assert torch.equal(out[:19], good[:19])
    with pytest.raises(ctr.CtrError):
        s["plan"].check()
    s["starts"].copy_(torch.tensor([-4, 20, 25, 29], dtype=torch.int32))     # the first and the last
    out = run(s)
    assert torch.equal(out[20:25], good[20:25]) and (out[:20] == 77).all() and (out[25:] == 77).all()
    with pytest.raises(ctr.CtrError):
        s["plan"].check()
    # Tokens past the table's capacity attend to all of it.
    s = make(4, 2, 64, 16, [60], [20], dtype, max_pages=5)
    s["lens"][0] = 70
    check(s, run(s))
    with pytest.raises(ctr.CtrError):
        s["plan"].check()
    s["lens"][0] = 2 ** 31 - 1
    run(s)
    with pytest.raises(ctr.CtrError):
        s["plan"].check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_chunk_of_one_is_the_decode_step(dtype):
    """One token a sequence: the same as PagedAttention.forward on the cache with that token in it.  Each is
    within its own bound of the formula (the decode step's terms are no larger: sums of longest / 16 terms
    and probabilities of 15 bits), so the two are within twice the chunk's bound of one another."""
    s = make(8, 2, 128, 16, [300, 17, 0, 64], [1, 1, 1, 1], dtype)
    out = run(s)
    check(s, out)
    step = s["plan"].forward(s["q"], s["tables"], s["lens"] + 1)
    want, ds, mass = ref.attention(f64(s["q"]), f64(s["k"]), f64(s["v"]), s["tables"].cpu().numpy(),
                                   s["lens"].cpu().numpy(), s["starts"].cpu().numpy(), 16)
    bound = ref.attention_bound(want, ds, mass, 301, dtype)
    assert (np.abs(f64(out) - f64(step)) <= 2 * bound).all()


def test_pieces_of_a_prompt_are_the_prompt():
    s = make(8, 2, 128, 16, [0], [400], "f32")
    whole = run(s)
    check(s, whole)
    want, ds, mass = ref.attention(f64(s["q"]), f64(s["k"]), f64(s["v"]), s["tables"].cpu().numpy(), [0],
                                   [0, 400], 16)
    bound = torch.from_numpy(2 * ref.attention_bound(want, ds, mass, 400, "f32"))
    at = 0
    for n in (1, 130, 64, 205):
        out = s["plan"].forward_chunk(s["q"][at:at + n], s["tables"],
                                      torch.tensor([at], dtype=torch.int32, device="cuda"),
                                      torch.tensor([0, n], dtype=torch.int32, device="cuda"))
        assert ((out.double() - whole[at:at + n].double()).abs().cpu() <= bound[at:at + n]).all()
        at += n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scale_window_and_weights(dtype):
    s = make(4, 2, 64, 16, [100], [40], dtype, scale=0.3)
    check(s, run(s), scale=0.3)
    s = make(4, 2, 64, 16, [100], [40], dtype, scale=-0.2)
    check(s, run(s), scale=-0.2)
    s = make(4, 2, 64, 16, [100], [40], dtype, weights=True)     # accumulates none here
    check(s, run(s))
    s = make(4, 2, 64, 16, [100], [40], dtype, window=10 ** 12)
    s["window"] = 0
    check(s, run(s))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(dtype):
    """Rising scores: the running maximum moves at every tile."""
    s = make(1, 1, 64, 16, [1000], [40], dtype, peaked=20.0)
    check(s, run(s))
    s["k"].copy_(s["k"] * torch.linspace(0.1, 4.0, s["k"].shape[0], device="cuda")[:, None, None, None])
    check(s, run(s))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed_on_new_inputs(dtype):
    s = make(4, 2, 64, 16, [500, 20], [30, 5], dtype)
    out = torch.full(s["q"].shape, 77.0, dtype=DT[dtype], device="cuda")
    s["plan"].forward_chunk(s["q"], s["tables"], s["lens"], s["starts"], out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s["plan"].forward_chunk(s["q"], s["tables"], s["lens"], s["starts"], out=out)
    s["lens"].copy_(torch.tensor([300, 21], dtype=torch.int32))
    s["starts"].copy_(torch.tensor([2, 20, 24], dtype=torch.int32))
    s["q"].mul_(1.5)
    out.fill_(77.0)
    graph.replay()
    torch.cuda.synchronize()
    check(s, out)


def test_another_stream():
    s = make(4, 2, 64, 16, [500, 20], [30, 5], "bf16")
    want = run(s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    got = s["plan"].forward_chunk(s["q"], s["tables"], s["lens"], s["starts"], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_no_tokens_and_argument_checks():
    s = make(4, 2, 64, 16, [50, 20], [3, 5], "bf16")
    p, q, t, n, st = s["plan"], s["q"], s["tables"], s["lens"], s["starts"]
    zero = torch.zeros_like(st)
    assert p.forward_chunk(q[:0], t, n, zero).shape == (0, 4, 64)
    out = torch.full_like(q, 5.0).contiguous()
    assert (p.forward_chunk(q, t, n, zero, out=out) == 5.0).all()
    for bad in (lambda: p.forward_chunk(q[:, :2], t, n, st), lambda: p.forward_chunk(q, t[:1], n, st),
                lambda: p.forward_chunk(q, t, n, st[:2]), lambda: p.forward_chunk(q, t, n[:1], st),
                lambda: p.forward_chunk(q, t, n, st, out=out[:3])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: p.forward_chunk(q.float(), t, n, st), lambda: p.forward_chunk(q, t.long(), n, st)):
        with pytest.raises(TypeError):
            bad()
    plain = ctr.PagedAttention(2, 4, 2, 64, 16, 4, num_pages=4, dtype=torch.bfloat16)
    with pytest.raises(ctr.CtrError) as e:
        plain.forward_chunk(q, t, n, st)
    assert e.value.status == ctr.CTR_ERR_NOT_PREPARED
    # Rows that are not on 16 bytes.
    buf = torch.zeros(8 * 260, dtype=torch.bfloat16, device="cuda").as_strided((8, 4, 64), (260, 64, 1))
    with pytest.raises(ctr.CtrError) as e:
        p.forward_chunk(buf, t, n, st)
    assert e.value.status == ctr.CTR_ERR_MISALIGNED
