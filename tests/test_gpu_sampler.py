"""GPU tests of Sampler against the 64-bit form of its formula.  The token has to be the
formula's, or one that fp32 rounding of two nearly equal scores (or of a filter's limit) could
give instead; decode_reference.sample returns that set, which is nearly always one token."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import decode_reference as ref  # noqa: E402
import transposed_convolution_gb300 as ctr  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FILTERS = [  # (T, k, p, min_p)
    (1.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (-1.0, 5, 0.5, 0.1), (0.7, 50, 0.95, 0.02),
    (1.3, 0, 0.9, 0.0), (0.8, 1, 1.0, 0.0), (1.0, 250, 1.0, 0.0), (1.0, 0, 0.3, 0.0),
    (2.0, 0, 1.0, 0.1), (1.0, 10 ** 6, 0.999, 0.0), (0.05, 0, 0.9, 0.0), (1.0, 7, 0.0, 0.0),
    (1.0, 0, 1.0, 2.0), (50.0, 0, 0.9999, 0.0), (1.0, 3, 0.6, 0.0), (100.0, 1500, 0.5, 0.0),
]


def tokens(logits, noise, rows_of_filters, dtype, **kw):
    cols = list(zip(*rows_of_filters))
    f = [torch.tensor(c, dtype=d).cuda() for c, d in
         zip(cols, (torch.float32, torch.int32, torch.float32, torch.float32))]
    plan = ctr.Sampler(logits.shape[0], logits.shape[1], dtype=DT[dtype])
    return plan.forward(logits, noise, f[0], f[1], f[2], f[3], **kw).cpu().tolist()


def check(logits, noise, rows_of_filters, got):
    l, e = logits.float().cpu().numpy(), noise.cpu().numpy()
    sets = 0
    for i, (T, k, p, mp) in enumerate(rows_of_filters):
        want = ref.sample(l[i], e[i], float(np.float32(T)), k, float(np.float32(p)),
                          float(np.float32(mp)))
        assert got[i] in want, "row %d %r: %d, want %r" % (i, rows_of_filters[i], got[i], want)
        sets += len(want) > 1
    assert sets <= 1 + len(rows_of_filters) // 50    # the slack decides almost nothing


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 2048, 2049, 8191, 32768, 50001, 131072, 262147])
def test_filters(V, dtype):
    g = torch.Generator(device="cuda").manual_seed(V)
    n = len(FILTERS) * (4 if V <= 2049 else 1)
    filters = (FILTERS * 4)[:n]
    logits = (torch.randn(n, V, generator=g, device="cuda") * 3).to(DT[dtype])
    noise = torch.empty(n, V, device="cuda").exponential_(generator=g)
    check(logits, noise, filters, tokens(logits, noise, filters, dtype))


@pytest.mark.parametrize("V", [5, 777, 40000])
@pytest.mark.parametrize("kind", ["equal", "two values", "one peak", "steps", "wide", "masked",
                                  "nan", "inf", "close"])
def test_odd_logits(kind, V):
    """Ties in their thousands, masks, infinities and NaN, ranges that underflow."""
    g = torch.Generator(device="cuda").manual_seed(V)
    n = len(FILTERS)
    x = torch.randn(n, V, generator=g, device="cuda")
    if kind == "equal":
        x[:] = -3.5
    elif kind == "two values":
        x = (x > 0.5).float() * 0.25
    elif kind == "one peak":
        x[:, V // 2] = 60.0
    elif kind == "steps":
        x = (x * 2).round()
    elif kind == "wide":
        x = x * 1e4
    elif kind == "masked":
        x[:, torch.rand(V, generator=g, device="cuda") < 0.7] = float("-inf")
        x[:, V - 1] = 1.0
        x[3, :V - 1] = torch.finfo(torch.float32).min     # the type's lowest value as a mask
    elif kind == "nan":
        x[:, ::2] = float("nan")
        x[:, 1] = 0.5
        x[2, :] = float("nan")
        x[5, :] = float("-inf")
    elif kind == "inf":
        x[:, 3] = float("inf")
        x[::2, V - 1] = float("inf")
    elif kind == "close":
        x = x * 1e-6
    noise = torch.empty(n, V, device="cuda").exponential_(generator=g)
    got = tokens(x, noise, FILTERS, "f32")
    check(x, noise, FILTERS, got)
    if kind == "nan":
        assert got[2] == -1 and got[5] == -1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,V", [(1, 100001), (3, 50000), (20, 9000), (170, 6000), (160, 70001)])
def test_flat_logits_by_blocks_a_row(rows, V, dtype):
    """Logits so flat that the tokens near the maximum are too many to list, in clusters of 8, 4, 2 and
    1 block, staged and not; and peaked ones in between."""
    g = torch.Generator(device="cuda").manual_seed(V)
    spread = torch.tensor([0.01, 0.3, 1.0, 4.0], device="cuda")[torch.arange(rows, device="cuda") % 4]
    logits = (torch.randn(rows, V, generator=g, device="cuda") * spread[:, None]).to(DT[dtype])
    noise = torch.empty(rows, V, device="cuda").exponential_(generator=g)
    some = [(1.0, 0, 0.9, 0.0), (0.7, 0, 0.5, 0.001), (1.0, V // 2, 0.99, 0.0), (1.0, 5000, 1.0, 0.0),
            (1.2, 3, 0.9, 0.5), (1.0, V - 1, 0.999, 0.0), (1.0, 0, 1.0, 1e-5)]
    filters = [some[(i * 3) % len(some)] for i in range(rows)]
    check(logits, noise, filters, tokens(logits, noise, filters, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,V", [(1, 150001), (6, 20000), (40, 33333), (100, 9001), (260, 5003)])
def test_cuts_below_the_list(rows, V, dtype):
    """Cuts far from the maximum, where every block of a row searches its part, a mask in front, and
    rows in between whose list will do."""
    g = torch.Generator(device="cuda").manual_seed(V + 1)
    logits = (torch.randn(rows, V, generator=g, device="cuda") * 3).to(DT[dtype])
    logits[::3, :V // 3] = float("-inf")
    noise = torch.empty(rows, V, device="cuda").exponential_(generator=g)
    some = [(1.3, 0, 0.95, 0.0), (1.3, 999, 1.0, 0.0), (0.9, 3, 1.0, 0.0), (1.3, 3000, 0.9, 0.0),
            (2.0, 0, 0.99, 1e-6), (2.5, 0, 1.0, 0.001), (1.5, V - 2, 1.0, 0.0), (1.1, 700, 0.8, 0.01)]
    filters = [some[i % len(some)] if rows > 1 else some[0] for i in range(rows)]
    check(logits, noise, filters, tokens(logits, noise, filters, dtype))


def test_equal_scores_take_the_lowest_index():
    x = torch.zeros(4, 5000, device="cuda")
    noise = torch.full((4, 5000), 0.5, device="cuda")
    noise[2, :100] = 0.75
    noise[3, 17] = 0.0          # below FLT_MIN
    noise[3, 4000] = 1e-40
    assert tokens(x, noise, [(1.0, 0, 1.0, 0.0)] * 4, "f32") == [0, 0, 100, 17]
    # Ties at the edge of top-k: the lowest indices are the ones kept.
    x[:, 3000] = 1.0
    noise = torch.arange(5000, 0, -1, device="cuda").float().expand(4, -1).contiguous()
    assert tokens(x, noise, [(1.0, 3, 1.0, 0.0)] * 4, "f32") == [3000] * 4
    noise[:, 3000] = 1e9
    assert tokens(x, noise, [(1.0, 3, 1.0, 0.0)] * 4, "f32") == [1] * 4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_defaults_strides_and_offsets(dtype):
    """No filters; rows inside larger buffers that start on no 16-byte boundary."""
    g = torch.Generator(device="cuda").manual_seed(1)
    big = (torch.randn(6, 3001, generator=g, device="cuda") * 2).to(DT[dtype])
    noise = torch.empty(6, 2999, device="cuda").exponential_(generator=g)
    logits, e = big[:, 3:2900], noise[:, 1:2898]
    plan = ctr.Sampler(6, 2897, dtype=DT[dtype])
    got = plan.forward(logits, e).cpu().tolist()
    check(logits, e, [(1.0, 0, 1.0, 0.0)] * 6, got)
    out = torch.full((6,), -7, dtype=torch.int64, device="cuda")
    assert plan.forward(logits, e, out=out) is out and out.tolist() == got


def test_every_row_its_own_filters_and_repeatable():
    g = torch.Generator(device="cuda").manual_seed(3)
    filters = (FILTERS * 20)[:300]
    logits = (torch.randn(300, 1025, generator=g, device="cuda") * 3).half()
    noise = torch.empty(300, 1025, device="cuda").exponential_(generator=g)
    got = tokens(logits, noise, filters, "f16")
    check(logits, noise, filters, got)
    for _ in range(5):
        assert tokens(logits, noise, filters, "f16") == got


def test_draws_follow_the_distribution():
    """20000 draws of 8 tokens: each frequency within five standard deviations."""
    n = 20000
    x = torch.tensor([0.0, 1.0, -1.0, 2.0, 0.5, -3.0, 1.5, float("-inf")], device="cuda")
    noise = torch.empty(n, 8, device="cuda").exponential_(
        generator=torch.Generator(device="cuda").manual_seed(4))
    plan = ctr.Sampler(n, 8)
    got = plan.forward(x.expand(n, 8).contiguous(), noise).cpu().numpy()
    p = torch.softmax(x.double(), 0).cpu().numpy()
    count = np.bincount(got, minlength=8)
    assert count[7] == 0
    assert (np.abs(count - n * p) <= 5 * np.sqrt(n * p * (1 - p)) + 1e-9).all()


def test_no_rows_other_stream_and_graph():
    assert ctr.Sampler(0, 10).forward(torch.empty(0, 10, device="cuda"),
                                      torch.empty(0, 10, device="cuda")).shape == (0,)
    g = torch.Generator(device="cuda").manual_seed(6)
    logits = torch.randn(9, 5000, generator=g, device="cuda")
    noise = torch.empty(9, 5000, device="cuda").exponential_(generator=g)
    plan = ctr.Sampler(9, 5000)
    want = plan.forward(logits, noise)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = plan.forward(logits, noise, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.forward(logits, noise, out=out)
    noise.exponential_(generator=g)
    graph.replay()
    assert torch.equal(out, plan.forward(logits, noise))


def test_refusals():
    x, e = torch.randn(3, 100, device="cuda"), torch.ones(3, 100, device="cuda")
    plan = ctr.Sampler(3, 100)
    one = torch.ones(3, device="cuda")
    for kind, args in ((ValueError, (x[:2], e)), (ValueError, (x, e[:, :99])),
                       (TypeError, (x.half(), e)), (ValueError, (x.cpu(), e)),
                       (ValueError, (x.T.contiguous().T, e)), (TypeError, (x, e.double())),
                       (TypeError, (x, e, one.double())), (ValueError, (x, e, one[:2])),
                       (TypeError, (x, e, one, one))):
        with pytest.raises(kind):
            plan.forward(*args)
    wide = torch.as_strided(x, (3, 100), (50, 1))        # rows that overlap
    with pytest.raises(ctr.CtrError) as err:
        plan.forward(wide, e)
    assert err.value.status == ctr.CTR_ERR_INVALID_ARG
    for rows, V, status in ((-1, 5, ctr.CTR_ERR_INVALID_ARG), (1, 0, ctr.CTR_ERR_INVALID_ARG),
                            (1, 2 ** 20 + 1, ctr.CTR_ERR_UNSUPPORTED)):
        with pytest.raises(ctr.CtrError) as err:
            ctr.Sampler(rows, V)
        assert err.value.status == status
    with pytest.raises(TypeError):
        ctr.Sampler(1, 5, dtype=torch.float64)
