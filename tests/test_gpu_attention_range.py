"""GPU tests of PagedAttention.forward over the whole range of the softmax: one slot that takes nearly
all weight beside thousands whose weights are 2^-17 to 2^-29 of its, and very large scores.

Error bound: that of decode_reference, plus what 16-bit caches of type fp16 may lose below its range.
They multiply V with probabilities whose last bit is at least 2^-37 of the largest one, so each
slot may be off by that much of its |V|."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import decode_reference as ref  # noqa: E402
import transposed_convolution_gb300 as ctr  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
PAGE = 16


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def one_sequence(scores, v, Hq, D, dtype, weights=False, scale=1.0):
    """out [Hq, D] (and the weights) of n slots whose scores, for every head, are the given ones times
    ``scale``: K's first column holds them and q is the first unit vector."""
    n = len(scores)
    pages = -(-n // PAGE)
    k = torch.zeros(pages * PAGE, D)
    k[:n, 0] = torch.from_numpy(scores).float()
    rows = torch.zeros(pages * PAGE, D)
    rows[:n] = torch.from_numpy(v).float()
    k, rows = (x.to(DT[dtype]).view(pages, 1, PAGE, D).cuda() for x in (k, rows))
    q = torch.zeros(1, Hq, D, dtype=DT[dtype], device="cuda")
    q[:, :, 0] = 1
    plan = ctr.PagedAttention(1, Hq, 1, D, PAGE, pages, k_pages=k, v_pages=rows, scale=scale, weights=weights)
    tables = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    w = torch.zeros(1, 1, plan.capacity, device="cuda") if weights else None
    out = plan.forward(q, tables, lens, weights=w)
    plan.check()
    return f64(out)[0], None if w is None else f64(w)[0, 0, :n]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("Hq,D", [(4, 64), (2, 128), (12, 80), (1, 256)])
@pytest.mark.parametrize("n,at", [(8192, 5), (8192, 4100), (8192, 8191), (20000, 777), (200, 3)])
@pytest.mark.parametrize("gap", [12.0, 14.25, 17.0, 20.0])
def test_one_slot_takes_nearly_all(gap, n, at, Hq, D, dtype):
    """A sink whose value is 0, and others ``gap`` nats below it with values that add up."""
    rng = np.random.default_rng(n + at + D)
    scores = np.full(n, 1.0 - gap)          # exact in every type
    scores[at] = 1.0
    v = 1.0 + rng.integers(-32, 32, (n, D)) / 64.0
    v[at] = 0.0
    out, w = one_sequence(scores, v, Hq, D, dtype, weights=True)
    e = np.exp(scores - scores.max())
    p = e / e.sum()
    want = np.broadcast_to(p @ v, out.shape)
    # Scores are exact; log2(e) times them is rounded once, at up to 20 nats.
    ds = np.full((1, Hq), 32 * 2.0 ** -24)
    bound = ref.attention_bound(want[None], ds, want[None], n, dtype)[0]
    if dtype == "f16":
        bound = bound + 2.0 ** -37 * np.abs(v).sum(0)
    err = np.abs(out - want)
    assert (err <= bound).all(), "worst error %.3g of its bound" % (err / bound).max()
    rel = (2 * ds.max() + (n / 16 + 64) * 2.0 ** -24) * 1.01
    assert (np.abs(w - Hq * p) <= rel * Hq * p + 4 * 2.0 ** -24 * Hq * p + 1e-30).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 1000.0, 4096.0, 2.0 ** 20])
@pytest.mark.parametrize("size", [100.0, 2048.0, 61440.0])
@pytest.mark.parametrize("Hq,D", [(1, 64), (16, 128)])
def test_large_equal_scores_average(size, scale, Hq, D, dtype):
    """All scores alike, however large (fp32 holds them to 4096 at the worst): the mean of V."""
    rng = np.random.default_rng(D)
    for n in (1, 100, 3000):
        for sign in (1.0, -1.0):
            v = rng.integers(-64, 64, (n, D)) / 64.0
            out, _ = one_sequence(np.full(n, sign * size), v, Hq, D, dtype, scale=scale)
            want = np.broadcast_to(v.mean(0), out.shape)
            mass = np.broadcast_to(np.abs(v).mean(0), out.shape)
            bound = ref.attention_bound(want[None], np.zeros((1, Hq)), mass[None], n, dtype)[0]
            assert (np.abs(out - want) <= bound).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_rising_scores(dtype):
    """Every slot's score is above the one before: the running maximum is raised again and again, by
    less and by more than it may lag."""
    rng = np.random.default_rng(1)
    for step in (0.0625, 1.0, 16.0):
        n = min(3000, int(60000 / step))
        scores = np.arange(n) * step - 1000.0
        scores = scores.astype(np.float16).astype(np.float64)      # bf16 rounds again below
        scores = torch.from_numpy(scores).to(DT[dtype]).double().numpy()
        v = rng.integers(1, 64, (n, 64)) / 64.0
        out, _ = one_sequence(scores, v, 8, 64, dtype)
        e = np.exp(scores - scores.max())
        want = np.broadcast_to((e / e.sum()) @ v, out.shape)
        # Scores of size s become s log2(e), rounded at 2^-24 of that, and differences thereof.
        ds = np.full((1, 8), np.abs(scores).max() * 4 * 2.0 ** -24)
        bound = ref.attention_bound(want[None], ds, want[None], n, dtype)[0]
        if dtype == "f16":
            bound = bound + 2.0 ** -37 * np.abs(v).sum(0)
        assert (np.abs(out - want) <= bound).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("what", ["nan score", "inf score", "nan value"])
@pytest.mark.parametrize("n,at,window", [(100, 40, 0), (700, 3, 0), (700, 699, 0), (9000, 5000, 0), (700, 600, 200)])
def test_not_a_number_reaches_outputs_and_weights(n, at, window, what, dtype):
    """A score that is NaN or infinite makes a head's softmax, and with it every weight of the step, NaN;
    heads of the other group and slots before the window keep theirs."""
    D, pages = 64, -(-n // PAGE)
    g = torch.Generator(device="cuda").manual_seed(n)
    k, v = (torch.randn(pages, 2, PAGE, D, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    q = torch.randn(1, 4, D, generator=g, device="cuda").to(DT[dtype])
    q[:, :, 0] = 1
    if what == "nan value":
        v[at // PAGE, 0, at % PAGE, 7] = float("nan")
    else:
        k[at // PAGE, 0, at % PAGE, 0] = float(what[:3])
    plan = ctr.PagedAttention(1, 4, 2, D, PAGE, pages, k_pages=k, v_pages=v, weights=True, window=window)
    tables = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    w = torch.full((1, 2, plan.capacity), 0.5, device="cuda")
    out = plan.forward(q, tables, lens, weights=w)
    plan.check()
    first = max(0, n - window) if window else 0
    assert torch.isfinite(out[0, 2:]).all() and torch.isfinite(w[0, 1]).all()
    assert (w[0, :, :first] == 0.5).all() and (w[0, :, n:] == 0.5).all()
    if what == "nan value":
        assert torch.isnan(out[0, :2, 7]).all() and torch.isfinite(out[0, :2, :7]).all()
        assert torch.isfinite(out[0, :2, 8:]).all() and torch.isfinite(w[0, 0]).all()
    else:
        assert torch.isnan(out[0, :2]).all()
        assert torch.isnan(w[0, 0, first:n]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("Hq,D", [(1, 64), (5, 80), (8, 128), (16, 128), (2, 256)])
@pytest.mark.parametrize("n,at", [(1, 0), (100, 40), (700, 3), (5000, 4999)])
def test_infinite_values(n, at, Hq, D, dtype):
    """An infinite value whose slot has a weight gives that infinity in its column, two of opposite
    signs NaN, and the other columns are as without them."""
    pages = -(-n // PAGE)
    g = torch.Generator(device="cuda").manual_seed(n + D)
    k, v = (torch.randn(pages, 1, PAGE, D, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    q = torch.randn(1, Hq, D, generator=g, device="cuda").to(DT[dtype])
    plan = ctr.PagedAttention(1, Hq, 1, D, PAGE, pages, k_pages=k, v_pages=v)
    tables = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    plain = plan.forward(q, tables, lens)
    row = v[at // PAGE, 0, at % PAGE]
    inf = float("inf")
    row[3], row[D - 1], row[17] = inf, -inf, inf
    other = (at * 7 + 11) % n
    v[other // PAGE, 0, other % PAGE, 17] = -inf
    out = plan.forward(q, tables, lens)
    plan.check()
    assert (out[:, :, 3] == inf).all() and (out[:, :, D - 1] == -inf).all()
    if other == at:
        assert (out[:, :, 17] == -inf).all()
    else:
        assert torch.isnan(out[:, :, 17]).all()
    keep = [c for c in range(D) if c not in (3, 17, D - 1)]
    assert torch.equal(out[:, :, keep], plain[:, :, keep])
