"""GPU tests of Rotary.forward and PagedAttention.put against the 64-bit form of the formula."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import chunk_reference as ref  # noqa: E402
import transposed_convolution_gb300 as ctr  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def near(got, want, err, dtype):
    bound = err * 1.01 + ref.UNIT[dtype] * 1.01 * (np.abs(want) + err) + 2.0 ** -24
    off = np.abs(f64(got) - want)
    assert np.isfinite(off).all() and (off <= bound).all(), "worst %.3g of its bound" % (off / bound).max()


def projections(T, Hq, Hkv, D, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device="cuda").to(DT[dtype])
    return qkv, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]


SHAPES = [  # (T, Hq, Hkv, D, R)
    (1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (7, 3, 1, 80, 32), (130, 16, 4, 96, 48), (33, 2, 2, 256, 256),
    (5, 4, 2, 16, 2), (9, 2, 1, 10, 6), (3, 1, 2, 7, 4), (1300, 2, 1, 64, 40), (2, 5, 3, 512, 512)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,Hq,Hkv,D,R", SHAPES)
def test_formula(T, Hq, Hkv, D, R, layout, dtype):
    _, q, k, _ = projections(T, Hq, Hkv, D, dtype, seed=T + D)
    rng = np.random.default_rng(D)
    pos = rng.integers(-5, 1 << 20, T)
    rope = ctr.Rotary(D, R, layout=layout, dtype=DT[dtype])
    got = rope.forward(q, k, torch.from_numpy(pos.astype(np.int32)).cuda())
    for x, y in zip((q, k), got):
        want, err = ref.rotary(f64(x), pos, ref.frequencies(R), layout)
        near(y, want, err, dtype)
        assert torch.equal(y[..., R:], x[..., R:])


@pytest.mark.parametrize("kw", [
    dict(base=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="parts", factor=8.0, original=8192,
                                                                   low=1.0, high=4.0),
    dict(scaling="parts", factor=0.5, original=100.0, low=0.0, high=2.0, base=100.0)])
def test_scaling(kw):
    D, T = 128, 40
    _, q, _, _ = projections(T, 2, 1, D, "f32")
    rope = ctr.Rotary(D, dtype=torch.float32, magnitude=1.25, **kw)
    f = ref.frequencies(D, **kw)
    np.testing.assert_allclose(rope.frequencies, f, rtol=1e-14)
    pos = np.array([0, 1, -1, 4095, 8191, 131072, 1 << 30, 2 ** 31 - 1] * 5)
    got, none = rope.forward(q, None, torch.from_numpy(pos.astype(np.int32)).cuda())
    assert none is None
    want, err = ref.rotary(f64(q), pos, f, magnitude=1.25)
    near(got, want, err, "f32")
    own = ctr.Rotary(D, frequencies=f, magnitude=1.25, dtype=torch.float32)
    again, _ = own.forward(q, None, torch.from_numpy(pos.astype(np.int32)).cuda())
    want, err = ref.rotary(f64(q), pos, f, magnitude=1.25)
    near(again, want, err, "f32")


def test_frequencies_above_a_turn_and_below_zero():
    f = [7.5, -0.25]
    rope = ctr.Rotary(4, frequencies=f, dtype=torch.float32)
    x = torch.randn(6, 1, 4, device="cuda")
    pos = np.array([0, 1, 2, 3, 1000, -7])
    got, _ = rope.forward(x, None, torch.from_numpy(pos.astype(np.int32)).cuda())
    near(got, *ref.rotary(f64(x), pos, np.array(f)), "f32")


def test_negated_positions_are_the_gradient():
    """y = R x: the gradient of sum(y * w) is R^T w, and differences of the call itself agree."""
    D, T = 64, 5
    rope = ctr.Rotary(D, 48, layout="interleaved", magnitude=1.5, dtype=torch.float32)
    pos = torch.tensor([0, 3, 1000, 77, 123456], dtype=torch.int32, device="cuda")
    x, w, d = (torch.randn(T, 3, D, device="cuda") for _ in range(3))
    grad = rope.forward(w, None, -pos)[0]
    # The copied columns have no magnitude in either direction.
    want, err = ref.rotary(f64(w), -pos.cpu().numpy(), ref.frequencies(48), "interleaved", 1.5)
    near(grad, want, err, "f32")
    up, down = (rope.forward(x + s * d, None, pos)[0].double() for s in (0.5, -0.5))
    left, right = ((up - down) * w.double()).sum(), (grad.double() * d.double()).sum()
    # 960 products of numbers around 1, each off by a few 2^-22.
    assert abs(left - right) < 960 * 10 * 2.0 ** -22


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_in_place_and_strides(layout, dtype):
    qkv, q, k, v = projections(19, 6, 2, 80, dtype)
    before, pos = qkv.clone(), torch.arange(19, dtype=torch.int32, device="cuda")
    rope = ctr.Rotary(80, 64, layout=layout, dtype=DT[dtype])
    want = rope.forward(q, k, pos)
    got = rope.forward(q, k, pos, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before[:, 8:])
    # Rows at odd addresses: the scalar path gives the same.
    buf = torch.empty(19 * 641 + 1, dtype=DT[dtype], device="cuda")
    odd = buf[1:].as_strided((19, 6, 80), (641, 80, 1))
    odd.copy_(before[:, :6])
    out = rope.forward(odd, None, pos)[0]
    assert torch.equal(out, want[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("style,R", [("half", 64), ("interleaved", 64), ("half", 24), (None, 0)])
def test_put(style, R, layout, dtype):
    T, Hq, Hkv, D, page, pages = 37, 6, 2, 64, 5, 11
    _, q, k, v = projections(T, Hq, Hkv, D, dtype, seed=R)
    g = torch.Generator().manual_seed(R)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[3] = slots[20] = -1
    pos = torch.randint(0, 5000, (T,), generator=g).to(torch.int32)
    shape = (pages, Hkv, page, D) if layout == "head" else (pages, page, Hkv, D)
    kp, vp = (torch.randn(shape, generator=g).to(DT[dtype]).cuda() for _ in range(2))
    k0, v0 = kp.clone(), vp.clone()
    plan = ctr.PagedAttention(1, Hq, Hkv, D, page, pages, k_pages=kp, v_pages=vp, layout=layout)
    if style is None:
        assert plan.put(k, v, slots.cuda()) is None
        k_want = k
    else:
        rope = ctr.Rotary(D, R, layout=style, dtype=DT[dtype])
        q_want, k_want = rope.forward(q, k, pos.cuda())
        got = plan.put(k, v, slots.cuda(), q=q, positions=pos.cuda(), rotary=rope)
        assert torch.equal(got, q_want)
    plan.check()
    for t, slot in enumerate(slots.tolist()):
        if slot < 0:
            continue
        at = (slot // page, slice(None), slot % page) if layout == "head" else (slot // page, slot % page)
        k0[at], v0[at] = k_want[t], v[t]
    assert torch.equal(kp, k0) and torch.equal(vp, v0)
    # Without q, in place of q, and no tokens at all.
    if style is not None:
        plan.put(k, v, slots.cuda(), positions=pos.cuda(), rotary=rope)
        plan.put(k, v, slots.cuda(), q=q, positions=pos.cuda(), rotary=rope, q_out=q)
        assert torch.equal(q, q_want) and torch.equal(kp, k0)
        none = plan.put(k[:0], v[:0], slots[:0].cuda(), q=q[:0], positions=pos[:0].cuda(), rotary=rope)
        assert none.shape == (0, Hq, D)


def test_put_past_the_cache_is_reported():
    plan = ctr.PagedAttention(1, 2, 1, 16, 4, 4, num_pages=3, dtype=torch.float32)
    k = torch.ones(3, 1, 16, device="cuda")
    plan.put(k, k, torch.tensor([12, 1 << 40, 11], device="cuda"))
    with pytest.raises(ctr.CtrError):
        plan.check()
    assert plan.k_pages.sum() == 16 and plan.v_pages[2, 0, 3].sum() == 16
    plan.check()


def test_nothing_is_not_a_number():
    """Infinities and NaN stay in their pair."""
    rope = ctr.Rotary(16, dtype=torch.float32)
    x = torch.randn(4, 2, 16, device="cuda")
    want = rope.forward(x, None, torch.arange(4, dtype=torch.int32, device="cuda"))[0]
    x[2, 1, 3] = float("nan")
    got = rope.forward(x, None, torch.arange(4, dtype=torch.int32, device="cuda"))[0]
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[2, 1, 3] = bad[2, 1, 11] = True
    assert got[bad].isnan().all() and torch.equal(got[~bad], want[~bad])


def test_argument_checks():
    rope = ctr.Rotary(64, dtype=torch.float32)
    x = torch.randn(4, 2, 64, device="cuda")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: rope.forward(x, None, pos[:3]), lambda: rope.forward(x[..., :32], None, pos),
                lambda: rope.forward(x.transpose(1, 2), None, pos), lambda: rope.forward(x[0], None, pos),
                lambda: rope.forward(None, None, pos, q_out=x)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        rope.forward(x, None, pos.long())
    with pytest.raises(TypeError):
        rope.forward(x.half(), None, pos)
    assert rope.forward(None, None, pos) == (None, None)
    plan = ctr.PagedAttention(1, 2, 2, 64, 4, 4, num_pages=4, dtype=torch.float32)
    slots = torch.arange(4, device="cuda")
    for kw in (dict(q=x), dict(positions=pos), dict(rotary=rope), dict(q_out=x),
               dict(rotary=ctr.Rotary(32, dtype=torch.float32), positions=pos),
               dict(rotary=ctr.Rotary(64, dtype=torch.float16), positions=pos)):
        with pytest.raises(ValueError):
            plan.put(x, x, slots, **kw)
    with pytest.raises(TypeError):
        plan.put(x, x, slots.int())
    for kw in (dict(layout="other"), dict(scaling="other"), dict(scaling="parts"),
               dict(scaling="linear", frequencies=[1.0] * 32)):
        with pytest.raises(ValueError):
            ctr.Rotary(64, **kw)
    for kw in (dict(rotary_dim=65), dict(rotary_dim=3), dict(base=0.5), dict(magnitude=float("inf")),
               dict(frequencies=[1.0]), dict(scaling="linear", factor=0.0)):
        with pytest.raises(ctr.CtrError):
            ctr.Rotary(64, **kw)
