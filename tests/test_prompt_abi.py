"""The host half of the operators of a chunk of new tokens, without a GPU: creation, settings and the
statuses of refused calls.  No call here launches a kernel."""
import ctypes

import numpy as np
import pytest

import chunk_reference as ref


@pytest.fixture(scope="module")
def ctr():
    from transposed_convolution_gb300 import build
    build.build()
    import transposed_convolution_gb300 as t
    t.load_library()
    return t


P = ctypes.c_void_p
A = 1 << 20


def test_chunks_setting_and_workspace(ctr):
    for dtype in (ctr.CTR_F32, ctr.CTR_BF16, ctr.CTR_F16):
        for D in (16, 64, 80, 128, 256):
            h = ctr.ctr_attn_create(3, 8, 2, D, 16, 10, dtype)
            try:
                small = ctr.ctr_attn_workspace_bytes(h)
                ctr.ctr_attn_set_chunks(h, 1)
                assert ctr.ctr_attn_workspace_bytes(h) > small
                assert "chunks" in ctr.ctr_attn_describe(h)
                ctr.ctr_attn_bind_workspace(h, A, 1 << 40)
                ctr.ctr_attn_set_chunks(h, 0)
                assert ctr.ctr_attn_workspace_bytes(h) == small
                assert ctr.lib.ctr_attn_reset(h, None) == ctr.CTR_ERR_NO_WORKSPACE
                assert ctr.lib.ctr_attn_set_chunks(h, 2) == ctr.CTR_ERR_INVALID_ARG
            finally:
                ctr.ctr_attn_destroy(h)
    assert ctr.lib.ctr_attn_set_chunks(None, 1) == ctr.CTR_ERR_INVALID_ARG


def test_chunk_calls_refused_before_any_launch(ctr):
    h = ctr.ctr_attn_create(2, 8, 2, 64, 16, 4, ctr.CTR_F16)

    def forward(plan=h, q=A, qs=512, T=10, t=A, n=A, s=A, o=A):
        return ctr.lib.ctr_attn_forward_chunk(plan, q, qs, T, t, n, s, o, None)

    try:
        bad = ctr.CTR_ERR_INVALID_ARG
        for kw in (dict(plan=None), dict(q=None), dict(t=None), dict(n=None), dict(s=None), dict(o=None),
                   dict(qs=511), dict(qs=0), dict(qs=-512), dict(T=-1)):
            assert forward(**kw) == bad, kw
        for kw in (dict(T=(1 << 24) + 1), dict(T=1 << 62)):
            assert forward(**kw) == ctr.CTR_ERR_UNSUPPORTED, kw
        for kw in (dict(q=A + 8), dict(o=A + 4), dict(t=A + 2), dict(n=A + 1), dict(s=A + 2), dict(qs=513)):
            assert forward(**kw) == ctr.CTR_ERR_MISALIGNED, kw
        assert forward() == ctr.CTR_ERR_NOT_PREPARED               # no cache
        ctr.ctr_attn_bind_cache(h, A, A, 8)
        ctr.ctr_attn_bind_workspace(h, A, 1 << 30)
        assert forward() == ctr.CTR_ERR_NOT_PREPARED               # chunks not set
        ctr.ctr_attn_set_chunks(h, 1)
        assert forward() == ctr.CTR_ERR_NO_WORKSPACE
        ctr.ctr_attn_bind_workspace(h, A, 1 << 30)
        assert forward() == ctr.CTR_ERR_NOT_PREPARED               # not reset
    finally:
        ctr.ctr_attn_destroy(h)
    h = ctr.ctr_attn_create(2, 128, 1, 64, 16, 4, ctr.CTR_F16)
    try:
        assert forward(plan=h, qs=128 * 64, T=1 << 24) == ctr.CTR_ERR_UNSUPPORTED
    finally:
        ctr.ctr_attn_destroy(h)


def test_put_refused_before_any_launch(ctr):
    h = ctr.ctr_attn_create(2, 8, 2, 64, 16, 4, ctr.CTR_F16)
    r = ctr.ctr_rope_create(64, 32, ctr.CTR_F16)
    other_d, other_t = ctr.ctr_rope_create(80, 32, ctr.CTR_F16), ctr.ctr_rope_create(64, 32, ctr.CTR_F32)

    def put(plan=h, rope=r, q=A, qs=512, k=A, v=A, kvs=128, p=A, s=A, T=3, qo=A, qos=512):
        return ctr.lib.ctr_attn_put(plan, rope, q, qs, k, v, kvs, p, s, T, qo, qos, None)

    try:
        for kw in (dict(plan=None), dict(rope=None), dict(rope=other_d), dict(rope=other_t), dict(q=None),
                   dict(qo=None), dict(k=None), dict(v=None), dict(s=None), dict(p=None), dict(kvs=127),
                   dict(qs=511), dict(qos=511), dict(T=-1)):
            assert put(**kw) == ctr.CTR_ERR_INVALID_ARG, kw
        assert put(T=(1 << 24) + 1) == ctr.CTR_ERR_UNSUPPORTED
        for kw in (dict(q=A + 8), dict(k=A + 2), dict(v=A + 8), dict(qo=A + 4), dict(p=A + 2), dict(s=A + 4),
                   dict(kvs=132), dict(qs=516), dict(qos=517)):
            assert put(**kw) == ctr.CTR_ERR_MISALIGNED, kw
        assert put() == ctr.CTR_ERR_NOT_PREPARED
        ctr.ctr_attn_bind_cache(h, A, A, 8)
        assert put() == ctr.CTR_ERR_NO_WORKSPACE
        ctr.ctr_attn_bind_workspace(h, A, 1 << 30)
        assert put() == ctr.CTR_ERR_NOT_PREPARED
    finally:
        ctr.ctr_attn_destroy(h)
        for x in (r, other_d, other_t):
            ctr.ctr_rope_destroy(x)


@pytest.mark.parametrize("args,status", [
    ((0, 0, 0), "CTR_ERR_INVALID_ARG"), ((64, 0, 0), "CTR_ERR_INVALID_ARG"),
    ((64, 3, 0), "CTR_ERR_INVALID_ARG"), ((64, 66, 0), "CTR_ERR_INVALID_ARG"),
    ((64, 64, 3), "CTR_ERR_INVALID_ARG"), ((514, 64, 0), "CTR_ERR_UNSUPPORTED"),
    ((1 << 62, 64, 0), "CTR_ERR_UNSUPPORTED")])
def test_rope_create_refuses(ctr, args, status):
    h = P(1)
    assert ctr.lib.ctr_rope_create(ctypes.byref(h), *args) == getattr(ctr, status)
    assert not h.value
    assert ctr.lib.ctr_rope_create(None, *args) == ctr.CTR_ERR_INVALID_ARG


def test_rope_settings_and_frequencies(ctr):
    h = ctr.ctr_rope_create(128, 96, ctr.CTR_BF16)
    lib, bad, nan, inf = ctr.lib, ctr.CTR_ERR_INVALID_ARG, float("nan"), float("inf")
    try:
        for base, kw in ((10000.0, {}), (500000.0, dict(scaling="linear", factor=4.0)),
                         (1e6, dict(scaling="parts", factor=32.0, original=8192.0, low=1.0, high=4.0)),
                         (1.0, dict(scaling="parts", factor=0.5, original=3.0, low=0.0, high=0.1))):
            ctr.ctr_rope_set_base(h, base)
            kinds = {None: 0, "linear": 1, "parts": 2}
            ctr.ctr_rope_set_scaling(h, kinds[kw.get("scaling")], kw.get("factor", 1.0),
                                     kw.get("original", 0.0), kw.get("low", 0.0), kw.get("high", 0.0))
            np.testing.assert_allclose(ctr.ctr_rope_frequencies(h, 48), ref.frequencies(96, base, **kw),
                                       rtol=1e-14)
        ctr.ctr_rope_set_frequencies(h, [0.25 * i for i in range(48)])
        assert ctr.ctr_rope_frequencies(h, 48) == [0.25 * i for i in range(48)]
        assert "own frequencies" in ctr.ctr_rope_describe(h)
        ctr.ctr_rope_set_base(h, 100.0)                            # drops them
        assert "base=100" in ctr.ctr_rope_describe(h) and ctr.ctr_rope_frequencies(h, 48)[0] != 0.0
        ctr.ctr_rope_set_layout(h, ctr.CTR_ROPE_INTERLEAVED)
        assert "interleaved" in ctr.ctr_rope_describe(h) and "bf16" in ctr.ctr_rope_describe(h)
        assert lib.ctr_rope_set_layout(h, 2) == bad
        for base in (0.0, 0.5, -2.0, nan, inf):
            assert lib.ctr_rope_set_base(h, base) == bad
        for args in ((3, 1.0, 1.0, 1.0, 2.0), (-1, 1.0, 1.0, 1.0, 2.0), (1, 0.0, 1.0, 1.0, 2.0),
                     (1, nan, 1.0, 1.0, 2.0), (2, 2.0, 0.0, 1.0, 2.0), (2, 2.0, 5.0, 2.0, 2.0),
                     (2, 2.0, 5.0, -1.0, 2.0), (2, 2.0, 5.0, 1.0, inf)):
            assert lib.ctr_rope_set_scaling(h, *args) == bad, args
        for m in (nan, inf):
            assert lib.ctr_rope_set_magnitude(h, m) == bad
        f = (ctypes.c_double * 48)(*([1.0] * 47 + [inf]))
        assert lib.ctr_rope_set_frequencies(h, f, 48) == bad
        assert lib.ctr_rope_set_frequencies(h, f, 47) == bad
        assert lib.ctr_rope_frequencies(h, f, 47) == bad
        assert lib.ctr_rope_frequencies(h, None, 48) == bad
    finally:
        ctr.ctr_rope_destroy(h)
    ctr.ctr_rope_destroy(None)


def test_rope_calls_refused_before_any_launch(ctr):
    h = ctr.ctr_rope_create(64, 64, ctr.CTR_BF16)

    def forward(plan=h, q=A, qs=256, hq=4, k=A, ks=128, hk=2, p=A, T=5, qo=A, qos=256, ko=A, kos=128):
        return ctr.lib.ctr_rope_forward(plan, q, qs, hq, k, ks, hk, p, T, qo, qos, ko, kos, None)

    try:
        for kw in (dict(plan=None), dict(q=None), dict(k=None), dict(p=None), dict(qo=None), dict(ko=None),
                   dict(qs=255), dict(ks=127), dict(qos=255), dict(kos=0), dict(T=-1), dict(hq=-1),
                   dict(hk=-1)):
            assert forward(**kw) == ctr.CTR_ERR_INVALID_ARG, kw
        for kw in (dict(T=(1 << 24) + 1), dict(hq=1 << 15), dict(hk=1 << 40)):
            assert forward(**kw) == ctr.CTR_ERR_UNSUPPORTED, kw
        for kw in (dict(q=A + 1), dict(k=A + 1), dict(qo=A + 1), dict(ko=A + 1), dict(p=A + 2)):
            assert forward(**kw) == ctr.CTR_ERR_MISALIGNED, kw
        assert forward(T=0, q=None, p=None) == ctr.CTR_OK          # nothing to do
        assert forward(hq=0, hk=0, q=None, k=None) == ctr.CTR_OK
    finally:
        ctr.ctr_rope_destroy(h)


def test_pages_calls_refused_before_any_launch(ctr):
    lib, bad = ctr.lib, ctr.CTR_ERR_INVALID_ARG
    h = P(1)
    for args, status in (((0, 1, 1), bad), ((1, 0, 1), bad), ((1, 1, 0), bad),
                         ((1025, 1, 1), ctr.CTR_ERR_UNSUPPORTED),
                         ((1, 1 << 20, 1 << 9), ctr.CTR_ERR_UNSUPPORTED),
                         ((1, 1 << 62, 1 << 62), ctr.CTR_ERR_UNSUPPORTED)):
        assert lib.ctr_pages_create(ctypes.byref(h), *args) == status
        assert not h.value
    assert lib.ctr_pages_create(None, 1, 1, 1) == bad
    h = ctr.ctr_pages_create(4, 16, 8)

    def reserve(plan=h, t=A, n=A, c=A + 64, rows=10, g=A + 128, st=A, s=A, p=A, lo=A + 256):
        return lib.ctr_pages_reserve(plan, t, n, c, rows, g, st, s, p, lo, None)

    def release(plan=h, t=A, n=A, k=A + 64, lo=A + 128):
        return lib.ctr_pages_release(plan, t, n, k, lo, None)

    try:
        assert ctr.ctr_pages_workspace_bytes(h) == 256 and lib.ctr_pages_workspace_bytes(None) == 0
        for kw in (dict(plan=None), dict(t=None), dict(n=None), dict(c=None), dict(g=None), dict(st=None),
                   dict(s=None), dict(p=None), dict(lo=None), dict(rows=-1), dict(lo=A), dict(lo=A + 64),
                   dict(g=A), dict(g=A + 64), dict(g=A + 256)):
            assert reserve(**kw) == bad, kw
        assert reserve(rows=(1 << 30) + 1) == ctr.CTR_ERR_UNSUPPORTED
        for kw in (dict(t=A + 2), dict(n=A + 1), dict(c=A + 2), dict(g=A + 2), dict(st=A + 2), dict(s=A + 4),
                   dict(p=A + 2), dict(lo=A + 2)):
            assert reserve(**kw) == ctr.CTR_ERR_MISALIGNED, kw
        for kw in (dict(plan=None), dict(t=None), dict(n=None), dict(k=None), dict(lo=None), dict(lo=A),
                   dict(lo=A + 64)):
            assert release(**kw) == bad, kw
        assert release(k=A + 2) == ctr.CTR_ERR_MISALIGNED
        assert reserve() == release() == lib.ctr_pages_reset(h, 0, None) == ctr.CTR_ERR_NOT_PREPARED
        for args in ((None, A, 4), (A, None, 4), (A, A, 4), (A, A + 64, 0)):
            assert lib.ctr_pages_bind_list(h, *args) == bad
        assert lib.ctr_pages_bind_list(h, A + 2, A + 64, 4) == ctr.CTR_ERR_MISALIGNED
        assert lib.ctr_pages_bind_list(h, A, A + 64, 1 << 31) == ctr.CTR_ERR_UNSUPPORTED
        ctr.ctr_pages_bind_list(h, A, A + 64, 4)
        assert reserve() == release() == lib.ctr_pages_check(h, None) == ctr.CTR_ERR_NO_WORKSPACE
        assert lib.ctr_pages_bind_workspace(h, A + 64, 256) == ctr.CTR_ERR_MISALIGNED
        assert lib.ctr_pages_bind_workspace(h, A, 255) == ctr.CTR_ERR_NO_WORKSPACE
        assert lib.ctr_pages_bind_workspace(h, None, 256) == bad
        assert lib.ctr_pages_reset(h, 2, None) == bad
        ctr.ctr_pages_bind_workspace(h, A, 256)
        assert reserve() == release() == ctr.CTR_ERR_NOT_PREPARED  # not reset
        assert "page=16" in ctr.ctr_pages_describe(h)
    finally:
        ctr.ctr_pages_destroy(h)
    ctr.ctr_pages_destroy(None)
