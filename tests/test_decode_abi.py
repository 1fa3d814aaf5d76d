"""The decode-step operators' host half, without a GPU: creation, sizes, settings and the statuses
of refused calls.  No call here launches a kernel."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def ctr():
    from transposed_convolution_gb300 import build
    build.build()
    import transposed_convolution_gb300 as t
    t.load_library()
    return t


P = ctypes.c_void_p


@pytest.mark.parametrize("args,status", [
    ((0, 8, 8, 64, 16, 4, 0), "CTR_ERR_INVALID_ARG"),
    ((1, 0, 8, 64, 16, 4, 0), "CTR_ERR_INVALID_ARG"),
    ((1, 8, 0, 64, 16, 4, 0), "CTR_ERR_INVALID_ARG"),
    ((1, 8, 3, 64, 16, 4, 0), "CTR_ERR_INVALID_ARG"),
    ((1, 8, 8, 0, 16, 4, 0), "CTR_ERR_INVALID_ARG"),
    ((1, 8, 8, 64, 0, 4, 0), "CTR_ERR_INVALID_ARG"),
    ((1, 8, 8, 64, 16, 0, 0), "CTR_ERR_INVALID_ARG"),
    ((1, 8, 8, 64, 16, 4, 3), "CTR_ERR_INVALID_ARG"),
    ((1, 8, 8, 64, 16, 4, -1), "CTR_ERR_INVALID_ARG"),
    ((1, 8, 8, 72, 16, 4, 0), "CTR_ERR_UNSUPPORTED"),
    ((1, 8, 8, 272, 16, 4, 0), "CTR_ERR_UNSUPPORTED"),
    ((1025, 8, 8, 64, 16, 4, 0), "CTR_ERR_UNSUPPORTED"),
    ((1, 129, 1, 64, 16, 4, 0), "CTR_ERR_UNSUPPORTED"),
    ((1, 8, 8, 64, 1 << 20, 1 << 20, 0), "CTR_ERR_UNSUPPORTED"),
    ((1, 8, 8, 64, 1 << 62, 4, 0), "CTR_ERR_UNSUPPORTED"),
    ((1024, 1 << 40, 1 << 40, 64, 16, 4, 0), "CTR_ERR_UNSUPPORTED"),
])
def test_attention_create_refuses(ctr, args, status):
    h = P(1)
    assert ctr.lib.ctr_attn_create(ctypes.byref(h), *args) == getattr(ctr, status)
    assert not h.value
    assert ctr.lib.ctr_attn_create(None, *args) == ctr.CTR_ERR_INVALID_ARG


def test_attention_settings_and_workspace(ctr):
    h = ctr.ctr_attn_create(3, 8, 2, 64, 16, 10, ctr.CTR_BF16)
    try:
        small = ctr.ctr_attn_workspace_bytes(h)
        ctr.ctr_attn_set_weights(h, 1)
        with_scores = ctr.ctr_attn_workspace_bytes(h)
        assert with_scores >= small + 3 * 8 * 160 * 4
        ctr.ctr_attn_set_layout(h, ctr.CTR_CACHE_TOKEN_MAJOR)
        ctr.ctr_attn_set_window(h, 7)
        ctr.ctr_attn_set_scale(h, 0.5)
        text = ctr.ctr_attn_describe(h)
        assert "bf16" in text and "token-major" in text and "window=7" in text
        lib, bad = ctr.lib, ctr.CTR_ERR_INVALID_ARG
        assert lib.ctr_attn_set_layout(h, 2) == bad
        assert lib.ctr_attn_set_window(h, -1) == bad
        assert lib.ctr_attn_set_weights(h, 2) == bad
        for v in (float("nan"), float("inf")):
            assert lib.ctr_attn_set_scale(h, v) == bad
        assert lib.ctr_attn_bind_workspace(h, P(4096 + 64), 1 << 40) == ctr.CTR_ERR_MISALIGNED
        assert lib.ctr_attn_bind_workspace(h, P(4096), small) == ctr.CTR_ERR_NO_WORKSPACE
        assert lib.ctr_attn_bind_workspace(h, None, 1 << 40) == bad
        assert lib.ctr_attn_bind_cache(h, P(4096 + 8), P(4096), 4) == ctr.CTR_ERR_MISALIGNED
        assert lib.ctr_attn_bind_cache(h, P(4096), None, 4) == bad
        assert lib.ctr_attn_bind_cache(h, P(4096), P(4096), 0) == bad
        assert lib.ctr_attn_bind_cache(h, P(4096), P(4096), 1 << 31) == ctr.CTR_ERR_UNSUPPORTED
        assert lib.ctr_attn_reset(h, None) == ctr.CTR_ERR_NO_WORKSPACE
        assert lib.ctr_attn_check(h, None) == ctr.CTR_ERR_NO_WORKSPACE
    finally:
        ctr.ctr_attn_destroy(h)
    ctr.ctr_attn_destroy(None)
    assert ctr.lib.ctr_attn_workspace_bytes(None) == 0
    assert ctr.lib.ctr_attn_set_window(None, 0) == ctr.CTR_ERR_INVALID_ARG


def test_attention_calls_refused_before_any_launch(ctr):
    h = ctr.ctr_attn_create(2, 8, 2, 64, 16, 4, ctr.CTR_F16)
    lib, a = ctr.lib, 1 << 20

    def forward(plan=h, q=a, qs=512, k=a, v=a, kvs=128, t=a, n=a, wi=None, wo=None, o=a):
        return lib.ctr_attn_forward(plan, q, qs, k, v, kvs, t, n, wi, wo, o, None)

    def evict(plan=h, t=a, n=a, w=a, d=a, dp=4, budget=32, sinks=0, recent=0, s=a, lo=a + 64,
              wo=a + 64, wp=32):
        return lib.ctr_attn_evict(plan, t, n, w, d, dp, budget, sinks, recent, s, lo, wo, wp, None)

    try:
        bad = ctr.CTR_ERR_INVALID_ARG
        for kw in (dict(plan=None), dict(q=None), dict(t=None), dict(n=None), dict(o=None),
                   dict(v=None), dict(qs=511), dict(kvs=127), dict(wi=a), dict(wo=a)):
            assert forward(**kw) == bad, kw
        for kw in (dict(q=a + 8), dict(k=a + 2), dict(o=a + 4), dict(t=a + 2), dict(qs=513),
                   dict(kvs=132)):
            assert forward(**kw) == ctr.CTR_ERR_MISALIGNED, kw
        for kw in (dict(plan=None), dict(t=None), dict(n=None), dict(w=None), dict(d=None),
                   dict(s=None), dict(lo=None), dict(lo=a), dict(wo=a), dict(budget=0),
                   dict(sinks=-1), dict(recent=33), dict(sinks=20, recent=13), dict(dp=1),
                   dict(wp=31)):
            assert evict(**kw) == bad, kw
        assert evict(w=a + 2) == ctr.CTR_ERR_MISALIGNED
        assert evict(budget=1 << 29, dp=1 << 40, wp=1 << 30) == ctr.CTR_ERR_UNSUPPORTED
        # No cache bound; then no workspace; then not reset.
        assert forward() == evict() == ctr.CTR_ERR_NOT_PREPARED
        ctr.ctr_attn_bind_cache(h, a, a, 8)
        assert forward() == evict() == ctr.CTR_ERR_NO_WORKSPACE
        ctr.ctr_attn_bind_workspace(h, a, 1 << 30)
        assert forward() == evict() == ctr.CTR_ERR_NOT_PREPARED
    finally:
        ctr.ctr_attn_destroy(h)


def test_sampler_calls_refused_before_any_launch(ctr):
    lib, a, bad = ctr.lib, 1 << 20, ctr.CTR_ERR_INVALID_ARG
    h = P(1)
    for args, status in (((-1, 5, 0), bad), ((1, 0, 0), bad), ((1, 5, 9), bad),
                         ((1, (1 << 20) + 1, 0), ctr.CTR_ERR_UNSUPPORTED),
                         (((1 << 20) + 1, 1, 0), ctr.CTR_ERR_UNSUPPORTED)):
        assert lib.ctr_sampler_create(ctypes.byref(h), *args) == status
        assert not h.value
    h = ctr.ctr_sampler_create(4, 100, ctr.CTR_BF16)

    def forward(plan=h, x=a, xs=100, e=a, es=100, T=None, k=None, p=None, mp=None, o=a):
        return lib.ctr_sampler_forward(plan, x, xs, e, es, T, k, p, mp, o, None)

    try:
        assert "bf16" in ctr.ctr_sampler_describe(h) and "vocab=100" in ctr.ctr_sampler_describe(h)
        for kw in (dict(plan=None), dict(x=None), dict(e=None), dict(o=None), dict(xs=99),
                   dict(es=99)):
            assert forward(**kw) == bad, kw
        for kw in (dict(x=a + 1), dict(e=a + 2), dict(T=a + 2), dict(k=a + 1), dict(p=a + 2),
                   dict(mp=a + 3), dict(o=a + 4)):
            assert forward(**kw) == ctr.CTR_ERR_MISALIGNED, kw
    finally:
        ctr.ctr_sampler_destroy(h)
    ctr.ctr_sampler_destroy(None)
    h = ctr.ctr_sampler_create(0, 100, ctr.CTR_F32)
    try:
        assert forward(plan=h, x=None, e=None, o=None) == ctr.CTR_OK     # no rows: nothing to do
    finally:
        ctr.ctr_sampler_destroy(h)
