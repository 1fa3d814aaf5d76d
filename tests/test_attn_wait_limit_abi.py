"""ctr_attn_set_wait_limit_ns, the host half: any limit is taken, and no plan is refused.  No GPU."""
import pytest


@pytest.fixture(scope="module")
def ctr():
    from transposed_convolution_gb300 import build
    build.build()
    import transposed_convolution_gb300 as t
    t.load_library()
    return t


def test_wait_limit(ctr):
    h = ctr.ctr_attn_create(2, 8, 2, 64, 16, 4, ctr.CTR_F16)
    try:
        before = ctr.ctr_attn_workspace_bytes(h)
        for limit in (0, 1, 10 ** 10, 2 ** 64 - 1):
            ctr.ctr_attn_set_wait_limit_ns(h, limit)
        assert ctr.ctr_attn_workspace_bytes(h) == before
        assert ctr.lib.ctr_attn_set_wait_limit_ns(None, 1) == ctr.CTR_ERR_INVALID_ARG
    finally:
        ctr.ctr_attn_destroy(h)
