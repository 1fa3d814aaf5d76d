"""PagedAttention.put refuses a closed rotary plan, which the C call would take for none.  No GPU: the call is
refused before anything is launched, and the cache's plan is not ready for one."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ctr():
    from transposed_convolution_gb300 import build
    build.build()
    import transposed_convolution_gb300 as t
    t.load_library()
    return t


@pytest.mark.parametrize("with_q", [False, True])
def test_a_closed_rotary_plan_is_refused(ctr, with_q):
    plan = ctr.PagedAttention.__new__(ctr.PagedAttention)
    plan.handle = ctr.ctr_attn_create(2, 4, 2, 64, 16, 4, ctr.CTR_F32)
    plan._index, plan.device, plan.dtype = -1, torch.device("cpu"), torch.float32
    plan.H_q, plan.H_kv, plan.D = 4, 2, 64
    plan._put, plan._stream = ctr.load_library().ctr_attn_put, lambda *a: None
    rotary = ctr.Rotary(64, dtype=torch.float32, device="cuda:0")
    x = torch.zeros(3, 8, 64)
    args = (x[:, 4:6], x[:, 6:], torch.arange(3))
    kw = dict(positions=torch.arange(3, dtype=torch.int32), rotary=rotary)
    if with_q:
        kw["q"] = x[:, :4]
    with pytest.raises(ctr.CtrError) as e:
        plan.put(*args, **kw)
    assert e.value.status == ctr.CTR_ERR_NOT_PREPARED      # as far as an open one gets
    rotary.close()
    with pytest.raises(ValueError, match="closed"):
        plan.put(*args, **kw)
    plan.close()
