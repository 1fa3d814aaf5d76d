"""GPU test of put and forward_chunk on a cache of more than 2^32 elements: the same tokens on its last pages and on
a small cache give the same bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import transposed_convolution_gb300 as ctr  # noqa: E402

PAGES, NEED = 70000, 12


@pytest.mark.parametrize("layout", ["head", "token"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pages_past_two_to_the_32_elements(dtype, layout):
    H_q, H_kv, D, page = 16, 8, 128, 64
    far = torch.tensor([PAGES - 1, 0, 65535, 65536, PAGES - 2, 32767, 32768, 1, 49152, 69000, 65537, 2],
                       dtype=torch.int32, device="cuda")
    assert len(far) == NEED and PAGES * page * H_kv * D > 2 ** 32
    T = NEED * page - 5
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn(T, H_q + 2 * H_kv, D, generator=g, device="cuda").to(dtype)
    q, k, v = qkv.split([H_q, H_kv, H_kv], dim=1)
    rope = ctr.Rotary(D, dtype=dtype)
    positions = torch.arange(T, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(pages, table):
        plan = ctr.PagedAttention(1, H_q, H_kv, D, page, NEED, chunks=True, dtype=dtype, layout=layout,
                                  **pages)
        slots = (table.long() * page)[positions.long() // page] + positions.long() % page
        turned = plan.put(k, v, slots, q=q, positions=positions, rotary=rope)
        out = plan.forward_chunk(turned, table[None].contiguous(), lens, starts)
        step = plan.forward(turned[-1:], table[None].contiguous(), lens + T)
        plan.check()
        return out, step

    shape = (PAGES, H_kv, page, D) if layout == "head" else (PAGES, page, H_kv, D)
    big = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(2)]
    got = run(dict(k_pages=big[0], v_pages=big[1]), far)
    want = run(dict(num_pages=NEED), torch.arange(NEED, dtype=torch.int32, device="cuda"))
    for a, b in zip(got, want):
        assert torch.isfinite(b).all() and torch.equal(a, b)
