"""GPU tests of PagePool: tables, lists, slots and positions have to equal a list-of-lists simulation."""
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import chunk_reference as ref  # noqa: E402
import transposed_convolution_gb300 as ctr  # noqa: E402


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Both:
    """A pool and its simulation, kept equal."""

    def __init__(self, B, page, max_pages, num_pages):
        self.pool = ctr.PagePool(B, page, max_pages, num_pages)
        self.sim = ref.Pool(B, page, max_pages, num_pages)
        self.tables = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = [0] * B
        self.same()

    def same(self):
        n = len(self.sim.free)
        assert self.pool.count.item() == n
        assert self.pool.free[:n].tolist() == self.sim.free
        assert self.tables.tolist() == self.sim.tables

    def reserve(self, counts, rows):
        want = self.sim.reserve(self.lens, counts, rows)
        # Guards on both sides of the outputs that have `rows` rows.
        slots = torch.full((rows + 2,), 77, dtype=torch.int64, device="cuda")
        positions = torch.full((rows + 2,), 77, dtype=torch.int32, device="cuda")
        got = self.pool.reserve(self.tables, i32(self.lens), i32(counts), rows,
                                slots=slots[1:rows + 1], positions=positions[1:rows + 1])
        for a, b in zip(got, want):
            assert a.tolist() == b
        for x in (slots, positions):
            assert x[0] == 77 and x[-1] == 77
        self.same()
        if want[5]:
            with pytest.raises(ctr.CtrError):
                self.pool.check()
        self.pool.check()
        self.lens = want[4]
        return want[0]

    def release(self, keep):
        want = self.sim.release(self.lens, keep)
        assert self.pool.release(self.tables, i32(self.lens), i32(keep)).tolist() == want
        self.same()
        self.pool.check()
        self.lens = want


@pytest.mark.parametrize("B,page,max_pages,num_pages", [
    (1, 1, 1, 1), (3, 4, 5, 15), (7, 16, 9, 40), (64, 20, 8, 300), (257, 3, 7, 1000), (1024, 16, 4, 3000)])
def test_random_steps(B, page, max_pages, num_pages):
    rng = random.Random(B)
    s = Both(B, page, max_pages, num_pages)
    for step in range(12):
        most = rng.choice([1, page, 3 * page])
        counts = [rng.choice([0, 1, rng.randint(0, most)]) for _ in range(B)]
        rows = rng.choice([sum(counts), sum(counts) + 3, max(0, sum(counts) - 2), 2500])
        s.reserve(counts, rows)
        s.release([rng.choice([n, n - 1, rng.randint(-1, n + 2)]) if n >= 0 else 0 for n in s.lens])


def test_refusals_of_requests():
    s = Both(4, 8, 4, 6)
    assert s.reserve([9, 40, -1, 8], 64) == [9, 0, 0, 8]         # 40 is past the table, -1 no count
    assert s.reserve([7, 25, 8, 0], 64) == [7, 0, 0, 0]          # 25 needs 4 pages of 3; first come
    assert s.reserve([0, 8, 0, 9], 10) == [0, 8, 0, 0]           # out of rows
    s.release([-1, 8, 0, 8])
    assert s.lens == [-1, 8, 0, 8]
    assert s.reserve([5, 0, 24, 0], 64) == [0, 0, 24, 0]         # an idle sequence asks for nothing
    assert s.reserve([0, 0, 0, 1], 0) == [0, 0, 0, 0]            # no rows at all


def test_release_and_reserve_give_the_same_pages():
    s = Both(5, 16, 8, 40)
    s.reserve([100, 3, 17, 64, 5], 256)
    tables = s.tables.clone()
    full, keep = list(s.lens), [10, 0, 16, 33, 5]
    s.release(keep)
    s.reserve([a - b for a, b in zip(full, keep)], 256)
    assert torch.equal(s.tables, tables)


def test_all_free_list_and_bad_entries_are_reported():
    pool = ctr.PagePool(2, 4, 4, 8)
    assert pool.free.tolist() == list(range(8))[::-1] and pool.count.item() == 8
    tables = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    # A page number out of range on the list: its slots are -1, and so is its table entry.
    pool.free[7] = 8
    granted, starts, slots, positions, lens = pool.reserve(tables, i32([0, 0]), i32([5, 0]), 6)
    assert granted.tolist() == [5, 0] and tables[0].tolist() == [-1, 1, -1, -1]
    assert slots.tolist() == [-1, -1, -1, -1, 4, -1] and positions.tolist() == [0, 1, 2, 3, 4, 0]
    with pytest.raises(ctr.CtrError) as e:
        pool.check()
    assert e.value.status == ctr.CTR_ERR_INVALID_ARG
    pool.check()
    # More pages than there are: the list stays within its bounds.
    guard = torch.full((6,), 7, dtype=torch.int32, device="cuda")
    pool = ctr.PagePool(2, 4, 4, free=guard[1:5], count=i32([3]))
    tables = i32([[0, 1, 2, 3], [0, 1, 2, 3]])
    assert pool.release(tables, i32([16, 16]), i32([-1, 0])).tolist() == [-1, 0]
    assert pool.count.item() == 4 and guard[0] == 7 and guard[5] == 7
    assert (tables == -1).all()
    with pytest.raises(ctr.CtrError):
        pool.check()
    # A count out of range reads as the nearest one.
    pool = ctr.PagePool(1, 4, 4, free=i32([0, 1]), count=i32([9]))
    assert pool.reserve(i32([[-1] * 4]), i32([0]), i32([9]), 9)[0].tolist() == [0]
    with pytest.raises(ctr.CtrError):
        pool.check()


def test_a_captured_step_replays():
    s = Both(3, 4, 6, 18)
    lens, counts = i32([0, 0, 0]), i32([5, 1, 9])
    outs = [torch.empty(n, dtype=d, device="cuda") for n, d in
            ((3, torch.int32), (4, torch.int32), (16, torch.int64), (16, torch.int32), (3, torch.int32))]
    args = dict(zip(("granted", "starts", "slots", "positions", "lens_out"), outs))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.pool.reserve(s.tables, lens, counts, 16, **args)
        lens.copy_(args["lens_out"])
    for c in ([5, 1, 9], [1, 1, 1], [0, 4, 2]):
        counts.copy_(i32(c))
        want = s.sim.reserve(s.lens, c, 16)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert a.tolist() == b
        s.same()
        s.lens = want[4]


def test_another_stream():
    pool = ctr.PagePool(2, 4, 4, 8)
    tables = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    lens, counts = i32([0, 0]), i32([5, 2])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    got = pool.reserve(tables, lens, counts, 8, stream=side)
    torch.cuda.synchronize()
    assert got[0].tolist() == [5, 2] and got[1].tolist() == [0, 5, 7]
    assert got[2].tolist() == [0, 1, 2, 3, 4, 8, 9, -1]


def test_argument_checks():
    pool = ctr.PagePool(2, 4, 4, 8)
    tables, lens = i32([[0] * 4] * 2), i32([1, 1])
    with pytest.raises(ValueError):
        pool.reserve(tables[:1], lens, lens, 4)
    with pytest.raises(TypeError):
        pool.reserve(tables, lens.long(), lens, 4)
    with pytest.raises(ValueError):
        pool.reserve(tables.t().contiguous().t(), lens, lens, 4)
    with pytest.raises(ctr.CtrError):
        pool.reserve(tables, lens, lens, 4, lens_out=lens)
    with pytest.raises(ctr.CtrError):
        pool.reserve(tables, lens, lens, -1)
    with pytest.raises(ctr.CtrError):
        pool.release(tables, lens, i32([0, 0]), lens_out=lens)
    with pytest.raises(ValueError):
        ctr.PagePool(2, 4, 4)
    with pytest.raises(ValueError):
        ctr.PagePool(2, 4, 4, free=lens)
