"""sv_kv_pages on the GPU against the oracle, which moves one page at a time:
whole numbers, compared exactly."""
import numpy as np
import pytest
import torch

import draft_token_verification_spec_amd as sv
from oracle import serve as osv
from test_gpu_kv import I32

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a HIP device")]


class Pool:
    """A cache's pages on the device and in the oracle."""

    def __init__(self, B, max_pages, num_pages, size, seed=0, shared=None):
        self.size, self.capacity, self.shared = size, num_pages, shared
        order = np.random.default_rng(seed).permutation(num_pages).tolist()
        self.table, self.held, self.free = [[-1] * max_pages for _ in range(B)], [0] * B, order
        self.upload()

    def upload(self):
        wide = torch.full((len(self.table), len(self.table[0]) + 3), -5, dtype=torch.int32, device="cuda")
        self.d_table = wide[:, 1:-2]  # rows farther apart than their entries
        self.d_table.copy_(I32(self.table))
        self.wide = wide
        self.d_held, self.d_count = I32(self.held), I32([len(self.free)])
        self.d_free = I32(self.free + [-9] * (self.capacity - len(self.free)))

    def step(self, kv_len, start=None, rows=0, **kw):
        shared = None if self.shared is None else I32(self.shared)
        out = {}
        if start is not None:
            out = {n: torch.full((rows,), -77, dtype=torch.int64, device="cuda") for n in ("slots", "positions")}
        o = sv.sv_kv_pages(self.d_table, self.d_held, self.d_free, self.d_count, I32(kv_len), page_size=self.size,
                           shared_pages=shared, query_start=None if start is None else I32(start), rows=rows, out=out, **kw)
        granted = osv.pages(self.table, self.held, self.free, kv_len, self.size, self.capacity, self.shared)
        assert o["granted"].tolist() == granted
        assert self.d_held.tolist() == self.held and self.d_count.tolist() == [len(self.free)]
        assert self.d_free[:len(self.free)].tolist() == self.free
        assert np.array_equal(self.d_table.cpu().numpy(), np.array(self.table))
        assert (self.wide[:, 0] == -5).all() and (self.wide[:, -2:] == -5).all()
        if start is not None:
            where, place = osv.slots(self.table, self.held, kv_len, start, self.size, self.capacity)
            inside = slice(start[0], start[-1])
            assert o["slots"][inside].tolist() == where and o["positions"][inside].tolist() == place
            for n in ("slots", "positions"):  # rows of no request
                assert (o[n][:start[0]] == -77).all() and (o[n][start[-1]:] == -77).all()
        return granted


@pytest.mark.parametrize("B,max_pages,num_pages,size,rows_each", [
    (1, 40, 33, 16, 5), (7, 9, 30, 4, 3), (256, 20, 2000, 16, 5), (1000, 12, 5000, 1, 2), (1024, 6, 4000, 64, 8),
    (1025, 6, 4000, 64, 8), (3000, 5, 9000, 2, 1), (3, 5000, 9000, 8, 6000), (2, 1, 1, 65536, 0),
])
def test_steps_of_a_pool(B, max_pages, num_pages, size, rows_each):
    """Lengths up and down for several steps, with a pool that is too small at times, rows before and behind."""
    rng = np.random.default_rng(B)
    pool = Pool(B, max_pages, num_pages, size, seed=B)
    refused = 0
    for step in range(7):
        most = min(max_pages * size, int(2.2 * num_pages * size / B) + 2) if step % 3 else max_pages * size // 2 + 1
        kv_len = rng.integers(-1, most + 1, B)
        kv_len[rng.random(B) < 0.2] = 0
        new = rng.integers(0, rows_each + 1, B)
        start = (np.cumsum([0] + list(new)) + 3).tolist()
        granted = pool.step(kv_len.tolist(), start, start[-1] + 5)
        refused += B - sum(granted)
    assert refused or B * max_pages <= 3 * num_pages  # (lengths are half of what a row holds on average)


def test_taking_is_undone_by_giving_back():
    """The lengths of before put every array back, entry by entry, whatever was taken in between."""
    for B, T in ((300, 0), (300, 9000), (2000, 0)):
        pool = Pool(B, 30, 20 * B, 16)
        before = np.random.default_rng(1).integers(0, 200, B)
        pool.step(before.tolist())
        state = [x.clone() for x in (pool.d_table, pool.d_held, pool.d_free, pool.d_count)]
        start = np.minimum(np.arange(B + 1) * 30, T).tolist()
        assert all(pool.step((before + 30).tolist(), start, T))
        pool.step(before.tolist())
        for x, y in zip(state, (pool.d_table, pool.d_held, pool.d_free, pool.d_count)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("B", [5, 1500])
def test_shared_pages_are_kept(B):
    pool = Pool(B, 20, 40 * B, 8, shared=[4] * B)
    pool.step([100] * B)
    pool.step([0] * B)  # down to the shared ones
    assert pool.held == [4] * B
    pool.step([33, 12] * (B // 2) + [70] * (B % 2))
    pool.shared = [-3, 0, 50, 1, 2] + [3] * (B - 5)
    pool.step([9] * B)
    pool.step([160] * B)


@pytest.mark.parametrize("B", [6, 1100])
def test_lengths_beyond_the_table_and_the_pool(B):
    """2^31 - 1 tokens, a row of the table too short, an empty pool, one page short of enough."""
    pool = Pool(B, 8, 7 * B, 16)
    assert pool.step([2 ** 31 - 1, 129, 128] + [-2 ** 31, 1, 16] + [5] * (B - 6)) == [0, 0, 1, 1, 1, 1] + [1] * (B - 6)
    assert pool.step([0, 2 ** 31 - 1] + [128] * (B - 2))[1] == 0
    assert 0 in pool.step([128] * B)  # (the pool has 7 pages for each)
    empty = Pool(3, 4, 0, 16)
    assert empty.step([0, 1, 64], [0, 0, 1, 2], 2) == [1, 0, 0]


@pytest.mark.parametrize("B", [4, 1030])
def test_arrays_that_do_not_fit_together(B):
    """Held pages beyond the row, negative ones, a count beyond the stack, pages of no cache: nothing is touched outside
    the arrays, slots of bad pages are absent."""
    pool = Pool(B, 4, 4 * B, 4)
    pool.step([9] * B)
    pool.held[0], pool.held[1] = 4, 4  # (their fourth entries are -1)
    pool.upload()
    pool.d_held[0], pool.d_held[1] = 100, 4
    pool.step([16, 2] + [9] * (B - 2), [0, 16, 18] + [18] * (B - 2), 18)
    assert -1 in pool.free
    pool.d_held[2] = -7
    pool.held[2] = 0
    pool.step([16, 2, 3] + [9] * (B - 3))
    pool.table[3][1] = 4 * B  # beyond the cache
    pool.upload()
    pool.step([16, 2, 3, 9] + [9] * (B - 4), [0, 0, 0, 0, 9] + [9] * (B - 4), 9)
    pool.free = pool.free + [0] * (4 * B - len(pool.free))
    pool.upload()
    pool.d_count[0] = 2 ** 30
    pool.step([0] * B)  # what is given back finds no place


def test_rows_that_start_nowhere():
    """query_start beyond the rows, and descending: nothing outside [0, T) is written."""
    pool = Pool(3, 10, 30, 4)
    for start, rows in (([-4, 2, 5, 9], 7), ([5, 2, 8, 8], 8), ([0, 2, 5, 9], 9000), ([-4, 2, 5, 90000], 8500)):
        o = {n: torch.full((rows + 8,), -77, dtype=torch.int64, device="cuda") for n in ("slots", "positions")}
        v = {n: x[4:4 + rows] for n, x in o.items()}
        sv.sv_kv_pages(pool.d_table, pool.d_held, pool.d_free, pool.d_count, I32([10, 11, 12]), page_size=4,
                       query_start=I32(start), rows=rows, out=v)
        for x in o.values():
            assert (x[:4] == -77).all() and (x[4 + rows:] == -77).all()
        if start[1:3] == [2, 5]:
            assert v["positions"][2:5].tolist() == [8, 9, 10]


def test_steps_captured():
    """A captured step replayed as lengths and the pool go on changing: the same as eager steps of the oracle."""
    for B, T in ((200, 1000), (1500, 7500)):
        pool = Pool(B, 30, 12 * B, 8, seed=3)
        kv_len, start = I32([0] * B), (np.arange(B + 1) * (T // B)).tolist()
        qs = I32(start)
        call = lambda: sv.sv_kv_pages(pool.d_table, pool.d_held, pool.d_free, pool.d_count, kv_len, page_size=8,
                                      query_start=qs, rows=T)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = call()
        rng = np.random.default_rng(5)
        for rep in range(5):
            lens = rng.integers(0, 120, B).tolist()
            kv_len.copy_(I32(lens))
            g.replay()
            torch.cuda.synchronize()
            granted = osv.pages(pool.table, pool.held, pool.free, lens, 8, 12 * B)
            assert o["granted"].tolist() == granted and pool.d_held.tolist() == pool.held
            assert np.array_equal(pool.d_table.cpu().numpy(), np.array(pool.table))
            assert pool.d_free[:len(pool.free)].tolist() == pool.free
            where, place = osv.slots(pool.table, pool.held, lens, start, 8, 12 * B)
            assert o["slots"].tolist() == where and o["positions"].tolist() == place


def test_many_requests_scratch():
    """A scratch of the caller's: what it holds does not matter, nothing beyond it is written, too small is refused."""
    B = 5000
    size = sv.sv_kv_pages_workspace_size(B, 0)
    assert size > 256 and sv.sv_kv_pages_workspace_size(1024, 100) == 256
    ws = torch.full((size + 64,), 255, dtype=torch.uint8, device="cuda")
    pool = Pool(B, 6, 4 * B, 4)
    rng = np.random.default_rng(0)
    for _ in range(3):
        pool.step(rng.integers(0, 25, B).tolist(), workspace=ws[:size])
        assert (ws[size:] == 255).all()
    with pytest.raises(RuntimeError, match="workspace"):
        pool.step([0] * B, workspace=ws[:size - 1])


def test_largest_batch():
    """2^18 requests: up, partly refused, and down."""
    B = 1 << 18
    pool = Pool(B, 3, B, 4, seed=1)
    rng = np.random.default_rng(2)
    first = rng.integers(0, 7, B)
    granted = pool.step(first.tolist())
    assert 0 < sum(granted) < B
    start = np.minimum(np.arange(B + 1) * 2, 100000).tolist()
    pool.step((first // 2).tolist(), start, 100000)
    pool.step([0] * B)
    assert len(pool.free) == B


def test_one_long_context_given_back():
    """Pages of one request by several workgroups, among requests that hold few; and with few rows by one."""
    for rows in (9000, 3):
        pool = Pool(40, 20000, 21000, 16, seed=4)
        pool.step([16 * (i % 5) for i in range(39)] + [16 * 20000 - 3])
        start = np.minimum(np.arange(41) * 230, rows).tolist()
        pool.step([16 * (i % 3) for i in range(39)] + [100], start, rows)


def test_outputs_that_are_not_asked_for():
    """The C call with any of granted, slots and positions missing moves the same pages and writes the others alike."""
    from draft_token_verification_spec_amd import attn

    lens, start, T = [33, 7, 0, 50], [0, 3, 4, 4, 9], 9
    want = Pool(4, 6, 20, 16, seed=2)
    want.step(lens, start, T)
    o = sv.sv_kv_pages(want.d_table, want.d_held, want.d_free, want.d_count, I32(lens), page_size=16, query_start=I32(start),
                       rows=T)
    for asked in range(8):
        pool = Pool(4, 6, 20, 16, seed=2)
        out = [torch.full((n,), -77, dtype=t, device="cuda") for n, t in ((4, torch.int32), (T, torch.int64), (T, torch.int64))]
        ptr = [x.data_ptr() if asked >> i & 1 else None for i, x in enumerate(out)]
        kl, qs = I32(lens), I32(start)
        attn._call(0, "sv_kv_pages", 4, T, 16, 6, 20, kl.data_ptr(), None, qs.data_ptr(), pool.d_table.data_ptr(),
                   pool.d_table.stride(0), pool.d_held.data_ptr(), pool.d_free.data_ptr(), pool.d_count.data_ptr(), *ptr, None, 0)
        assert torch.equal(pool.d_table, want.d_table) and torch.equal(pool.d_held, want.d_held)
        for i, n in enumerate(("granted", "slots", "positions")):
            assert torch.equal(out[i], o[n]) if asked >> i & 1 else (out[i] == -77).all(), (asked, n)
