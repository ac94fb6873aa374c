"""GPU: fs_pages_update against a host's allocator (tests/_step_ref.py); whole numbers,
compared exactly."""
import numpy as np
import pytest

from continuous_transformer_decode_gb300 import fs
from tests import _step_ref as R

pytestmark = pytest.mark.gpu
ROWS = ("row_lane", "row_position", "row_length", "row_slot")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from continuous_transformer_decode_gb300 import build
    build.build()


def _cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Pool:
    """A pool on the GPU beside the same one on the host."""

    def __init__(self, n_pages, n_lanes, wide, page, used=0.0, rng=None):
        self.page = page
        h = np.zeros(n_pages, np.int32)
        if used:
            h[rng.random(n_pages) < used] = 3
        self.host = dict(holders=h, table=np.full((n_lanes, wide), -1, np.int32), lengths=np.zeros(n_lanes, np.int32))
        self.dev = {k: _cuda(v) for k, v in self.host.items()}

    def update(self, grow, keep=None, max_rows=0, stream=None):
        import torch
        n = len(grow)
        grow = np.asarray(grow, np.int32)
        keep = None if keep is None else np.asarray(keep, np.int32)
        out = {k: torch.full((max_rows + 3,), -77, dtype=torch.int64 if k == "row_slot" else torch.int32,
                             device="cuda") for k in ROWS}
        start = torch.full((n + 1,), -77, dtype=torch.int32, device="cuda")
        status = torch.full((4,), -77, dtype=torch.int32, device="cuda")
        fs.fs_pages_update(self.dev["holders"], self.dev["table"], self.dev["lengths"], _cuda(grow), self.page, status,
                           keep=None if keep is None else _cuda(keep), row_start=start,
                           **{k: v[:max_rows] for k, v in out.items()}, stream=stream)
        want = R.pages_update(**self.host, grow=grow, page=self.page, keep=keep, max_rows=max_rows)
        torch.cuda.synchronize()
        for k in ("holders", "table", "lengths"):
            assert np.array_equal(self.dev[k].cpu().numpy(), want[k]), k
            self.host[k] = want[k]
        assert np.array_equal(status.cpu().numpy(), want["status"])
        assert np.array_equal(start.cpu().numpy(), want["row_start"])
        for k in ROWS:
            got = out[k].cpu().numpy()
            assert np.array_equal(got[:max_rows], want[k]), k
            assert (got[max_rows:] == -77).all()
        return want


@pytest.mark.parametrize("page", [1, 3, 16, 24, 100])
@pytest.mark.parametrize("n_lanes,n_pages", [(1, 9), (7, 301), (64, 5000), (1500, 40000)])
def test_growing_and_cutting(page, n_lanes, n_pages):
    rng = np.random.default_rng(page * n_lanes)
    per = max(2, n_pages // n_lanes)
    pool = Pool(n_pages, n_lanes, per + 2, page, 0.3 if n_lanes > 1 else 0.0, rng)
    codes = set()
    for step in range(6):
        keep = rng.integers(0, per * page, n_lanes)
        keep[rng.random(n_lanes) < 0.3] = 0
        grow = rng.integers(0, max(2, per * page // 3), n_lanes)
        grow[rng.random(n_lanes) < 0.2] = 0
        w = pool.update(grow, None if step == 0 else keep, int(grow.sum()) + [0, 5, 130][step % 3])
        codes.add(int(w["status"][0]))
    assert R.OK in codes


def test_decode_steps_over_page_borders():
    pool = Pool(40, 5, 9, 4)
    for step in range(30):
        w = pool.update([1] * 5, max_rows=5)
    assert list(w["status"]) == [0, 5, 0, 0] and list(w["lengths"]) == [30] * 5
    w = pool.update([3] * 5, max_rows=15)  # a page each, and none is left
    assert list(w["status"]) == [R.KV_FULL, 15, 5, 0] and list(w["lengths"]) == [30] * 5
    w = pool.update([3] * 4 + [0], keep=[99] * 4 + [0], max_rows=15)  # one lane goes, four pages taken
    assert list(w["status"]) == [0, 12, 4, 8]
    assert list(w["row_lane"]) == [0] * 3 + [1] * 3 + [2] * 3 + [3] * 3 + [-1] * 3


def test_all_or_nothing():
    pool = Pool(10, 3, 6, 4)
    assert list(pool.update([8, 8, 8], max_rows=24)["status"]) == [0, 24, 6, 10]
    for grow, rows, code in [([9, 9, 0], 24, R.KV_FULL),      # 6 pages wanted, 4 free
                             ([17, 0, 0], 24, R.KV_FULL),     # past the lane's 24 tokens
                             ([4, 4, 4], 11, R.SCRATCH)]:     # more rows than there is room for
        w = pool.update(grow, max_rows=rows)
        assert w["status"][0] == code and list(w["lengths"]) == [8, 8, 8] and (w["row_lane"] == -1).all()
    w = pool.update([2**31 - 1] * 3, keep=[8, 3, 0], max_rows=5)  # counts saturate, the cut happens
    assert list(w["status"]) == [R.KV_FULL, 2**31 - 1, 3 * 2**29, 7] and list(w["lengths"]) == [8, 3, 0]


def test_lengths_of_zero_and_one_and_nothing_at_all():
    pool = Pool(1, 1, 1, 1)
    assert list(pool.update([0], max_rows=0)["status"]) == [0, 0, 0, 1]
    assert list(pool.update([1], max_rows=1)["status"]) == [0, 1, 1, 1]
    assert list(pool.update([1], max_rows=1)["status"]) == [R.KV_FULL, 1, 1, 0]
    assert list(pool.update([1], keep=[0], max_rows=1)["status"]) == [0, 1, 1, 1]
    assert list(pool.update([-5], keep=[-5], max_rows=1)["status"]) == [0, 0, 0, 1]


def test_shared_pages_and_entries_out_of_range():
    """A page of two holders stays taken until both let go; bad table entries are cleared
    and nothing else is touched; a page that nobody holds stays free."""
    pool = Pool(8, 3, 4, 4)
    pool.host["table"][:] = [[2, 5, -1, -1], [2, 8, 9999, -1], [-7, 6, 6, -1]]
    pool.host["holders"][:] = [0, 0, 2, 0, 0, 1, 1, 0]
    pool.host["lengths"][:] = [8, 12, 12]
    pool.dev = {k: _cuda(v) for k, v in pool.host.items()}
    w = pool.update([0, 0, 0], keep=[0, 12, 12])
    assert list(w["holders"]) == [0, 0, 1, 0, 0, 0, 1, 0]
    w = pool.update([4, 0, 0], keep=[9, 0, 0], max_rows=4)  # 6 twice: it goes to 0, not below
    assert list(w["holders"]) == [1, 0, 0, 0, 0, 0, 0, 0] and list(w["status"]) == [0, 4, 1, 8]


def test_lengths_outside_the_lane():
    pool = Pool(20, 2, 4, 4)
    pool.host["lengths"][:] = [1000, -3]
    pool.host["table"][0] = [1, 3, 5, 7]
    pool.host["holders"][[1, 3, 5, 7]] = 1
    pool.dev = {k: _cuda(v) for k, v in pool.host.items()}
    w = pool.update([0, 5], keep=[7, 1], max_rows=6)
    assert list(w["lengths"]) == [7, 5]


def test_large_pool_and_many_lanes():
    rng = np.random.default_rng(3)
    pool = Pool(300001, 8192, 9, 16, 0.5, rng)
    pool.update(rng.integers(0, 60, 8192), max_rows=600000)
    pool.update(rng.integers(0, 9, 8192), keep=rng.integers(0, 80, 8192), max_rows=140000)


def test_long_lane_retired():
    pool = Pool(9000, 2, 8200, 16)
    pool.update([131072, 1], max_rows=131080)
    w = pool.update([3, 131071], keep=[0, 1], max_rows=131080)
    assert w["status"][0] == 0


def test_rows_without_arrays():
    """No row arrays: max_rows limits the rows all the same."""
    import torch
    n = 3
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    holders, table, lengths = t([0] * 9), torch.full((n, 3), -1, dtype=torch.int32, device="cuda"), t([0] * n)
    start, status = t([-1] * (n + 1)), t([-1] * 4)
    fs.fs_pages_update(holders, table, lengths, t([2, 3, 4]), 4, status, row_start=start)
    assert status.tolist() == [R.SCRATCH, 9, 3, 9] and start.tolist() == [0] * 4 and lengths.tolist() == [0] * 3
    fs.fs_pages_update(holders, table, lengths, t([2, 3, 4]), 4, status, row_start=start, max_rows=9)
    assert status.tolist() == [0, 9, 3, 9] and start.tolist() == [0, 2, 5, 9] and table[:, 0].tolist() == [0, 1, 2]


def test_graph_replays_steps():
    """A captured call, replayed: each replay is a step more."""
    import torch
    pool = Pool(64, 4, 10, 4)
    dev = pool.dev
    grow, start = torch.ones(4, dtype=torch.int32, device="cuda"), torch.empty(5, dtype=torch.int32, device="cuda")
    status, slot = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(6, dtype=torch.int64, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fs.fs_pages_update(dev["holders"], dev["table"], dev["lengths"], grow, 4, status, row_start=start, row_slot=slot)
    for step in range(12):
        grow.fill_(1 + step % 2)
        g.replay()
        torch.cuda.synchronize()
        w = R.pages_update(**pool.host, grow=np.full(4, 1 + step % 2), page=4, max_rows=6)
        for k in ("holders", "table", "lengths"):
            assert np.array_equal(dev[k].cpu().numpy(), w[k])
            pool.host[k] = w[k]
        assert np.array_equal(slot.cpu().numpy(), w["row_slot"]) and np.array_equal(status.cpu().numpy(), w["status"])
