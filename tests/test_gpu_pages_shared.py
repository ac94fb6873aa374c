"""GPU: fs_pages_update and pages that several lanes hold: no lane grows into one."""
import pytest

from continuous_transformer_decode_gb300 import fs

pytestmark = pytest.mark.gpu
PAGE = 4
STATE, FULL, SCRATCH = (fs.CODES[f"FS_ERR_{k}"] for k in ("STATE", "KV_FULL", "SCRATCH"))
# (pages of the pool, lanes): one block, a cluster, two lanes a thread
SIZES = [(40, 4), (40000, 4), (5000, 1500)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from continuous_transformer_decode_gb300 import build
    build.build()


class Pool:
    """Lane n - 1 has 6 tokens in pages 3 and 7, lane n - 2 has 8 in 3 and 9, lane 0 has 2 in 11."""

    def __init__(self, n_pages, n):
        import torch
        t = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
        self.n, self.a, self.b = n, n - 1, n - 2
        self.holders, self.table, self.lengths, self.grow, self.keep = t(n_pages), t(n, 3) - 1, t(n), t(n), t(n) + 99
        self.start, self.lane, self.status = t(n + 1), t(20), t(4)
        self.slot = torch.zeros(20, dtype=torch.int64, device="cuda")
        self.table[self.a, :2] = torch.tensor([3, 7])
        self.table[self.b, :2] = torch.tensor([3, 9])
        self.table[0, 0] = 11
        self.lengths[self.a], self.lengths[self.b], self.lengths[0] = 6, 8, 2
        self.holders[3], self.holders[7], self.holders[9], self.holders[11] = 2, 1, 1, 1

    def update(self, max_rows=20, keep=None, **grow):
        import torch
        self.grow.zero_(), self.keep.fill_(99)
        for k, v in grow.items():
            self.grow[getattr(self, k)] = v
        for k, v in (keep or {}).items():
            self.keep[getattr(self, k)] = v
        before = [t.clone() for t in (self.holders, self.table, self.lengths)]
        fs.fs_pages_update(self.holders, self.table, self.lengths, self.grow, PAGE, self.status, keep=self.keep,
                           row_start=self.start, row_lane=self.lane[:max_rows], row_slot=self.slot[:max_rows])
        code = self.status.tolist()[0]
        if code:  # no lane grew
            assert not self.start.any() and (self.lane[:max_rows] == -1).all() and (self.slot[:max_rows] == -1).all()
            if keep is None:
                assert all(torch.equal(x, y) for x, y in zip(before, (self.holders, self.table, self.lengths)))
        return code


@pytest.mark.parametrize("n_pages,n", SIZES)
def test_no_lane_grows_into_a_shared_page(n_pages, n):
    p = Pool(n_pages, n)
    assert p.update(a=1) == 0  # page 7 is its own
    p = Pool(n_pages, n)
    p.holders[7] = 2
    assert p.update(a=1) == STATE and p.status.tolist()[1:3] == [1, 0]
    assert p.update(a=2, b=1) == STATE  # nor does another
    assert p.update(b=4) == 0 and p.lengths[p.b] == 12  # its last page is full: it starts a new one
    assert p.table[p.a].tolist() == [3, 7, -1] and p.lengths[p.a] == 6
    # cut to a shared page's inside, and to its end
    p = Pool(n_pages, n)
    assert p.update(a=1, keep=dict(a=3)) == STATE
    assert p.lengths[p.a] == 3 and p.table[p.a].tolist() == [3, -1, -1] and p.holders[7] == 0  # the cut has happened
    p = Pool(n_pages, n)
    assert p.update(a=1, keep=dict(a=4)) == 0 and p.table[p.a].tolist() == [3, 0, -1]
    assert p.slot.tolist()[:2] == [0, -1] and p.lane.tolist()[:2] == [p.a, -1]


@pytest.mark.parametrize("n_pages,n", SIZES)
def test_a_page_that_the_others_let_go_in_the_same_call(n_pages, n):
    p = Pool(n_pages, n)
    assert p.update(a=2, keep=dict(a=3, b=0)) == 0
    assert p.holders[3] == 1 and p.lengths[p.a] == 5 and p.table[p.b].tolist() == [-1] * 3
    assert p.slot.tolist()[:3] == [15, 0, -1]


@pytest.mark.parametrize("n_pages,n", SIZES)
def test_a_last_page_that_is_none(n_pages, n):
    """Entries outside the pool, and a page that nobody holds, which the next lane would get."""
    for entry, holders in ((-1, 1), (-2, 1), (-2**31, 1), (n_pages, 1), (2**31 - 1, 1), (7, 0)):
        p = Pool(n_pages, n)
        p.table[p.a, 1], p.holders[7] = entry, holders
        assert p.update(a=1) == STATE, entry
        assert p.update() == 0  # a lane that takes nothing
        assert p.update(a=1, keep=dict(a=4)) == 0  # or a new page


@pytest.mark.parametrize("n_pages,n", SIZES)
def test_which_reason_is_given(n_pages, n):
    p = Pool(n_pages, n)
    p.holders[7] = 2
    assert p.update(a=7) == FULL  # past the lane's 12 tokens
    assert p.update(a=5, max_rows=4) == SCRATCH
    assert p.update(a=5) == STATE
    p.table[p.a, 1], p.holders[7], p.holders[20] = 20, 1, 1  # a copy of its own
    assert p.update(a=5) == 0 and p.slot.tolist()[:6] == [82, 83, 0, 1, 2, -1]


def test_captured():
    import torch
    p = Pool(40, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fs.fs_pages_update(p.holders, p.table, p.lengths, p.grow, PAGE, p.status, row_start=p.start, row_slot=p.slot)
    p.grow[p.a] = 1
    for holders, code, length in ((2, STATE, 6), (1, 0, 7), (3, STATE, 7), (1, 0, 8), (2, 0, 9)):
        p.holders[7] = holders
        g.replay()
        assert p.status.tolist()[0] == code and p.lengths[p.a] == length
