"""GPU: the rows of fs_pages_update: none wanted, arrays that start anywhere, and the sizes at
which the launch changes."""
import ctypes as C

import numpy as np
import pytest

from continuous_transformer_decode_gb300 import fs
from tests import _step_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from continuous_transformer_decode_gb300 import build
    build.build()


def _kernels(call):
    """Launches of a call."""
    import torch
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    n = C.c_size_t()
    assert C.CDLL("libcuda.so.1").cuGraphGetNodes(C.c_void_p(g.raw_cuda_graph()), None, C.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("n,n_pages", [(1, 9), (3, 40000), (1500, 9000)])
def test_a_limit_of_rows_without_arrays_for_them(n, n_pages):
    """No row is written, so no launch is needed for them, and no walk up to the limit."""
    import torch
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    holders, table, lengths, start, status = i32(n_pages), i32(n, 3) - 1, i32(n), i32(n + 1), i32(4)
    grow = i32(n) + 5
    call = lambda most, **rows: fs.fs_pages_update(holders, table, lengths, grow, 4, status, row_start=start,
                                                   max_rows=most, **rows)
    for most in (16385, 2**31 - 1):
        assert _kernels(lambda: call(most)) == 1
        call(most)
        assert status.tolist()[:2] == [0, 5 * n] and start.tolist() == [5 * i for i in range(n + 1)]
        assert (lengths == 5).all() and sorted(table[:, :2].flatten().tolist()) == list(range(2 * n))
        holders.zero_(), table.fill_(-1), lengths.zero_()
    lanes = i32(16385)
    assert _kernels(lambda: call(16385, row_lane=lanes)) == 2
    call(5 * n - 1)
    assert status.tolist()[:2] == [fs.CODES["FS_ERR_SCRATCH"], 5 * n]


def _check(n_pages, n, page, grow, max_rows, off=(0, 0, 0, 0), held=0):
    """A call against the host's allocator, the row arrays `off` elements into their buffers."""
    import torch
    wide = -(-(int(grow.max()) + held) // page) + 1
    rng = np.random.default_rng(n_pages + n + max_rows)
    holders = np.where(rng.random(n_pages) < 0.2, 2, 0).astype(np.int32)
    table, lengths = np.full((n, wide), -1, np.int32), np.zeros(n, np.int32)
    if held:  # a page of its own each, partly filled
        own = np.nonzero(holders == 0)[0][-n:]
        holders[own], table[:, 0], lengths[:] = 1, own, held
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    dev = dict(holders=t(holders), table=t(table), lengths=t(lengths))
    rows = [torch.full((max_rows + 9,), -77, dtype=torch.int64 if i == 3 else torch.int32, device="cuda") for i in range(4)]
    assert all(r.data_ptr() % 16 == 0 for r in rows)
    start, status = t(np.zeros(n + 1, np.int32)), t(np.zeros(4, np.int32))
    args = [r[o:o + max_rows] for r, o in zip(rows, off)]
    fs.fs_pages_update(dev["holders"], dev["table"], dev["lengths"], t(grow), page, status, row_start=start, row_lane=args[0],
                       row_position=args[1], row_length=args[2], row_slot=args[3])
    want = R.pages_update(holders, table, lengths, grow, page, max_rows=max_rows)
    assert want["status"][0] == 0
    got = dict(dev, status=status, row_start=start, row_lane=args[0], row_position=args[1], row_length=args[2], row_slot=args[3])
    for k, v in got.items():
        assert np.array_equal(v.cpu().numpy(), want[k]), k
    for r, o in zip(rows, off):
        assert (r[:o] == -77).all() and (r[o + max_rows:] == -77).all()


def _grow(n, total):
    """What n lanes take, total in all."""
    g = np.full(n, total // n, np.int32)
    g[: total - int(g.sum())] += 1
    return g


@pytest.mark.parametrize("off", [(1, 1, 1, 1), (1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (2, 3, 4, 5)])
@pytest.mark.parametrize("n_pages,max_rows", [(3000, 1001), (40000, 1001), (3000, 5003), (9000, 17001)])
def test_rows_arrays_that_start_anywhere(n_pages, max_rows, off):
    """One block, a cluster for its pages or its rows, and the rows' own kernel."""
    _check(n_pages, 7, 16, _grow(7, max_rows - 6), max_rows, off, held=5)


@pytest.mark.parametrize("n_pages,n,max_rows", [
    (3000, 5, 4096), (3000, 5, 4097), (9000, 5, 16384), (9000, 5, 16385), (32768, 5, 300), (32769, 5, 300),
    (9000, 1024, 4096), (9000, 1025, 4096), (40000, 1024, 16384), (40000, 1025, 16385), (32768 * 8 + 1, 3, 40)])
def test_sizes_at_which_the_launch_changes(n_pages, n, max_rows):
    for rows in (max_rows, max_rows - 3):  # without and with padding
        _check(n_pages, n, 16, _grow(n, rows), max_rows, held=3)
