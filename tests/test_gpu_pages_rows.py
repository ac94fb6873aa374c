"""GPU: the rows of fs_pages_update: none wanted."""
import ctypes as C

import pytest

from continuous_transformer_decode_gb300 import fs

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
