"""GPU: fs_pages_update on pools of up to 2^31 - 1 pages."""
import pytest

from continuous_transformer_decode_gb300 import fs

pytestmark = pytest.mark.gpu
MOST = 2**31 - 1


@pytest.fixture(scope="module", autouse=True)
def _built():
    from continuous_transformer_decode_gb300 import build
    build.build()


def _i32(*s, fill=0):
    import torch
    return torch.full(s, fill, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n_pages", [MOST - 32, MOST])
def test_the_last_pages_are_found(n_pages):
    """All pages are somebody's but some at both ends and in the middle."""
    import torch
    holders = _i32(n_pages, fill=3)
    free = [0, 40000, 2**30 + 5, n_pages - 33, n_pages - 2, n_pages - 1]
    holders[torch.tensor(free, device="cuda")] = 0
    table, lengths, start, status, slot = _i32(2, 4, fill=-1), _i32(2), _i32(3), _i32(4), torch.zeros(96, dtype=torch.int64, device="cuda")
    fs.fs_pages_update(holders, table, lengths, torch.tensor([64, 33], dtype=torch.int32, device="cuda"), 16, status,
                       row_start=start, row_slot=slot, max_rows=96)
    assert status.tolist() == [fs.CODES["FS_ERR_KV_FULL"], 97, 7, 6]
    fs.fs_pages_update(holders, table, lengths, torch.tensor([64, 32], dtype=torch.int32, device="cuda"), 16, status,
                       row_start=start, row_slot=slot)
    assert status.tolist() == [0, 96, 6, 6] and table.flatten().tolist() == free + [-1, -1]
    assert slot.tolist() == [16 * p + i for p in free for i in range(16)]
    assert holders[torch.tensor(free, device="cuda")].tolist() == [1] * 6 and int((holders == 3).sum()) == n_pages - 6


def test_all_of_them_at_once():
    """Two lanes of 2^30 and 2^30 - 1 pages take the whole pool and let it go."""
    import torch
    holders, table, lengths = _i32(MOST), _i32(2, 2**30, fill=-1), _i32(2)
    grow, start, status = torch.tensor([2**30, 2**30 - 1], dtype=torch.int32, device="cuda"), _i32(3), _i32(4)
    fs.fs_pages_update(holders, table, lengths, grow, 1, status, row_start=start, max_rows=MOST)
    assert status.tolist() == [0, MOST, MOST, MOST] and start.tolist() == [0, 2**30, MOST]
    step = 2**28
    for at in range(0, 2**31, step):
        got = table.flatten()[at:at + step]
        want = torch.arange(at, at + step, device="cuda")
        if at + step == 2**31:
            assert got[-1] == -1
            got, want = got[:-1], want[:-1]
        assert torch.equal(got.long(), want)
    assert bool((holders == 1).all())
    fs.fs_pages_update(holders, table, lengths, _i32(2), 1, status, keep=_i32(2), row_start=start, max_rows=MOST)
    assert status.tolist() == [0, 0, 0, MOST] and not holders.any() and bool((table == -1).all())
