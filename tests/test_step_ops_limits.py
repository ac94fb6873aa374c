"""The limits that include/fs.h gives for the operators for what differs from request to
request, at them and one past them, and which of fs_pages_update's arrays may be NULL. The
checks come before any CUDA call; the addresses are never read."""
import pytest

from continuous_transformer_decode_gb300 import fs
from tests.test_step_ops_refusals import ARG, lora, pages, refused_by_a_check, rope, sample

TB = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def _built():
    from continuous_transformer_decode_gb300 import build
    build.build()


def passes(rc):
    """Nothing but its addresses is wrong with the call."""
    return rc == ARG and fs.fs_last_error(None) in ("no CUDA device", "not a device pointer")


def test_rows_arrays_may_each_be_null_but_row_start():
    for name in ("lane", "pos", "len", "slot", "keep"):
        assert passes(pages(**{name: None})), name
    assert passes(pages(lane=None, pos=None, len=None, slot=None, rows=2**31 - 1))
    assert pages(start=None) == ARG
    refused_by_a_check()


@pytest.mark.parametrize("call,at,past", [
    (rope, dict(H=65535, qs=65535 * 64, qos=65535 * 64, q=TB, qo=TB), dict(H=65536, qs=65536 * 64, qos=65536 * 64, q=TB, qo=TB)),
    (rope, dict(Hkv=65535, ks=65535 * 64, kos=65535 * 64, k=TB, ko=TB), dict(Hkv=65536, ks=65536 * 64, kos=65536 * 64, k=TB, ko=TB)),
    (lora, dict(K=1 << 24, xs=1 << 24, x=TB, A=2 * TB), dict(K=(1 << 24) + 8, xs=(1 << 24) + 8, x=TB, A=2 * TB)),
    (lora, dict(N=1 << 24, bs=1 << 24, os=1 << 24, base=TB, out=TB, B=2 * TB),
     dict(N=(1 << 24) + 1, bs=(1 << 24) + 1, os=(1 << 24) + 1, base=TB, out=TB, B=2 * TB)),
    (sample, dict(n=2**28 - 1, z=TB, tok=2 * TB, kept=3 * TB), dict(n=2**28, z=TB, tok=2 * TB, kept=3 * TB)),
    (sample, dict(V=1 << 20, ld=1 << 20, z=TB), dict(V=(1 << 20) + 1, ld=(1 << 20) + 1, z=TB)),
    (pages, dict(n_lanes=8192, table=TB, lengths=2 * TB, keep=3 * TB, grow=4 * TB, start=5 * TB),
     dict(n_lanes=8193, table=TB, lengths=2 * TB, keep=3 * TB, grow=4 * TB, start=5 * TB)),
    (pages, dict(max_pages=1 << 16, page=1 << 14, table=TB), dict(max_pages=1 << 16, page=(1 << 14) + 1, table=TB))])
def test_limits(call, at, past):
    assert passes(call(**at)), fs.fs_last_error(None)
    assert call(**past) == ARG
    refused_by_a_check()
