"""GPU: the 8-bit paged KV cache (fs_kv_q8_append, fs_kv_q8_read,
fs_kv_q8_attention) against its definition in 64 bits (tests/_q8_ref.py).

Codes are compared exactly: a code is the rounding of the real quotient. The
scale is one f32 rounding of amax / 127; a rotated key's amax is f32 first, three
roundings of a pair no larger than sqrt(2) amax, so 2^-21 relative. Read values
are one f32 product (and one bf16 rounding): compared bit for bit. Attention:
the bound that _q8_ref.attention derives, and half a bf16 step (2^-9 of the next
power of two, at most 2^-8 relative) for bf16 outputs.
"""
import numpy as np
import pytest

from continuous_transformer_decode_gb300 import fs
from tests import _q8_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from continuous_transformer_decode_gb300 import build
    build.build()


def _cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Pages:
    """A cache of random codes and scales on the device, and its page table: lane
    l has room for cap[l] tokens in scattered pages (entries beyond: -1)."""

    def __init__(self, rng, cap, Hkv, hd, ps, spare=2, scale=0.02):
        need = [-(-c // ps) for c in cap]
        self.n_pages = sum(need) + spare
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(cap), max(1, max(need))), -1, np.int32)
        at = 0
        for l, m in enumerate(need):
            self.table[l, :m] = order[at:at + m]
            at += m
        shape = (self.n_pages, Hkv, ps, hd)
        self.host = [rng.integers(1, 256, shape).astype(np.uint8) for _ in range(2)]
        self.host += [(scale * rng.uniform(0.3, 1.7, shape[:3])).astype(np.float32)
                      for _ in range(2)]
        self.dev = [_cuda(a) for a in self.host]
        self.d_table = _cuda(self.table)
        self.view = fs.fs_kv_q8_view(*self.dev, self.d_table)

    def ref(self):
        return R.Cache(*self.host, self.table)

    def now(self):
        return R.Cache(*[d.cpu().numpy() for d in self.dev], self.table)


def _attend(pages, q, lanes, lens, rope=None, max_len=0, split_len=0, scale=None, stream=None):
    import torch
    out = torch.full_like(q, 7.0)
    need = fs.fs_kv_q8_attention_workspace(pages.view, len(lens), q.shape[1], max_len, split_len)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # any content
    fs.fs_kv_q8_attention(pages.view, q, _cuda(np.int32(lanes)), _cuda(np.int32(lens)), out,
                          max_len=max_len, split_len=split_len, rope=rope, workspace=ws,
                          scale=scale, stream=stream)
    torch.cuda.synchronize()
    return out


def _check_attention(got, ref, tol):
    import torch
    bf = got.dtype == torch.bfloat16
    got = got.float().cpu().numpy().astype(np.float64)
    if bf:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    bad = np.abs(got - ref) > tol
    assert np.isfinite(got).all()
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - ref).max(), tol.max())


# ---------------------------------------------------------------- write and read
@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("io,Hkv,ps,n,rope", [
    ("f32", 3, 16, 1, True), ("bf16", 1, 1, 37, True), ("f32", 8, 24, 130, False),
    ("bf16", 2, 64, 515, False), ("f32", 2, 7, 2049, True)])
def test_append_then_read(hd, io, Hkv, ps, n, rope):
    import torch
    rng = np.random.default_rng(hd + n)
    L = 5
    pg = Pages(rng, [n // L + 40] * L, Hkv, hd, ps)
    before = [h.copy() for h in pg.host]
    # distinct (lane, token) pairs in any order
    lane = np.arange(n) % L
    pos = 31 + np.arange(n) // L
    o = rng.permutation(n)
    lane, pos = lane[o].astype(np.int32), pos[o].astype(np.int32)
    x = rng.standard_normal((2, n, Hkv, hd)).astype(np.float32) * 3
    x[:, 0, 0] = 0                                  # a row of zeros
    x[0, n // 2, 0, :] = 1e-38                      # tiny rows
    x[1, n // 2, 0, :] *= 1e30
    if io == "bf16":
        x = R.bf16(x)
        x[1, -1, -1, 0], x[1, -1, -1, 1] = 8.0, 4.0  # 63.5 codes: a tie, if 8 is the largest
        x[1, -1, -1] = np.clip(x[1, -1, -1], -8, 8)
    tables = R.rope_tables(31 + n // L + 1, hd)
    # rows inside a wider panel (the projection's [q | k | v])
    t = torch.float32 if io == "f32" else torch.bfloat16
    panel = torch.zeros(n, 1 + 2 * Hkv, hd, dtype=t, device="cuda")
    panel[:, 1:1 + Hkv] = _cuda(x[0]).to(t)
    panel[:, 1 + Hkv:] = _cuda(x[1]).to(t)
    d_lane, d_pos = _cuda(lane), _cuda(pos)
    fs.fs_kv_q8_append(pg.view, panel[:, 1:1 + Hkv], panel[:, 1 + Hkv:], d_lane, d_pos,
                       rope=tuple(_cuda(a) for a in tables) if rope else None)
    outs = [torch.empty(n, Hkv, hd, dtype=t, device="cuda") for _ in range(2)]
    fs.fs_kv_q8_read(pg.view, d_lane, d_pos, *outs)
    torch.cuda.synchronize()
    after = [d.cpu().numpy() for d in pg.dev]
    k = R.rotate(x[0], tables[0][pos], tables[1][pos]) if rope else x[0]
    page, slot = pg.table[lane, pos // ps], pos % ps
    for which, rows in ((0, k), (1, x[1])):
        codes, scale = R.quantise(rows)
        got = after[which][page, :, slot].astype(np.int64) - 128
        assert np.array_equal(got, codes), np.argwhere(got != codes)[:5]
        gs = after[2 + which][page, :, slot]
        rel = 2.0 ** -21 if rope and which == 0 else 2.0 ** -23
        assert (np.abs(gs - scale) <= rel * scale + 2.0 ** -149).all()
        want = got.astype(np.float32) * gs[..., None]
        if io == "bf16":
            want = R.bf16(want)
        assert np.array_equal(outs[which].float().cpu().numpy(), want)
        # every other slot is as it was
        after[which][page, :, slot] = before[which][page, :, slot]
        after[2 + which][page, :, slot] = before[2 + which][page, :, slot]
    for a, b in zip(after, before):
        assert np.array_equal(a, b)


def test_append_ties_and_borders():
    """Quotients that lie on a border of two codes go to the even one, for every
    code and for scales of many magnitudes."""
    import torch
    n = 64
    rng = np.random.default_rng(5)
    pg = Pages(rng, [n], 1, 128, 16)
    x = np.zeros((n, 1, 128), np.float32)
    for i in range(n):
        a = 2.0 ** (i - 32) * 127.0
        x[i, 0, 0] = a
        x[i, 0, 1:] = (np.arange(127) - 63 + 0.5) * 2.0 ** (i - 32)  # codes k + 1/2
    x[1::2, 0, 1:] *= np.float32(1 + 2.0 ** -23)                     # a bit above them
    x[1::4] *= -1
    lane, pos = np.zeros(n, np.int32), np.arange(n, dtype=np.int32)
    xx = _cuda(x)
    fs.fs_kv_q8_append(pg.view, xx, xx, _cuda(lane), _cuda(pos))
    torch.cuda.synchronize()
    codes, _ = R.quantise(x)
    for d in pg.dev[:2]:
        got = d.cpu().numpy()[pg.table[0, pos // 16], :, pos % 16].astype(np.int64) - 128
        assert np.array_equal(got, codes)


def test_append_not_finite():
    import torch
    rng = np.random.default_rng(6)
    pg = Pages(rng, [4], 1, 64, 4)
    x = rng.standard_normal((4, 1, 64)).astype(np.float32)
    x[0, 0, 3], x[1, 0, 5], x[2, 0, 7] = np.nan, np.inf, -np.inf
    x[3] = np.nan
    xx = _cuda(x)
    fs.fs_kv_q8_append(pg.view, xx, xx, _cuda(np.zeros(4, np.int32)), _cuda(np.arange(4, dtype=np.int32)))
    torch.cuda.synchronize()
    codes, scale = R.quantise(x)
    got = pg.dev[0].cpu().numpy()[pg.table[0, 0], 0].astype(np.int64) - 128
    assert np.array_equal(got, codes[:, 0])
    assert np.isfinite(pg.dev[2].cpu().numpy()).all()
    assert np.allclose(pg.dev[2].cpu().numpy()[pg.table[0, 0], 0], scale[:, 0], rtol=2.0 ** -22)


@pytest.mark.parametrize("base", [-97, 0, 92])
def test_codes_of_every_bf16_quotient(base):
    """Rows of bf16 as they came: every significand over every largest one, a
    quotient of up to 127 down to a quarter of a code, both signs. Exact codes: a
    quotient is a tie or 1.5e-5 of itself away from one, which 64 bits tell apart."""
    import torch
    A, X = np.arange(128, 256), np.arange(128, 256)
    rows = []
    for e in range(11):
        x = np.where((X[None] <= A[:, None]) | (e > 0), X[None] * 2.0 ** -e, 0.0)
        row = np.concatenate([x, -x], 1)
        row[:, 127] = A  # the largest magnitude
        rows.append(row)
    x = (np.concatenate(rows) * 2.0 ** base).astype(np.float32)[:, None]
    assert np.array_equal(R.bf16(x), x)
    n = len(x)
    pg = Pages(np.random.default_rng(3), [n], 1, 256, 64)
    v = _cuda(x).to(torch.bfloat16)
    at = _cuda(np.zeros(n, np.int32)), _cuda(np.arange(n, dtype=np.int32))
    fs.fs_kv_q8_append(pg.view, v, -v, *at)
    torch.cuda.synchronize()
    codes, _ = R.quantise(x)
    t = np.arange(n)
    for which, want in ((0, codes), (1, -codes)):
        got = pg.dev[which].cpu().numpy()[pg.table[0, t // 64], :, t % 64].astype(np.int64) - 128
        assert np.array_equal(got, want), np.argwhere(got != want)[:5]


@pytest.mark.parametrize("hd", [64, 256])
def test_infinities_read_back_finite(hd):
    """An infinity is stored as the largest finite f32, and so is read back finite:
    the scale's rounding does not take 127 of it past the range."""
    import torch
    rng = np.random.default_rng(7)
    pg = Pages(rng, [3], 2, hd, 4)
    big = float(np.finfo(np.float32).max)
    x = rng.standard_normal((3, 2, hd)).astype(np.float32)
    x[0, 0, 3], x[1, 1, hd - 1], x[2, 0, 0], x[2, 1, 1] = np.inf, -np.inf, big, -3.4e38
    xx, out = _cuda(x), [torch.zeros(3, 2, hd, device="cuda") for _ in range(2)]
    at = _cuda(np.zeros(3, np.int32)), _cuda(np.arange(3, dtype=np.int32))
    fs.fs_kv_q8_append(pg.view, xx, xx, *at)
    fs.fs_kv_q8_read(pg.view, *at, *out)
    torch.cuda.synchronize()
    codes, scale = R.quantise(x)
    for o in out:
        got = o.cpu().numpy().astype(np.float64)
        assert np.isfinite(got).all()
        want = codes * scale[..., None]
        # the scale within 2^-23 of the quotient, one product rounded
        assert (np.abs(got - want) <= 2.0 ** -22 * np.abs(want)).all()


def test_rows_outside_the_cache():
    """Padding rows (-1), lanes and positions outside, positions past the
    rotation tables, page-table entries of no page: nothing is written, zeros are
    read, no weight is given."""
    import torch
    rng = np.random.default_rng(8)
    pg = Pages(rng, [40, 40], 2, 64, 16)
    pg.table[0, 1] = pg.n_pages          # tokens 16 .. 31 of lane 0 have no page
    pg.table[1, 0] = -7
    pg.d_table.copy_(_cuda(pg.table))
    before = [h.copy() for h in pg.host]
    lane = np.array([0, 2, -1, 0, 0, 0, 1, 0, 0, 1], np.int32)
    pos = np.array([-1, 3, 3, 48, 1 << 30, 17, 2, 2, 39, 20], np.int32)
    good = [7, 9]                        # (0, 2) and (1, 20); (0, 39) is past the tables below
    x = rng.standard_normal((len(lane), 2, 64)).astype(np.float32)
    tables = R.rope_tables(39, 64)
    fs.fs_kv_q8_append(pg.view, _cuda(x), _cuda(x), _cuda(lane), _cuda(pos),
                       rope=tuple(_cuda(a) for a in tables))
    out = torch.full((len(lane), 2, 64), 9.0, device="cuda")
    fs.fs_kv_q8_read(pg.view, _cuda(lane), _cuda(pos), v_out=out)
    torch.cuda.synchronize()
    codes, _ = R.quantise(x)
    after = [d.cpu().numpy() for d in pg.dev]
    out = out.cpu().numpy()
    for i in range(len(lane)):
        if i in good:
            p, s = pg.table[lane[i], pos[i] // 16], pos[i] % 16
            assert np.array_equal(after[1][p, :, s].astype(np.int64) - 128, codes[i])
            for w in range(4):
                after[w][p, :, s] = before[w][p, :, s]
        elif i != 8:
            assert (out[i] == 0).all()
    for a, b in zip(after, before):
        assert np.array_equal(a, b)
    # attention: absent tokens have no weight; rows of no lane and of no token are zero
    pg.host = [d.cpu().numpy() for d in pg.dev]
    lanes, lens = [0, 1, 2, -1, 0, 1, 1], [40, 40, 40, 40, 0, 16, -3]
    q = rng.standard_normal((7, 4, 64)).astype(np.float32)
    for split in (0, 64):
        got = _attend(pg, _cuda(q), lanes, lens, split_len=split)
        ref, tol = R.attention(pg.ref(), q, lanes, lens, 0.125)
        assert (ref[2:] == 0).all()
        _check_attention(got, ref, tol)


# ------------------------------------------------------------------- attention
CASES = [  # Hkv, G, hd, page_size, io, rope, lengths, split_len
    (1, 1, 64, 16, "f32", False, [1], 0),
    (3, 3, 64, 16, "f32", True, [17, 0, 1, 64, 65, 500], 0),
    (2, 8, 64, 1, "bf16", True, [63, 64, 130, 2], 64),
    (8, 4, 128, 16, "bf16", True, [1, 15, 16, 17, 300, 0, 1025], 0),
    (8, 4, 128, 16, "f32", False, [777, 64, 128, 129], 128),
    (1, 7, 128, 100, "f32", True, [99, 100, 101, 1500], 64),
    (2, 2, 128, 7, "bf16", False, [3, 700], 0),
    (2, 8, 256, 24, "f32", True, [5, 48, 601, 1], 0),
    (1, 5, 256, 64, "bf16", True, [64, 65, 333], 192),
    (4, 1, 256, 8, "f32", False, [2, 9, 130], 64),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attention(case):
    import torch
    Hkv, G, hd, ps, io, rope, lens, split = case
    rng = np.random.default_rng(hd * 7 + ps)
    pg = Pages(rng, [l + 3 for l in lens], Hkv, hd, ps)
    # the slots that no lane's length reaches hold scales of no number
    used = np.zeros(pg.host[2].shape[:1] + (ps,), bool)
    for l, n in enumerate(lens):
        t = np.arange(n)
        used[pg.table[l, t // ps], t % ps] = True
    for w in (2, 3):
        pg.host[w][np.broadcast_to(~used[:, None, :], pg.host[w].shape)] = np.nan
        pg.dev[w].copy_(_cuda(pg.host[w]))
    q = (3 * rng.standard_normal((len(lens), Hkv * G, hd))).astype(np.float32)
    if io == "bf16":
        q = R.bf16(q)
    tables = R.rope_tables(max(lens) + 1, hd) if rope else None
    t = torch.float32 if io == "f32" else torch.bfloat16
    got = _attend(pg, _cuda(q).to(t), range(len(lens)), lens,
                  rope=tuple(_cuda(a) for a in tables) if rope else None, max_len=max(lens),
                  split_len=split)
    ref, tol = R.attention(pg.ref(), q, range(len(lens)), lens, hd ** -0.5, tables)
    _check_attention(got, ref, tol)


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_attention_large_scores_and_scales(hd):
    """Scores in the thousands, values whose scales span 30 orders of magnitude,
    one dominant token, an all-zero key and value."""
    rng = np.random.default_rng(hd)
    lens = [200, 333]
    pg = Pages(rng, lens, 2, hd, 16)
    pg.host[3] *= (10.0 ** rng.uniform(-15, 15, pg.host[3].shape)).astype(np.float32)
    pg.host[2][:, :, 3] = 0
    pg.host[3][:, :, 5] = 0
    for w in (2, 3):
        pg.dev[w].copy_(_cuda(pg.host[w]))
    q = (100 * rng.standard_normal((2, 8, hd))).astype(np.float32)
    q[0, 0], q[0, 1] = 0, 1e-30
    for split in (0, 64):
        got = _attend(pg, _cuda(q), [0, 1], lens, split_len=split)
        ref, tol = R.attention(pg.ref(), q, [0, 1], lens, hd ** -0.5)
        _check_attention(got, ref, tol)


@pytest.mark.parametrize("split", [64, 4096])
def test_a_query_that_is_no_number_stays_in_its_head(split):
    import torch
    rng = np.random.default_rng(12)
    lens = [300, 40]
    pg = Pages(rng, lens, 2, 64, 16)
    q = rng.standard_normal((2, 8, 64)).astype(np.float32)
    ref, tol = R.attention(pg.ref(), q, [0, 1], lens, 0.125)
    q[0, 2, 5], q[0, 7, 0], q[1, 4, 63] = np.nan, np.inf, -np.inf
    got = _attend(pg, _cuda(q), [0, 1], lens, split_len=split)
    bad = torch.zeros(2, 8, dtype=torch.bool)
    bad[0, 2] = bad[0, 7] = bad[1, 4] = True
    assert torch.isnan(got.cpu()[bad]).all()
    # not the same bits: the heads of a KV head set their references together
    _check_attention(got.cpu()[~bad], ref[~bad.numpy()], tol[~bad.numpy()])


def test_attention_takes_rows_by_length():
    """A launch of many long ragged rows: the blocks take them by length; every row
    comes out as in a call of its own. Equal lengths, empty rows and rows past
    max_len among them."""
    import torch
    rng = np.random.default_rng(13)
    n, Hkv = 150, 8
    lens = np.where(rng.random(n) < 0.2, 0, rng.integers(1, 2300, n))
    lens[5:9] = 2100
    pg = Pages(rng, lens.tolist(), Hkv, 128, 16)
    q = _cuda(rng.standard_normal((n, Hkv, 128)).astype(np.float32))
    got = _attend(pg, q, range(n), lens, max_len=2200, split_len=2048)
    for i in list(range(12)) + [n - 1, int(lens.argmax()), int(lens.argmin())]:
        one = _attend(pg, q[i:i + 1], [i], lens[i:i + 1], max_len=2200, split_len=2048)
        assert torch.equal(one[0], got[i]), i
    pick = [0, 5, 77, n - 1]
    ref, tol = R.attention(pg.ref(), q.cpu().numpy()[pick], pick, np.minimum(lens[pick], 2200), 128 ** -0.5)
    _check_attention(got[pick], ref, tol)


def test_attention_long_offsets():
    """A cache of more than 2^31 code bytes: rows at both ends of it."""
    import torch
    hd, ps, Hkv = 128, 64, 8
    n_pages = (1 << 31) // (hd * ps * Hkv) + 40
    codes = [torch.full((n_pages, Hkv, ps, hd), 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((n_pages, Hkv, ps), 0.01, device="cuda") for _ in range(2)]
    table = np.array([[n_pages - 1, 0, n_pages - 2], [1, n_pages - 3, 2]], np.int32)
    view = fs.fs_kv_q8_view(*codes, *scales, _cuda(table))
    rng = np.random.default_rng(1)
    lane = np.repeat(np.arange(2, dtype=np.int32), 150)
    pos = np.tile(np.arange(150, dtype=np.int32), 2)
    x = rng.standard_normal((2, 300, Hkv, hd)).astype(np.float32)
    fs.fs_kv_q8_append(view, _cuda(x[0]), _cuda(x[1]), _cuda(lane), _cuda(pos))
    q = rng.standard_normal((2, 16, hd)).astype(np.float32)
    out = torch.empty(2, 16, hd, device="cuda")
    ws = torch.empty(fs.fs_kv_q8_attention_workspace(view, 2, 16, 150), dtype=torch.uint8, device="cuda")
    fs.fs_kv_q8_attention(view, _cuda(q), _cuda(np.int32([0, 1])), _cuda(np.int32([150, 149])), out,
                          max_len=150, workspace=ws)
    got = torch.empty(300, Hkv, hd, device="cuda")
    fs.fs_kv_q8_read(view, _cuda(lane), _cuda(pos), got)
    torch.cuda.synchronize()
    ck, sk = R.quantise(x[0])
    assert np.allclose(got.cpu().numpy(), ck * sk[..., None], rtol=2.0 ** -22, atol=0)
    pick = sorted(set(table.ravel().tolist()))
    small = {p: i for i, p in enumerate(pick)}
    ref = R.Cache(*[c[pick].cpu().numpy() for c in codes], *[s[pick].cpu().numpy() for s in scales],
                  np.vectorize(small.get)(table))
    want, tol = R.attention(ref, q, [0, 1], [150, 149], hd ** -0.5)
    _check_attention(out, want, tol)


def test_attention_row_bits_do_not_depend_on_the_batch():
    import torch
    rng = np.random.default_rng(3)
    lens = [900, 70, 333, 128, 5]
    pg = Pages(rng, lens, 2, 128, 16)
    q = _cuda(rng.standard_normal((5, 8, 128)).astype(np.float32))
    full = _attend(pg, q, range(5), lens, split_len=128)
    for i in range(5):
        one = _attend(pg, q[i:i + 1], [i], lens[i:i + 1], split_len=128)
        assert torch.equal(one[0], full[i])
    again = _attend(pg, q, range(5), lens, split_len=128)
    assert torch.equal(again, full)


def test_attention_rows_of_one_lane_and_capped_lengths():
    """Rows of a drafted continuation name one lane, each with its own length; a
    length past the capacity or past max_len reads what there is."""
    rng = np.random.default_rng(4)
    pg = Pages(rng, [96], 2, 64, 16)
    q = rng.standard_normal((4, 4, 64)).astype(np.float32)
    got = _attend(pg, _cuda(q), [0] * 4, [93, 94, 95, 10000])
    ref, tol = R.attention(pg.ref(), q, [0] * 4, [93, 94, 95, 96], 0.125)
    _check_attention(got, ref, tol)
    got = _attend(pg, _cuda(q), [0] * 4, [93, 20, 95, 10000], max_len=50)
    ref, tol = R.attention(pg.ref(), q, [0] * 4, [50, 20, 50, 50], 0.125)
    _check_attention(got, ref, tol)


def test_strided_rows_are_left_alone_between():
    import torch
    rng = np.random.default_rng(9)
    pg = Pages(rng, [200], 2, 128, 16)
    q = rng.standard_normal((1, 4, 128)).astype(np.float32)
    wide_q = torch.zeros(3, 6, 128, device="cuda")
    wide_q[:, 1:5] = _cuda(q)
    wide_o = torch.full((3, 6, 128), 5.0, device="cuda")
    ws = torch.empty(fs.fs_kv_q8_attention_workspace(pg.view, 3, 4, 200, 64), dtype=torch.uint8, device="cuda")
    fs.fs_kv_q8_attention(pg.view, wide_q[:, 1:5], _cuda(np.zeros(3, np.int32)),
                          _cuda(np.int32([200, 3, 0])), wide_o[:, 1:5], max_len=200, split_len=64,
                          workspace=ws)
    torch.cuda.synchronize()
    assert (wide_o[:, 0] == 5).all() and (wide_o[:, 5] == 5).all()
    ref, tol = R.attention(pg.ref(), np.repeat(q, 3, 0), [0, 0, 0], [200, 3, 0], 128 ** -0.5)
    _check_attention(wide_o[:, 1:5], ref, tol)


def test_graphs_and_streams():
    """Append and attention captured into two graphs with a workspace each,
    replayed at once on two streams; page table and lengths change between
    replays."""
    import torch
    rng = np.random.default_rng(11)
    pg = Pages(rng, [300, 300, 300, 300], 2, 64, 16)
    sides = []
    for s in range(2):
        st = torch.cuda.Stream()
        lanes, lens = _cuda(np.int32([2 * s, 2 * s + 1])), _cuda(np.int32([10, 20]))
        pos, x = lens - 1, _cuda(rng.standard_normal((2, 2, 2, 64)).astype(np.float32))
        q = _cuda(rng.standard_normal((2, 6, 64)).astype(np.float32))
        out = torch.zeros(2, 6, 64, device="cuda")
        ws = torch.empty(fs.fs_kv_q8_attention_workspace(pg.view, 2, 6, 300, 64), dtype=torch.uint8,
                         device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            raw = torch.cuda.current_stream()
            fs.fs_kv_q8_append(pg.view, x[0], x[1], lanes, pos, stream=raw)
            fs.fs_kv_q8_attention(pg.view, q, lanes, lens, out, max_len=300, split_len=64,
                                  workspace=ws, stream=raw)
        sides.append((st, g, lanes, lens, pos, x, q, out))
    for n in ([299, 140], [65, 1], [64, 300]):
        for st, g, lanes, lens, pos, x, q, out in sides:
            with torch.cuda.stream(st):
                lens.copy_(torch.tensor(n, dtype=torch.int32))
                pos.copy_(lens - 1)
                x.normal_()
        torch.cuda.synchronize()
        for _ in range(20):
            for st, g, *_ in sides:
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        ref = pg.now()
        for st, g, lanes, lens, pos, x, q, out in sides:
            want, tol = R.attention(ref, q.cpu().numpy(), lanes.tolist(), lens.tolist(), 0.125)
            _check_attention(out, want, tol)


def test_host_tensors_of_the_c_interface_are_refused():
    rng = np.random.default_rng(1)
    pg = Pages(rng, [16], 1, 64, 16)
    host = np.zeros((1, 64), np.float32)
    one = _cuda(np.zeros(1, np.int32))
    import ctypes as C
    rc = fs.lib().fs_kv_q8_append(C.byref(pg.view), host.ctypes.data, host.ctypes.data, 64, 64, 0,
                                  one.data_ptr(), one.data_ptr(), 1, None, None, 0, None)
    assert rc == fs.CODES["FS_ERR_ARG"]


def test_calls_without_a_stream_run_on_torchs_current_one():
    """Inputs made on a side stream by slow work, the operators called without a
    stream inside it, and the same captured into a graph."""
    import torch
    rng = np.random.default_rng(16)
    pg = Pages(rng, [200, 200], 2, 64, 16)
    kv = rng.standard_normal((2, 2, 2, 64)).astype(np.float32)
    q = rng.standard_normal((2, 4, 64)).astype(np.float32)
    z = rng.standard_normal((2, 300)).astype(np.float32)
    src = {k: _cuda(v) for k, v in dict(
        k=kv[0], v=kv[1], lanes=np.int32([0, 1]), pos=np.int32([150, 20]), lens=np.int32([151, 21]),
        q=q, z=z, start=np.int32([0, 1, 2]), temps=np.float32([0, 0]), u=np.float32([0.5, 0.5])).items()}
    dst = {k: torch.zeros_like(v) for k, v in src.items()}
    ws = torch.zeros(fs.fs_kv_q8_attention_workspace(pg.view, 2, 4, 200, 64), dtype=torch.uint8,
                     device="cuda")
    out, k_out = torch.zeros(2, 4, 64, device="cuda"), torch.zeros(2, 2, 64, device="cuda")
    acc, nxt = (torch.full((2,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    slow = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()

    def step():
        d = dst
        fs.fs_kv_q8_append(pg.view, d["k"], d["v"], d["lanes"], d["pos"])
        fs.fs_kv_q8_read(pg.view, d["lanes"], d["pos"], k_out)
        fs.fs_kv_q8_attention(pg.view, d["q"], d["lanes"], d["lens"], out, max_len=200, split_len=64,
                              workspace=ws)
        fs.fs_verify_draft(d["z"], d["start"], d["lanes"], None, d["temps"], d["u"], d["u"], acc, nxt)

    def look():
        torch.cuda.synchronize()
        codes, scale = R.quantise(kv[0])
        assert np.allclose(k_out.cpu().numpy(), codes * scale[..., None], rtol=2.0 ** -22, atol=0)
        ref, tol = R.attention(pg.now(), q, [0, 1], [151, 21], 0.125)
        _check_attention(out, ref, tol)
        assert np.array_equal(nxt.cpu().numpy(), z.argmax(-1))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(40):
            slow = slow @ slow * 1e-3
        for k in src:
            dst[k].copy_(src[k])
        step()
    look()
    out.zero_(), k_out.zero_(), nxt.fill_(-9)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    g.replay()
    look()


def test_a_failure_of_another_call_is_not_reported_as_this_ones():
    """An allocation that failed before (a handle of more pages than there is
    memory) leaves CUDA's last error set: the operators report their own launches."""
    import torch
    from continuous_transformer_decode_gb300 import synth
    from tests import _gpu_util as U
    cfg = dict(name="stale", L=1, d=64, H=1, Hkv=1, hd=64, F=64, V=64, rms_eps=1e-5, rope_theta=1e4,
               tied=True)
    W = synth.make_weights(cfg, seed=1, fmt="f32")
    rng = np.random.default_rng(14)
    pg = Pages(rng, [200], 1, 64, 16)
    x = _cuda(rng.standard_normal((1, 1, 64)).astype(np.float32))
    at = _cuda(np.int32([0])), _cuda(np.int32([7]))
    out = torch.zeros_like(x)
    z, one = torch.zeros(1, 8, device="cuda"), torch.zeros(1, device="cuda")
    acc, nxt = (torch.full((1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    calls = [
        lambda: fs.fs_kv_q8_append(pg.view, x, x, *at),
        lambda: fs.fs_kv_q8_read(pg.view, *at, out),
        lambda: _attend(pg, x, [0], [200], split_len=64),
        lambda: fs.fs_verify_draft(z, _cuda(np.int32([0, 1])), at[0], None, one, one, one, acc, nxt)]
    for call in calls:
        with pytest.raises(fs.FsError) as e:
            U.make_gpu(cfg, W, fs.FS_DTYPE_F32, max_lanes=1, n_pages=1 << 30)  # 2 TB a side
        assert e.value.code == fs.CODES["FS_ERR_OOM"]
        call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("odd", [0, 1])
def test_infinities_read_back_finite_in_bf16(odd):
    """A bf16 read rounds to the nearest finite bf16: a stored infinity (the largest
    f32) does not come back infinite. Rows at odd addresses take the scalar stores."""
    import torch
    rng = np.random.default_rng(7)
    pg = Pages(rng, [4], 2, 64, 4)
    x = rng.standard_normal((4, 2, 64)).astype(np.float32)
    x[0, 0, 3], x[1, 1, 63], x[2, 0, 0], x[2, 1, 1] = np.inf, -np.inf, 3.4e38, -3.39e38
    at = _cuda(np.zeros(4, np.int32)), _cuda(np.arange(4, dtype=np.int32))
    fs.fs_kv_q8_append(pg.view, _cuda(x), -_cuda(x), *at)
    big = float(torch.finfo(torch.bfloat16).max)
    outs = [torch.zeros(4, 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")[:, odd:odd + 128]
            .unflatten(1, (2, 64)) for _ in range(2)]
    fs.fs_kv_q8_read(pg.view, *at, *outs)
    full = [torch.zeros(4, 2, 64, device="cuda") for _ in range(2)]
    fs.fs_kv_q8_read(pg.view, *at, *full)
    torch.cuda.synchronize()
    for o, f in zip(outs, full):
        want = np.clip(R.bf16(np.clip(f.cpu().numpy(), -big, big)), -big, big)
        assert np.array_equal(o.float().cpu().numpy(), want)
        assert (np.abs(want) == big).sum() == 4


@pytest.mark.parametrize("split", [64, 4096])
def test_a_row_longer_than_max_len_is_a_row_of_max_len(split):
    """Its tokens and the position that rotates its q."""
    import torch
    rng = np.random.default_rng(15)
    pg = Pages(rng, [300], 2, 128, 16)
    q = _cuda(rng.standard_normal((3, 4, 128)).astype(np.float32))
    tables = R.rope_tables(400, 128)
    rope = tuple(_cuda(a) for a in tables)
    got = _attend(pg, q, [0] * 3, [150, 299, 10000], rope=rope, max_len=150, split_len=split)
    ref, tol = R.attention(pg.ref(), q.cpu().numpy(), [0] * 3, [150] * 3, 128 ** -0.5, tables)
    _check_attention(got, ref, tol)
