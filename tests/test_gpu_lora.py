"""GPU: fs_lora_add against products in 64 bits (tests/_step_ref.py).

Tolerance. Products of bf16 values are exact; an f32 x is cut into three bf16 parts, which
hold its 24 bits. Sums are f32 in chains of at most K / 16 + rank / 8 + 40 additions, each off
by at most 2^-23 of the sum of the terms' magnitudes |B| |s| |A| |x| (the tensor cores cut,
where a rounding would give 2^-24). s A x is kept to 24 bits for f32 results and 16 for bf16
ones (2^-17 of |B| |s A x|). The result rounds once: 2^-24 or 2^-8 of its magnitude, and
the sum with base once more in f32."""
import numpy as np
import pytest

from continuous_transformer_decode_gb300 import fs
from tests import _step_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from continuous_transformer_decode_gb300 import build
    build.build()


def _t(a, bf16=False):
    import torch
    x = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return x.bfloat16() if bf16 else x


def _np(t):
    return t.double().cpu().numpy()


def make(rng, n, K, N, ads, rank, xb, yb, adapter=None):
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    adapter = rng.integers(-1, ads, n).astype(np.int32) if adapter is None else np.asarray(adapter, np.int32)
    return dict(x=_t(f(n, K), xb), adapter=_t(adapter), A=_t(f(ads, rank, K) * K**-0.5, True),
                B=_t(f(ads, N, rank) * rank**-0.5, True), scale=_t(rng.uniform(0.25, 2, ads).astype(np.float32)),
                base=_t(f(n, N), yb))


def check(c, got, base="base"):
    v = {k: _np(t) if k != "adapter" else t.cpu().numpy() for k, t in c.items()}
    b = np.zeros_like(v["base"]) if base is None else v["base"]
    want, terms, low = R.lora(v["x"], v["adapter"], v["A"], v["B"], v["scale"], b)
    K, rank = v["A"].shape[2], v["A"].shape[1]
    bf16 = str(got.dtype) == "torch.bfloat16"
    tol = (K / 16 + rank / 8 + 40) * 2.0**-23 * terms + 2.0**-24 * (np.abs(want) + np.abs(b) + terms)
    if bf16:
        tol += 2.0**-17 * low + 2.0**-8 * (np.abs(want) + tol)
    has = (v["adapter"] >= 0) & (v["adapter"] < len(v["A"]))
    err = np.abs(_np(got) - want)
    assert (err[has] <= tol[has]).all(), (err - tol)[has].max()
    assert np.array_equal(_np(got)[~has], b[~has])  # rows without an adapter: base itself


def run(c, base="base", out=None):
    import torch
    out = torch.full_like(c["base"], 9.0) if out is None else out
    fs.fs_lora_add(c["x"], c["adapter"], c["A"], c["B"], c["scale"], out, base=None if base is None else c["base"])
    return out


@pytest.mark.parametrize("xb,yb", [(True, False), (True, True), (False, False), (False, True)])
@pytest.mark.parametrize("rank", [8, 16, 24, 40, 64, 104, 128])
@pytest.mark.parametrize("n,K,N", [(1, 8, 1), (1, 576, 960), (3, 72, 33), (17, 264, 130), (65, 1000, 517), (130, 136, 8)])
def test_shapes(n, K, N, rank, xb, yb):
    rng = np.random.default_rng(n + K + N + rank)
    c = make(rng, n, K, N, 5, rank, xb, yb)
    check(c, run(c))
    check(c, run(c, base=None), base=None)


@pytest.mark.parametrize("yb", [False, True])
def test_large_dimensions(yb):
    rng = np.random.default_rng(7)
    c = make(rng, 40, 14336, 4099, 3, 16, True, yb)
    check(c, run(c))
    c = make(rng, 9, 4096, 14336, 9, 64, True, yb)
    check(c, run(c))


@pytest.mark.parametrize("how", ["one", "all different", "runs", "none", "out of range", "few"])
@pytest.mark.parametrize("n", [1, 64, 300])
def test_mixes_of_adapters(how, n):
    rng = np.random.default_rng(n)
    ads = 300
    adapter = {"one": np.full(n, 7), "all different": rng.permutation(ads)[:n], "runs": np.sort(rng.integers(0, 6, n)),
               "none": np.full(n, -1), "out of range": rng.choice([-2**31, -1, ads, 2**31 - 1, 5], n),
               "few": rng.choice([-1, -1, -1, 3, 299], n)}[how]
    c = make(rng, n, 128, 200, ads, 16, True, False, adapter)
    check(c, run(c))


@pytest.mark.parametrize("xb,yb", [(True, False), (True, True), (False, False)])
def test_in_place_and_strided(xb, yb):
    """Columns of wider panels that start anywhere; the columns around them stay."""
    import torch
    rng = np.random.default_rng(8)
    for off in (0, 1, 8):
        c = make(rng, 37, 72, 77, 4, 24, xb, yb)
        xp = torch.full((37, 72 + 2 * off + 5), 3.0, dtype=c["x"].dtype, device="cuda")
        xp[:, off:off + 72] = c["x"]
        yp = torch.full((37, 77 + 2 * off + 3), 5.0, dtype=c["base"].dtype, device="cuda")
        yp[:, off:off + 77] = c["base"]
        y = yp[:, off:off + 77]
        fs.fs_lora_add(xp[:, off:off + 72], c["adapter"], c["A"], c["B"], c["scale"], y, base=y)
        check(c, y)
        assert (yp[:, :off] == 5.0).all() and (yp[:, off + 77:] == 5.0).all()


@pytest.mark.parametrize("n", [1, 5, 64, 200])
def test_a_rows_bits_do_not_depend_on_the_batch(n):
    import torch
    rng = np.random.default_rng(9)
    c = make(rng, 200, 320, 129, 6, 32, True, False)
    whole = run(c)
    order = rng.permutation(200)[:n]
    d = dict(c, x=c["x"][order].contiguous(), adapter=c["adapter"][order].contiguous(), base=c["base"][order].contiguous())
    assert torch.equal(run(d), whole[order])


@pytest.mark.parametrize("xb,yb", [(True, False), (False, True)])
def test_a_rows_bits_are_the_same_in_large_batches(xb, yb):
    """Batches of all sizes that are taken in tiles of other heights."""
    import torch
    rng = np.random.default_rng(9)
    c = make(rng, 3001, 1000, 77, 5, 40, xb, yb, np.repeat(rng.integers(-1, 5, 30), 101)[:3001])
    whole = run(c)
    check(c, whole)
    for n in (1, 130, 1000, 1024, 1025):
        order = rng.permutation(3001)[:n]
        d = dict(c, x=c["x"][order].contiguous(), adapter=c["adapter"][order].contiguous(), base=c["base"][order].contiguous())
        assert torch.equal(run(d), whole[order])


@pytest.mark.parametrize("xb,yb", [(True, False), (True, True), (False, False), (False, True)])
@pytest.mark.parametrize("rank", [8, 64, 104])
def test_a_rows_bits_are_the_same_in_batches_of_two_tiles(xb, yb, rank):
    """More than 4096 rows of few adapters: items of two row tiles."""
    import torch
    rng = np.random.default_rng(rank)
    c = make(rng, 5003, 264, 69, 4, rank, xb, yb, np.repeat(rng.integers(-1, 4, 51), 99)[:5003])
    whole = run(c)
    check(c, whole)
    assert torch.equal(run(c, base=None)[c["adapter"] < 0], torch.zeros_like(whole[c["adapter"] < 0]))
    for n in (3, 200, 700):
        order = rng.permutation(5003)[:n]
        d = dict(c, x=c["x"][order].contiguous(), adapter=c["adapter"][order].contiguous(), base=c["base"][order].contiguous())
        assert torch.equal(run(d), whole[order])


@pytest.mark.parametrize("xb,yb", [(True, False), (False, True)])
def test_a_rows_bits_are_the_same_however_many_blocks_take_it(xb, yb):
    """300 adapters of one row each (a block an item), 64 (four blocks), three (eight), with K
    that the shares and pieces do not divide."""
    import torch
    rng = np.random.default_rng(21)
    for rank, K, N in ((16, 1096, 333), (104, 328, 1001), (8, 8, 5)):
        c = make(rng, 300, K, N, 300, rank, xb, yb, rng.permutation(300))
        whole = run(c)
        check(c, whole)
        for n in (1, 3, 40, 64, 76):
            order = rng.permutation(300)[:n]
            d = dict(c, x=c["x"][order].contiguous(), adapter=c["adapter"][order].contiguous(), base=c["base"][order].contiguous())
            assert torch.equal(run(d), whole[order]), (rank, n)


def test_what_is_no_number_stays_in_its_row():
    import torch
    rng = np.random.default_rng(10)
    c = make(rng, 50, 64, 40, 3, 16, True, False, np.arange(50) % 3)
    clean = run(c)
    c["x"][11, 5] = float("nan")
    c["x"][20, :] = float("inf")
    got = run(c)
    assert torch.isnan(got[11]).all() and not torch.isfinite(got[20]).any()
    rest = [i for i in range(50) if i not in (11, 20)]
    assert torch.equal(got[rest], clean[rest])
    # an adapter that no row has is not looked at
    c = make(rng, 8, 64, 40, 3, 16, True, False, [0, 2] * 4)
    clean = run(c)
    c["A"][1] = float("nan")
    c["B"][1] = float("nan")
    c["scale"][1] = float("nan")
    assert torch.equal(run(c), clean)


def test_f32_rows_keep_their_24_bits():
    """x and the product are wanted to f32 where out is: values that bf16 parts of 16 bits
    would lose."""
    rng = np.random.default_rng(11)
    c = make(rng, 20, 64, 24, 2, 8, False, False, np.arange(20) % 2)
    check(c, run(c, base=None), base=None)


def test_many_rows():
    rng = np.random.default_rng(12)
    n = 2500
    c = make(rng, n, 256, 300, 11, 16, True, True, np.repeat(rng.integers(-1, 11, n // 100), 100))
    check(c, run(c))
    c = make(rng, n, 256, 300, 40, 16, True, False)
    check(c, run(c))


def test_streams_and_graphs():
    import torch
    rng = np.random.default_rng(13)
    c = make(rng, 30, 128, 96, 4, 16, True, False)
    want = run(c)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        c2 = {k: v.clone() for k, v in c.items()}
        got = run(c2)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(c["base"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(c, out=out)
    for seed in range(3):
        c["x"].copy_(_t(np.random.default_rng(seed).standard_normal((30, 128)).astype(np.float32)))
        c["adapter"].copy_(_t(np.random.default_rng(seed).integers(-1, 4, 30).astype(np.int32)))
        g.replay()
        check(c, out)
