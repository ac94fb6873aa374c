"""GPU: fs_sample_filtered against the rule in 64 bits (tests/_step_ref.py). Tokens and
counts are whole numbers and compared exactly: weights are good to 2^-36 and sums to more, so
a number would have to fall within about 1e-11 of a border to be answered otherwise."""
import numpy as np
import pytest

from continuous_transformer_decode_gb300 import fs
from tests import _step_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from continuous_transformer_decode_gb300 import build
    build.build()


def _cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run(z, T, u, k=None, p=None, m=None, stride=0):
    import torch
    n, V = z.shape
    f = lambda a, t: None if a is None else _cuda(np.broadcast_to(np.asarray(a, t), (n,)).copy())
    zd = _cuda(z)
    if stride:
        buf = torch.full((n, V + stride), 99.0, device="cuda")
        buf[:, :V] = zd
        zd = buf[:, :V]
    tok, kept = (torch.full((n + 1,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    fs.fs_sample_filtered(zd, f(T, np.float32), f(u, np.float32), tok[:n], f(k, np.int32), f(p, np.float32), f(m, np.float32),
                          kept[:n])
    torch.cuda.synchronize()
    assert tok[n] == -9 and kept[n] == -9
    return tok[:n].cpu().numpy(), kept[:n].cpu().numpy()


def check(z, T, u, k=None, p=None, m=None, stride=0):
    n = len(z)
    b = lambda a, none: np.broadcast_to(none if a is None else a, (n,))
    got = run(z, T, u, k, p, m, stride)
    want = [R.sample(*r) for r in zip(z, b(T, 1), b(u, 0), b(k, 0), b(p, 1.0), b(m, 0.0))]
    assert np.array_equal(got[1], [w[1] for w in want]), [(i, g, w[1]) for i, (g, w) in enumerate(zip(got[1], want)) if g != w[1]]
    assert np.array_equal(got[0], [w[0] for w in want]), [(i, g, w[0]) for i, (g, w) in enumerate(zip(got[0], want)) if g != w[0]]
    return got


VOCABS = [1, 2, 31, 257, 1000, 2049, 4099, 32000, 49152, 70001]


@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("spread", [0.3, 2.5, 12.0])
def test_rule(V, spread):
    """Every filter and mix of them, rows with settings of their own."""
    rng = np.random.default_rng(V)
    n = 24 if V < 20000 else 12
    z = (spread * rng.standard_normal((n, V))).astype(np.float32)
    T = np.where(rng.random(n) < 0.15, 0, rng.uniform(0.5, 1.5, n)).astype(np.float32)
    u = rng.random(n).astype(np.float32)
    k = np.where(rng.random(n) < 0.3, 0, np.exp(rng.uniform(0, np.log(V + 2), n))).astype(np.int32)
    p = np.where(rng.random(n) < 0.3, 1, rng.uniform(0.05, 0.999, n)).astype(np.float32)
    m = np.where(rng.random(n) < 0.5, 0, rng.uniform(0.001, 0.3, n)).astype(np.float32)
    check(z, T, u)
    check(z, T, u, k=k)
    check(z, T, u, p=p)
    check(z, T, u, m=m)
    check(z, T, u, k, p)
    check(z, T, u, k, p, m, stride=int(rng.integers(0, 8)))


def test_top_p_next_to_one_and_zero():
    rng = np.random.default_rng(1)
    z = (2.5 * rng.standard_normal((8, 5000))).astype(np.float32)
    u = rng.random(8).astype(np.float32)
    for p in (0.0, -1.0, 1e-30, 1e-4, 0.99, 0.9999, 0.999999, np.float32(1) - np.float32(2**-24), 1.0, 7.0, np.inf):
        check(z, 1.0, u, p=np.float32(p))
    got = run(z, 1.0, u, p=np.float32(np.nan))
    assert (got[1] == 5000).all()


def test_top_k_of_every_size():
    rng = np.random.default_rng(2)
    V = 3000
    k = np.array([-5, 0, 1, 2, 3, 50, 255, 256, 257, 1000, 2999, 3000, 3001, 2**31 - 1])
    z = (2.5 * rng.standard_normal((len(k), V))).astype(np.float32)
    got = check(z, 0.8, rng.random(len(k)).astype(np.float32), k=k)
    assert list(got[1]) == [3000, 3000, 1, 2, 3, 50, 255, 256, 257, 1000, 2999, 3000, 3000, 3000]


def test_min_p_of_every_size():
    rng = np.random.default_rng(3)
    m = np.array([-1, 0, 1e-38, 1e-30, 1e-20, 1e-7, 1e-3, 0.5, 1, 1.5, np.inf], np.float32)
    z = (9 * rng.standard_normal((len(m), 4000))).astype(np.float32)
    z[:, 17] = z.max(1)  # two that are largest
    got = check(z, 1.0, rng.random(len(m)).astype(np.float32), m=m)
    assert got[1][8] == 2 and got[1][9] == 1 and got[1][10] == 1
    got = run(z, 1.0, rng.random(len(m)).astype(np.float32), m=np.float32(np.nan))
    assert (got[1] == 4000).all()


@pytest.mark.parametrize("V", [300, 5000, 50000])
def test_equal_logits(V):
    """Ties go to the lowest index, in rows of a few distinct values."""
    rng = np.random.default_rng(V)
    n = 14
    z = rng.integers(-3, 4, (n, V)).astype(np.float32)
    z[0] = 0.0
    z[1, ::2] = -0.0
    z[2] = 5.0
    z[3] = np.where(rng.random(V) < 0.5, -0.0, 0.0)
    u = rng.random(n).astype(np.float32)
    k = rng.integers(1, V, n)
    p = rng.uniform(0.1, 0.99, n).astype(np.float32)
    check(z, 0.7, u, k=k)
    check(z, 0.7, u, p=p)
    check(z, 0.7, u, k=k, p=p, m=np.float32(0.02))


def test_infinities_and_nan():
    rng = np.random.default_rng(4)
    n, V = 12, 3000
    z = (2.5 * rng.standard_normal((n, V))).astype(np.float32)
    lowest = np.finfo(np.float32).min
    z[0, :] = -np.inf
    z[1, :] = np.nan
    z[2, 5:] = -np.inf
    z[3, [7, 900, 2500]] = np.inf
    z[4, ::3] = np.nan
    z[5, :] = lowest
    z[6, 1:] = lowest
    z[7, 1:] = -np.inf
    z[8, ::2] = -np.inf
    z[9, 3], z[9, 4] = np.finfo(np.float32).max, lowest
    z[10, [3, 9]], z[10, 11:] = np.inf, np.nan
    u = rng.random(n).astype(np.float32)
    for k, p, m in ((None, None, None), (2, None, None), (None, 0.7, None), (None, None, 0.1), (40, 0.9, 0.05), (2900, 0.99, None)):
        for T in (0.0, 0.9):
            got = check(z, T, u, k, None if p is None else np.float32(p), None if m is None else np.float32(m))
            assert list(got[0][:2]) == [0, 0] and list(got[1][:2]) == [0, 0]


def test_temperatures():
    rng = np.random.default_rng(5)
    T = np.array([1e-38, 1e-30, 1e-6, 1e-3, 0.1, 1, 10, 1e3, 1e6, 1e30, 3e38, np.inf, -1, np.nan], np.float32)
    z = (2.5 * rng.standard_normal((len(T), 2500))).astype(np.float32)
    u = rng.random(len(T)).astype(np.float32)
    check(z, T, u)
    check(z, T, u, k=300)
    check(z, T, u, p=np.float32(0.9))
    check(z, T, u, k=1000, p=np.float32(0.3), m=np.float32(0.01))


def test_random_numbers_at_their_ends():
    rng = np.random.default_rng(6)
    z = (2.5 * rng.standard_normal((5, 700))).astype(np.float32)
    u = np.array([0, 2**-126, 2**-24, 1 - 2**-24, 1], np.float32)
    check(z, 1.0, u)
    check(z, 1.0, u, k=9, p=np.float32(0.8))


@pytest.mark.parametrize("V", [600, 5000, 50000])
def test_the_smallest_weights_can_be_drawn(V):
    """u = 0 takes the first token whose weight is not 0, however small (2^-60 to 2^-120 of
    the largest here), also behind tokens without any."""
    rng = np.random.default_rng(V)
    z = np.full((6, V), -np.inf, np.float32)
    for i, bits in enumerate((45, 57, 59, 80, 100, 120)):
        z[i, 3 * i + 2:] = -bits * np.log(2)
        z[i, 3 * i] = -200.0  # a weight of 0
        z[i, rng.integers(V // 2, V)] = 0.0
    u = np.zeros(6, np.float32)
    z[:, 0] = -np.inf
    for T in (1.0, 0.98):
        for p, m in ((None, None), (np.float32(0.9999999), None), (None, np.float32(1e-30))):
            got = run(z, T, u, p=p, m=m)
            want = [R.sample(np.where(r == -200.0, -np.inf, r), T, 0.0, 0, 1.0 if p is None else p, 0.0 if m is None else m) for r in z]
            assert list(got[0]) == [w[0] for w in want]


@pytest.mark.parametrize("V,k", [(500, None), (4099, None), (49152, None), (49152, 100)])
def test_draws_next_to_borders(V, k):
    """Random numbers that are the nearest f32, and its neighbours, to borders of the
    running sum."""
    rng = np.random.default_rng(V)
    z = (2.0 * rng.standard_normal(V)).astype(np.float32)
    order, w = R.kept_ranks(z, 1.0, k or 0, 1.0, 0.0)
    places = np.sort(order)
    c = np.cumsum(w[places].astype(np.longdouble))
    at = rng.choice(len(places) - 1, 40)
    u = (c[at] / c[-1]).astype(np.float32)
    u = np.concatenate([u, np.nextafter(u, np.float32(0)), np.nextafter(u, np.float32(1))])
    check(np.broadcast_to(z, (len(u), V)).copy(), 1.0, u, k=k)


@pytest.mark.parametrize("V", [500, 4099, 49152])
def test_cuts_next_to_borders(V):
    """top_p that are the nearest f32, and its neighbours, to shares ahead of a token."""
    rng = np.random.default_rng(V)
    z = (2.0 * rng.standard_normal(V)).astype(np.float32)
    order, w = R.kept_ranks(z, 1.0, 0, 1.0, 0.0)
    c = np.cumsum(w[order].astype(np.longdouble))
    at = rng.choice(V - 1, 40)
    p = (c[at] / c[-1]).astype(np.float32)
    p = np.concatenate([p, np.nextafter(p, np.float32(0)), np.nextafter(p, np.float32(1))])
    check(np.broadcast_to(z, (len(p), V)).copy(), 1.0, rng.random(len(p)).astype(np.float32), p=p)


def test_many_small_weights():
    """A long tail of equal logits holds half of the mass."""
    V = 131072
    z = np.full((4, V), np.log(1.0 / V), np.float32)
    z[:, 77] = 0.0
    rng = np.random.default_rng(8)
    u = np.array([0.2, 0.7, 0.9999, 0.3], np.float32)
    check(z, 1.0, u)
    check(z, 1.0, u, p=np.array([0.3, 0.6, 0.9, 0.999], np.float32))
    check(z, 1.0, u, k=[1, 100, 70000, 131071])


def test_largest_vocabulary():
    rng = np.random.default_rng(9)
    z = (2.5 * rng.standard_normal((3, 1 << 20))).astype(np.float32)
    check(z, [1.0, 0.0, 0.7], rng.random(3).astype(np.float32), k=[0, 5, 300000], p=np.array([0.95, 1, 0.9], np.float32))


def test_many_rows():
    rng = np.random.default_rng(10)
    z = (2.5 * rng.standard_normal((700, 900))).astype(np.float32)
    check(z, 1.0, rng.random(700).astype(np.float32), k=rng.integers(0, 300, 700), p=rng.uniform(0.5, 1.1, 700).astype(np.float32))


def test_same_bits_whatever_the_batch_and_graphs():
    """A call on another stream, and captured and replayed with other inputs."""
    import torch
    rng = np.random.default_rng(11)
    z = [(2.5 * rng.standard_normal((9, 6000))).astype(np.float32) for _ in range(3)]
    u = rng.random(9).astype(np.float32)
    p = rng.uniform(0.5, 1, 9).astype(np.float32)
    zd, T, ud, pd = _cuda(z[0]), torch.full((9,), 0.8, device="cuda"), _cuda(u), _cuda(p)
    tok, kept = (torch.empty(9, dtype=torch.int32, device="cuda") for _ in range(2))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fs.fs_sample_filtered(zd, T, ud, tok, top_p=pd, kept=kept)
    side = torch.cuda.Stream()
    for x in z:
        zd.copy_(_cuda(x))
        torch.cuda.synchronize()
        g.replay()
        tok2, kept2 = torch.empty_like(tok), torch.empty_like(kept)
        fs.fs_sample_filtered(zd, T, ud, tok2, top_p=pd, kept=kept2, stream=side)
        torch.cuda.synchronize()
        want = [R.sample(r, 0.8, a, 0, b) for r, a, b in zip(x, u, p)]
        for t, n in ((tok, kept), (tok2, kept2)):
            assert t.tolist() == [w[0] for w in want] and n.tolist() == [w[1] for w in want]


@pytest.mark.parametrize("V,n", [(700, 12), (9000, 12), (9000, 300), (20000, 100), (32000, 40), (49152, 8), (49152, 30),
                                 (140001, 4), (400003, 2)])
def test_cuts_far_out(V, n):
    """Peaked rows, whose top-k, top-p and min-p end far down the tail: among weights of 2^-19
    and less, down to those that are 0."""
    rng = np.random.default_rng(V + n)
    z = (2.5 * rng.standard_normal((n, V))).astype(np.float32)
    u = rng.random(n).astype(np.float32)
    T = np.resize(np.array([0.5, 0.2, 0.06, 0.02], np.float32), n)
    k = np.exp(rng.uniform(0.6, 1.0, n) * np.log(V)).astype(np.int32)
    p = np.resize(np.array([0.998, 0.99, 0.9], np.float32), n)
    m = np.exp2(-rng.uniform(10, 120, n)).astype(np.float32)
    check(z, T, u, k=k)
    check(z, T, u, p=p)
    check(z, T, u, m=m)
    check(z, T, u, k=k, p=p)
    check(z, T, u, k=k, m=m)
    check(z, T, u, k=k, p=p, m=m)
    check(z, np.float32(0.6), u, p=np.float32(0.998), m=np.resize(np.array([0, 2.0**-18, 2.0**-19, 2.0**-17.5], np.float32), n))
    check(z, T, u, k=np.resize(np.array([1, 5, 40, 64, 65]), n), m=m)


@pytest.mark.parametrize("V", [5000, 49152])
@pytest.mark.parametrize("y", [17.5, 18.0, 19.0, 40.0, 124.5, 126.5, 140.0])
def test_one_token_and_a_plateau_far_below(V, y):
    """All others in one bin, equal or nearly, with weights of 2^-y."""
    rng = np.random.default_rng(5)
    n = 6
    z = np.full((n, V), -y * np.log(2), np.float32)
    z[3:] += (1e-3 * rng.standard_normal((3, V))).astype(np.float32)
    z[:, 1234] = 0.0
    u = np.array([0, 0.5, 0.99, 0, 0.5, 1 - 2.0**-24], np.float32)
    if y > 125:  # such weights may be 0, and u = 0 then draws another token
        u = np.maximum(u, np.float32(0.25))
    k = np.array([2, 100, V // 2, 40, 1000, V - 1])
    check(z, 1.0, u, k=k)
    check(z, 1.0, u, k=k, p=np.float32(0.9))
    check(z, 1.0, u, k=k, m=np.float32(2.0**-18))
