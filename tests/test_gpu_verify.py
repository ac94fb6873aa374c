"""GPU: verification of drafted tokens (fs_verify_draft) against the rule in 64
bits (tests/_q8_ref.py). Results are whole numbers and compared exactly: the
weights are good to 2^-36, so a number would have to fall within about 1e-11 of
a border to be answered otherwise."""
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


def softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def make(rng, drafts, V, probs=True, greedy=0.3, spread=2.5):
    drafts = np.asarray(drafts)
    start = np.concatenate([[0], np.cumsum(drafts + 1)]).astype(np.int32)
    rows, n = int(start[-1]), len(drafts)
    logits = (spread * rng.standard_normal((rows, V))).astype(np.float32)
    other = logits + 0.7 * rng.standard_normal((rows, V)).astype(np.float32)
    temps = np.where(rng.random(n) < greedy, 0, rng.uniform(0.5, 1.3, n)).astype(np.float32)
    seq = np.repeat(np.arange(n), drafts + 1)
    q = softmax(other / np.where(temps > 0, temps, 1)[seq][:, None]).astype(np.float32)
    draft = np.array([rng.choice(V, p=r.astype(np.float64) / r.astype(np.float64).sum()) for r in q], np.int32)
    draft = np.where(temps[seq] > 0, draft, other.argmax(-1)).astype(np.int32)
    return dict(logits=logits, row_start=start, draft=draft, probs=q if probs else None, temps=temps,
                u_accept=rng.random(rows).astype(np.float32), u_sample=rng.random(n).astype(np.float32))


def run(c, stream=None, out=None):
    import torch
    n = len(c["temps"])
    acc, nxt = out or (torch.full((n,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    fs.fs_verify_draft(_cuda(c["logits"]), _cuda(c["row_start"]), _cuda(c["draft"]),
                       None if c["probs"] is None else _cuda(c["probs"]), _cuda(c["temps"]),
                       _cuda(c["u_accept"]), _cuda(c["u_sample"]), acc, nxt, stream=stream)
    torch.cuda.synchronize()
    return acc.cpu().numpy(), nxt.cpu().numpy()


def check(c):
    got, want = run(c), R.verify(**c)
    assert np.array_equal(got[0], want[0]), (got[0], want[0])
    assert np.array_equal(got[1], want[1]), (got[1], want[1])
    return want


@pytest.mark.parametrize("V", [1, 2, 31, 257, 1000, 4099, 32000, 49152, 70001])
@pytest.mark.parametrize("probs", [True, False])
def test_rule(V, probs):
    rng = np.random.default_rng(V)
    big = V > 20000
    drafts = [4, 0, 7, 1] if big else [0, 1, 2, 5, 9, 3, 3, 0, 4, 4, 6, 2]
    check(make(rng, drafts, V, probs))


def test_every_outcome_is_met():
    """Acceptance of none, some and all drafted tokens, greedy and sampled."""
    rng = np.random.default_rng(0)
    for greedy in (0.0, 1.0):
        c = make(rng, [3] * 200, 50, True, greedy)
        acc, _ = check(c)
        assert set(acc.tolist()) == {0, 1, 2, 3}


def test_distribution_is_the_targets():
    """The first token that comes out is distributed as the target says, whatever
    the draft: 20000 sequences of one draft, chi-square of 8 tokens below its
    1 - 1e-6 quantile (7 degrees of freedom: 40.5)."""
    rng = np.random.default_rng(3)
    n, V = 20000, 8
    z = rng.standard_normal(V).astype(np.float32)
    q = softmax(rng.standard_normal(V)).astype(np.float32)
    p = softmax(z.astype(np.float64) / 0.8)
    c = dict(logits=np.tile(z, (2 * n, 1)), row_start=np.arange(0, 2 * n + 1, 2, dtype=np.int32),
             draft=rng.choice(V, size=2 * n, p=q / q.astype(np.float64).sum()).astype(np.int32),
             probs=np.tile(q, (2 * n, 1)), temps=np.full(n, 0.8, np.float32),
             u_accept=rng.random(2 * n).astype(np.float32), u_sample=rng.random(n).astype(np.float32))
    acc, nxt = run(c)
    first = np.where(acc > 0, c["draft"][::2], nxt)
    count = np.bincount(first, minlength=V)
    assert ((count - n * p) ** 2 / (n * p)).sum() < 40.5


def test_edges():
    rng = np.random.default_rng(1)
    c = make(rng, [2] * 12, 300, True, 0.0)
    z, d = c["logits"], c["draft"]
    z[0] = -np.inf                                   # no token at all
    z[3, :] = -np.inf
    z[3, 17] = 2.0                                   # one token
    z[6, 5] = z[6, 9] = np.inf                       # two tokens share everything
    z[9, ::2] = -np.inf                              # masked halves
    z[12, 1::2] = np.finfo(np.float32).min           # masks of the type's lowest value
    z[15, 4] = np.nan
    c["u_accept"][18], d[18] = 0.0, int(np.argmin(z[18]))
    d[21], d[24] = -1, 300                           # no such tokens
    c["u_sample"][:] = rng.random(12)
    c["u_sample"][8], c["u_sample"][9] = 0.0, np.float32(1 - 2.0 ** -24)
    c["probs"][27] = softmax(z[27] / c["temps"][9])  # the draft is the target
    c["temps"][10], c["temps"][11] = 1e-3, 1e4
    check(c)
    c["temps"][:6] = 0
    c["temps"][6], c["temps"][7] = -1.0, np.nan      # not positive: greedy
    check(c)
    c["probs"] = None
    check(c)


@pytest.mark.parametrize("probs", [True, False])
def test_extreme_temperatures(probs):
    rng = np.random.default_rng(11)
    c = make(rng, [3] * 8, 700, probs, 0.0)
    c["temps"] = np.float32([np.inf, 3e38, 1e30, 1e5, 1e-5, 1e-30, 1e-38, 1e-45])
    check(c)


def test_sequences_without_rows_and_clamped_starts():
    rng = np.random.default_rng(2)
    c = make(rng, [1, 2, 0], 40)
    c["row_start"] = np.array([0, 0, 2, 2, 5, 6, 9, -3], np.int32)  # 6 rows
    n = 7
    c["temps"] = np.full(n, 0.9, np.float32)
    c["u_sample"] = rng.random(n).astype(np.float32)
    acc, nxt = check(c)
    assert nxt[0] == -1 and nxt[2] == -1


def test_ties_of_greedy_go_to_the_lowest_index():
    rng = np.random.default_rng(4)
    c = make(rng, [1] * 40, 5000, True, 1.0)
    c["logits"] = np.round(c["logits"])
    check(c)


def test_strided_rows_streams_and_graphs():
    import torch
    rng = np.random.default_rng(5)
    cs = [make(rng, [3, 0, 5], 3001), make(rng, [1, 6, 1], 3001)]
    wide = [torch.zeros(int(c["row_start"][-1]), 4000, device="cuda") for c in cs]
    graphs = []
    for c, w in zip(cs, wide):
        w[:, 7:3008] = _cuda(c["logits"])
        args = [_cuda(c[k]) for k in ("row_start", "draft", "probs", "temps", "u_accept", "u_sample")]
        out = [torch.full((3,), -9, dtype=torch.int32, device="cuda") for _ in range(2)]
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            fs.fs_verify_draft(w[:, 7:3008], *args, *out, stream=torch.cuda.current_stream())
        graphs.append((st, g, out, args))
    for _ in range(10):
        for st, g, *_ in graphs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for c, (_, _, out, _) in zip(cs, graphs):
        want = R.verify(**c)
        assert np.array_equal(out[0].cpu().numpy(), want[0])
        assert np.array_equal(out[1].cpu().numpy(), want[1])


def test_draw_among_the_smallest_weights():
    """All that is left are weights of 2^-124.9 to 2^-118 of the largest: they are held
    to 2^-36 too, though the second half of such a pair is below f32's range."""
    rng = np.random.default_rng(21)
    n, V = 300, 60
    z = np.empty((2 * n, V), np.float32)
    q = np.zeros((2 * n, V), np.float32)
    us = []
    temps = rng.uniform(0.5, 1.5, n).astype(np.float32)
    for s in range(n):
        row = -(rng.uniform(118.0, 124.8, V) * np.log(2.0) * float(temps[s])).astype(np.float32)
        row[0] = 0.0
        z[2 * s:2 * s + 2] = row
        q[2 * s:2 * s + 2, 0] = 1.0   # takes all of the largest
        q[2 * s:2 * s + 2, 5] = 1.0   # the draft
        w = np.exp(row.astype(np.float64) / float(temps[s]))
        w[[0, 5]] = 0.0
        cum = np.cumsum(w)
        i = rng.integers(1, 4)
        for step in (0, 1, -1):
            u = np.float32(cum[i] / cum[-1])
            u = (u.view(np.int32) + np.int32(step)).view(np.float32)
            # a running sum of weights good to 2^-36, its own roundings, and the total
            if abs(float(u) * cum[-1] - cum[i]) > 2.0 ** -33 * cum[i]:
                break
        us.append(u)
    c = dict(logits=z, row_start=np.arange(0, 2 * n + 1, 2, dtype=np.int32),
             draft=np.full(2 * n, 5, np.int32), probs=q, temps=temps,
             u_accept=np.full(2 * n, 0.5, np.float32), u_sample=np.float32(us))
    acc, _ = check(c)
    assert (acc == 0).all()


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("V,depths", [(2, 300), (1500, 20), (5000, 3), (5000, 16), (60000, 2)])
def test_acceptance_next_to_its_border(V, depths, probs):
    """Drafts of 5 to 86 nats below the largest logit (a third of the probability in
    equal logits, whose roundings are alike), u * q(x) a few f32 steps to either side
    of p(x): nearer than an f32 weight is good to, further than one of 2^-36 (cases
    within 2^-33 are left out)."""
    rng = np.random.default_rng(V + depths)
    rows, q, ua, temps = [], [], [], []
    for d in rng.uniform(5.0, 86.0, depths):
        T, M = np.float32(rng.uniform(0.3, 2.0)), np.float32(5 * rng.standard_normal())
        z = np.empty(V, np.float32)
        z[:] = M - T * np.float32(np.log(2.0 * max(V - 2, 1)) + rng.uniform(-0.2, 0.2))
        z[0], z[V - 1] = M, M - np.float32(d) * T
        e = np.exp((z.astype(np.float64) - float(M)) / float(T))
        p = e[V - 1] / e.sum()
        for k in (-64, -32, -16, -11, -8, -5, -4, -3, -2, -1, 0, 1, 2, 3, 4, 5, 8, 11, 16, 32, 64):
            u = np.float32(rng.uniform(0.25, 1.0)) if probs else np.float32(p)
            near = np.float32(p / float(u)) if probs else u
            near = (np.float32(near).view(np.int32) + np.int32(k)).view(np.float32)
            u, x = (u, near) if probs else (near, np.float32(1.0))
            if abs(float(u) * float(x) - p) <= 2.0 ** -33 * p:
                continue
            rows += [z, z]
            one = np.zeros(V, np.float32)
            one[V - 1] = x
            q += [one, one]
            ua += [u, u]
            temps.append(T)
    n = len(temps)
    assert n > 15 * depths
    c = dict(logits=np.stack(rows), row_start=np.arange(0, 2 * n + 1, 2, dtype=np.int32),
             draft=np.full(2 * n, V - 1, np.int32), probs=np.stack(q) if probs else None,
             temps=np.float32(temps), u_accept=np.float32(ua),
             u_sample=rng.uniform(0.1, 0.5, n).astype(np.float32))
    acc, _ = check(c)
    assert 0 < acc.sum() < n  # both sides are met


def _next_to_borders(rng, cum, n, steps=24):
    """n numbers of u_sample, each a few f32 steps from the place of a running sum of
    cum, none within 2^-33 of one: what weights good to 2^-36 and their sums tell."""
    out = []
    for _ in range(100 * n):
        i = rng.integers(0, len(cum) - 1)
        u = np.float32(cum[i] / cum[-1])
        u = (u.view(np.int32) + np.int32(rng.integers(-steps, steps + 1))).view(np.float32)
        j = np.searchsorted(cum, float(u) * cum[-1])
        near = min(abs(cum[k] - float(u) * cum[-1]) for k in (max(j - 1, 0), min(j, len(cum) - 1)))
        if 0 <= u < 1 and near > 2.0 ** -33 * cum[-1]:
            out.append(u)
        if len(out) == n:
            return np.float32(out)
    raise AssertionError("no such numbers")


def _draws(z, T, us):
    """next_token of sequences of one row each, all of them the row z."""
    n = len(us)
    c = dict(logits=np.tile(z, (n, 1)), row_start=np.arange(n + 1, dtype=np.int32),
             draft=np.full(n, -1, np.int32), probs=None, temps=np.full(n, T, np.float32),
             u_accept=np.zeros(n, np.float32), u_sample=us)
    acc, nxt = run(c)
    assert (acc == 0).all()
    return nxt


def _equal_groups(rng, V):
    """One largest logit and two groups of equal ones of about its probability each,
    in runs or mixed: every weight of a group is rounded alike."""
    T, M = np.float32(rng.uniform(0.4, 1.5)), np.float32(4 * rng.standard_normal())
    below = [T * np.float32(np.log(V / 2.0) + rng.uniform(-0.3, 0.3)) for _ in range(2)]
    z = np.full(V, M - below[0], np.float32)
    z[V // 2:] = M - below[1]
    if rng.random() < 0.5:
        rng.shuffle(z)
    z[rng.integers(0, V)] = M
    return z, T


@pytest.mark.parametrize("V,n,rows", [(2000, 100, 3), (9000, 40, 3), (49152, 40, 4), (131072, 40, 4),
                                      (262144, 40, 6), (262144, 100, 6), (1 << 20, 80, 2)])
def test_draw_next_to_borders_among_equal_logits(V, n, rows):
    rng = np.random.default_rng(V + n)
    for r in range(rows):
        z, T = _equal_groups(rng, V)
        if r == 0 and V == 262144:  # 1e-6 too large and too small in f32
            T, z[:] = np.float32(0.7341579), np.float32(-5.716526)
            z[V // 2:], z[0] = np.float32(-5.7151575), np.float32(2.3561673)
        e = np.exp((z.astype(np.float64) - float(z.max())) / float(T))
        cum = np.cumsum(e)
        us = _next_to_borders(rng, cum, n)
        want = np.searchsorted(cum, us.astype(np.float64) * cum[-1])
        assert np.array_equal(_draws(z, T, us), want)


@pytest.mark.parametrize("V,n", [(9000, 30), (49152, 30), (262144, 8), (49152, 100)])
def test_residual_draw_next_to_borders(V, n):
    """The same of max(p - q, 0), after a draft of no probability, q in equal runs."""
    rng = np.random.default_rng(V + 7 * n)
    z, T = _equal_groups(rng, V)
    x = int(rng.integers(1, V - 1))
    z[x] = -np.inf
    e = np.exp((z.astype(np.float64) - float(z.max())) / float(T))
    p = e / e.sum()
    q = (p * np.where(np.arange(V) // 37 % 3 == 0, 1.5, rng.uniform(0.1, 0.9))).astype(np.float32)
    q[x] = 0.1
    cum = np.cumsum(np.maximum(p - q, 0.0))
    c = dict(logits=np.tile(z, (2 * n, 1)), row_start=np.arange(0, 2 * n + 1, 2, dtype=np.int32),
             draft=np.full(2 * n, x, np.int32), probs=np.tile(q, (2 * n, 1)),
             temps=np.full(n, T, np.float32), u_accept=np.full(2 * n, 0.5, np.float32),
             u_sample=_next_to_borders(rng, cum, n))
    acc, _ = check(c)
    assert (acc == 0).all()
