"""GPU: fs_lora_add with adapters that hold infinities and NaN, against the formula: base +
scale * B (A x) with IEEE infinities. What is finite there has the bits of the same call with
finite weights, as such values stay in the rows and columns that they belong to."""
import numpy as np
import pytest

from continuous_transformer_decode_gb300 import fs
from tests.test_gpu_lora import _np, _t, make, run

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from continuous_transformer_decode_gb300 import build
    build.build()


def formula(c, base=True):
    v = {k: _np(t) if k != "adapter" else t.cpu().numpy() for k, t in c.items()}
    out = v["base"].copy() if base else np.zeros_like(v["base"])
    with np.errstate(invalid="ignore"):
        for a in range(len(v["A"])):
            for i in np.nonzero(v["adapter"] == a)[0]:
                low = (v["A"][a] * v["x"][i]).sum(1) * v["scale"][a]
                out[i] += (v["B"][a] * low).sum(1)
    return out


def check(c, got, clean, base=True):
    import torch
    want = torch.from_numpy(formula(c, base))
    g = got.double().cpu()
    assert torch.equal(torch.isnan(g), torch.isnan(want))
    assert torch.equal(torch.where(torch.isinf(g), g, 0), torch.where(torch.isinf(want), want, 0))
    same = torch.isfinite(want)
    assert torch.equal(got.cpu()[same], clean.cpu()[same])
    return want


# rows and adapters: clusters of eight, of four, blocks alone, and items of two row tiles
KINDS = {"eight": (30, 3), "four": (90, 70), "alone": (300, 300), "two tiles": (4900, 3)}


@pytest.mark.parametrize("xb,yb", [(True, False), (True, True), (False, False), (False, True)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rank", [8, 40, 64, 128])
def test_b(kind, rank, xb, yb):
    n, ads = KINDS[kind]
    rng = np.random.default_rng(rank + n)
    adapter = rng.permutation(n) % (ads + 1) - 1 if kind != "two tiles" else np.sort(rng.integers(-1, ads, n))
    c = make(rng, n, 72, 70, ads, rank, xb, yb, adapter)
    c["x"][n // 2] = 0.0  # A x = 0: 0 times an infinity
    clean, bare = run(c), run(c, base=None)
    B = c["B"]
    B[1, 3, 2], B[1, 40, 0], B[1, 69, 7], B[1, 9, 1], B[1, 9, 5] = INF, -INF, NAN, INF, -INF
    B[2, 0, rank - 1], B[2, 33] = -INF, INF
    want = check(c, run(c), clean)
    assert want.isinf().any() and want.isnan().any()
    check(c, run(c, base=None), bare, base=False)
    y = c["base"].clone()  # in place
    check(c, run(dict(c, base=y), out=y), clean)


@pytest.mark.parametrize("xb,yb", [(True, False), (True, True), (False, False), (False, True)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rank", [8, 40, 64, 128])
def test_a(kind, rank, xb, yb):
    """Infinities of A, alone and with ones of B and of x."""
    n, ads = KINDS[kind]
    rng = np.random.default_rng(rank + n + 1)
    adapter = rng.permutation(n) % (ads + 1) - 1 if kind != "two tiles" else np.sort(rng.integers(-1, ads, n))
    c = make(rng, n, 136, 70, ads, rank, xb, yb, adapter)
    clean, finite = run(c), (c["A"].clone(), c["B"].clone())
    A, B = c["A"], c["B"]
    A[1, 3, 100], A[2, 0, 5], A[2, 0, 133] = INF, -INF, INF
    want = check(c, run(c), clean)
    assert want.isinf().any()
    B[1, 5, 3], B[1, 6, 3], B[1, 7, 2] = 0.0, -INF, INF
    check(c, run(c), clean)
    c["x"][n // 4, 5], c["x"][n // 5, 100] = 0.0, 0.0  # finite: rows of other adapters have other results
    clean = run(dict(c, A=finite[0], B=finite[1]))
    c["x"][n // 3, 100], c["x"][n // 2, 7] = INF, NAN
    c["base"][n // 6, 7] = -INF
    check(c, run(c), clean)
    if ads > 2:
        A[0, 1, 9] = NAN
        check(c, run(c), clean)


def test_a_captured_call():
    import torch
    rng = np.random.default_rng(5)
    c = make(rng, 30, 72, 70, 3, 16, False, False)
    clean, out = run(c), torch.empty_like(c["base"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(c, out=out)
    c["A"][1, 2, 30], c["B"][2, 9, 1] = INF, -INF
    g.replay()
    check(c, out, clean)
