"""Argument checks of the operators for what differs from request to request (they come
before any CUDA call, so they run without a GPU; the addresses below are never read), and
fs_rope_frequencies, which is host arithmetic."""
import ctypes as C
import math

import numpy as np
import pytest

from continuous_transformer_decode_gb300 import build, fs

ARG = fs.CODES["FS_ERR_ARG"]
MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def pages(**kw):
    d = dict(holders=1 * MB, n_pages=100, table=2 * MB, lengths=3 * MB, n_lanes=4, max_pages=8, page=16,
             keep=4 * MB, grow=5 * MB, start=6 * MB, lane=7 * MB, pos=8 * MB, len=9 * MB, slot=10 * MB,
             rows=64, status=11 * MB)
    d.update(kw)
    return fs.lib().fs_pages_update(d["holders"], d["n_pages"], d["table"], d["lengths"], d["n_lanes"],
                                    d["max_pages"], d["page"], d["keep"], d["grow"], d["start"], d["lane"],
                                    d["pos"], d["len"], d["slot"], d["rows"], d["status"], None)


def rope(f=None, **kw):
    f = np.ones(32) if f is None else f
    d = dict(q=1 * MB, qs=256, H=4, k=2 * MB, ks=128, Hkv=2, n=3, hd=64, dtype=0, pos=3 * MB, freq=f.ctypes.data,
             rot=64, factor=1.0, flags=0, qo=1 * MB, qos=256, ko=2 * MB, kos=128)
    d.update(kw)
    return fs.lib().fs_rope(d["q"], d["qs"], d["H"], d["k"], d["ks"], d["Hkv"], d["n"], d["hd"], d["dtype"],
                            d["pos"], d["freq"], d["rot"], d["factor"], d["flags"], d["qo"], d["qos"], d["ko"],
                            d["kos"], None)


def lora(**kw):
    d = dict(x=1 * MB, xs=64, xt=1, adapter=2 * MB, n=3, K=64, N=40, A=3 * MB, B=4 * MB, scale=5 * MB, ad=2,
             rank=16, base=6 * MB, bs=40, out=7 * MB, os=40, yt=0)
    d.update(kw)
    return fs.lib().fs_lora_add(d["x"], d["xs"], d["xt"], d["adapter"], d["n"], d["K"], d["N"], d["A"], d["B"],
                                d["scale"], d["ad"], d["rank"], d["base"], d["bs"], d["out"], d["os"], d["yt"],
                                None)


def sample(**kw):
    d = dict(z=1 * MB, ld=100, n=3, V=100, temps=2 * MB, k=3 * MB, p=4 * MB, m=5 * MB, u=6 * MB, tok=7 * MB,
             kept=8 * MB)
    d.update(kw)
    return fs.lib().fs_sample_filtered(d["z"], d["ld"], d["n"], d["V"], d["temps"], d["k"], d["p"], d["m"],
                                       d["u"], d["tok"], d["kept"], None)


def refused_by_a_check():
    """The last call was refused for its arguments, before its addresses were looked at."""
    assert fs.fs_last_error(None) not in ("", "no CUDA device", "not a device pointer")


def test_the_calls_that_are_varied_are_refused_for_their_addresses_alone():
    for call in (pages, rope, lora, sample):
        assert call() == ARG
        assert fs.fs_last_error(None) in ("no CUDA device", "not a device pointer")


@pytest.mark.parametrize("bad", [
    dict(holders=None), dict(table=None), dict(lengths=None), dict(grow=None), dict(start=None),
    dict(status=None), dict(n_pages=0), dict(n_lanes=0), dict(n_lanes=8193), dict(max_pages=0),
    dict(page=0), dict(page=-1), dict(rows=-1), dict(max_pages=1 << 16, page=(1 << 14) + 1),
    dict(holders=MB + 2), dict(keep=4 * MB + 1), dict(pos=8 * MB + 2), dict(slot=10 * MB + 4),
    dict(lengths=3 * MB, keep=3 * MB), dict(grow=3 * MB), dict(lane=8 * MB + 4), dict(status=2 * MB + 8),
    dict(holders=2 * MB - 396), dict(len=9 * MB, slot=9 * MB + 248)], ids=str)
def test_pages_refusals(bad):
    assert pages(**bad) == ARG
    refused_by_a_check()


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(qo=None), dict(pos=None), dict(freq=None), dict(k=None), dict(Hkv=0), dict(ko=None),
    dict(H=0), dict(n=-1), dict(hd=1), dict(hd=1025), dict(rot=0), dict(rot=3), dict(rot=66), dict(dtype=2),
    dict(flags=4), dict(factor=float("inf")), dict(factor=float("nan")), dict(factor=1e39), dict(qs=255),
    dict(q=MB + 2), dict(pos=3 * MB + 2), dict(qos=300), dict(kos=200), dict(qo=MB + 16), dict(ko=MB),
    dict(qo=2 * MB), dict(k=None, Hkv=0), dict(qo=3 * MB - 4, qos=256), dict(dtype=1, q=MB + 1)], ids=str)
def test_rope_refusals(bad):
    assert rope(**bad) == ARG
    refused_by_a_check()


def test_rope_frequencies_that_are_no_numbers_are_refused():
    for v in (np.nan, np.inf, -np.inf, 2.0**20 + 1):
        f = np.ones(32)
        f[31] = v
        assert rope(f) == ARG
        refused_by_a_check()


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(adapter=None), dict(A=None), dict(B=None), dict(scale=None), dict(out=None),
    dict(n=-1), dict(K=0), dict(K=60), dict(N=0), dict(ad=0), dict(rank=0), dict(rank=4), dict(rank=12),
    dict(rank=136), dict(xt=2), dict(yt=3), dict(xs=63), dict(os=39), dict(bs=39), dict(A=3 * MB + 8),
    dict(B=4 * MB + 2), dict(x=MB + 1), dict(out=7 * MB + 2), dict(scale=5 * MB + 1),
    dict(base=7 * MB, bs=44), dict(base=7 * MB + 8), dict(out=MB, os=64), dict(out=2 * MB + 4),
    dict(out=4 * MB + 16)], ids=str)
def test_lora_refusals(bad):
    assert lora(**bad) == ARG
    refused_by_a_check()


@pytest.mark.parametrize("bad", [
    dict(z=None), dict(temps=None), dict(u=None), dict(tok=None), dict(n=-1), dict(V=0), dict(V=MB + 1, ld=MB + 1),
    dict(ld=99), dict(z=MB + 2), dict(k=3 * MB + 1), dict(tok=7 * MB + 2), dict(kept=7 * MB + 4),
    dict(tok=MB + 400), dict(kept=6 * MB)], ids=str)
def test_sample_refusals(bad):
    assert sample(**bad) == ARG
    refused_by_a_check()


def test_nothing_to_do_is_no_error():
    assert rope(n=0, q=None, k=None, Hkv=0, ko=None) == 0
    assert lora(n=0) == 0 and sample(n=0) == 0


# ------------------------------------------------------------------ frequencies
def test_unscaled_and_linear_and_base():
    for rot in (2, 20, 64, 128, 512):
        j = np.arange(rot // 2)
        f, m = fs.fs_rope_frequencies(rot, 10000.0)
        assert m == 1.0
        np.testing.assert_allclose(f, 10000.0 ** (-2.0 * j / rot), rtol=1e-14)
        g, m = fs.fs_rope_frequencies(rot, 10000.0, dict(kind="linear", factor=4.0))
        assert m == 1.0
        np.testing.assert_allclose(g, f / 4, rtol=1e-14)
        g, m = fs.fs_rope_frequencies(rot, 10000.0, dict(kind="base", factor=4.0))
        theta = 10000.0 * 4.0 ** (rot / (rot - 2)) if rot > 2 else 10000.0
        np.testing.assert_allclose(g, theta ** (-2.0 * j / rot), rtol=1e-13)
        if rot > 2:  # the slowest pair is scaled by the whole factor
            assert math.isclose(g[-1], f[-1] / 4, rel_tol=1e-12)


def test_ramp():
    rot, theta, by, original = 128, 10000.0, 8.0, 4096
    f, _ = fs.fs_rope_frequencies(rot, theta)
    g, m = fs.fs_rope_frequencies(rot, theta, dict(kind="ramp", factor=by, original=original))
    assert math.isclose(m, 0.1 * math.log(by) + 1)
    # pairs that turn 32 times or more, and fewer than once, by the wavelength itself
    turns = original * f / (2 * math.pi)
    assert np.array_equal(g[turns > 40], f[turns > 40])
    np.testing.assert_allclose(g[turns < 0.7], f[turns < 0.7] / by, rtol=1e-13)
    low = math.floor(rot * math.log(original / (64 * math.pi)) / (2 * math.log(theta)))
    high = math.ceil(rot * math.log(original / (2 * math.pi)) / (2 * math.log(theta)))
    j = (low + high) // 2
    mix = (j - low) / (high - low)
    assert math.isclose(g[j], f[j] * (1 - mix) + f[j] / by * mix, rel_tol=1e-13)
    g, m = fs.fs_rope_frequencies(rot, theta, dict(kind="ramp", factor=1.0, original=original))
    assert m == 1.0
    np.testing.assert_allclose(g, f, rtol=1e-14)


def test_bands():
    rot, theta, by, original = 128, 500000.0, 8.0, 8192
    f, _ = fs.fs_rope_frequencies(rot, theta)
    g, m = fs.fs_rope_frequencies(rot, theta, dict(kind="bands", factor=by, original=original))
    assert m == 1.0
    wave = 2 * math.pi / f
    for j in range(rot // 2):
        if wave[j] < original / 4:
            want = f[j]
        elif wave[j] > original:
            want = f[j] / by
        else:
            s = (original / wave[j] - 1) / 3
            want = (1 - s) * f[j] / by + s * f[j]
        assert math.isclose(g[j], want, rel_tol=1e-13)


@pytest.mark.parametrize("rot,theta,scaling", [
    (0, 1e4, None), (3, 1e4, None), (514, 1e4, None), (64, 0.0, None), (64, float("nan"), None),
    (64, 1e4, dict(kind="linear", factor=0.0)), (64, 1e4, dict(kind="base", factor=float("inf"))),
    (64, 1e4, dict(kind="ramp", factor=2.0)), (64, 1.0, dict(kind="ramp", factor=2.0, original=100)),
    (64, 1e4, dict(kind="bands", factor=2.0, original=100, low=4.0, high=4.0)),
    (64, 1e4, dict(kind="bands", factor=2.0, original=100, low=0.0)), (64, 1e4, dict(kind="other")),
    (64, 1e4, dict(kind="linear", factor=2.0, original=100))], ids=str)
def test_frequencies_refusals(rot, theta, scaling):
    with pytest.raises(fs.FsError) as e:
        fs.fs_rope_frequencies(rot, theta, scaling)
    assert e.value.code == ARG


def test_frequencies_null_outputs():
    f, m = np.empty(32), C.c_double()
    assert fs.lib().fs_rope_frequencies(64, 1e4, None, None, C.byref(m)) == ARG
    assert fs.lib().fs_rope_frequencies(64, 1e4, None, f.ctypes.data, None) == ARG
