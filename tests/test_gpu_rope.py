"""GPU: fs_rope against rotations in 64 bits (tests/_step_ref.py).

Tolerance. Sine and cosine are good to one f32 step (2^-23), the first-order step and the
product by the factor round once each, a product of the pair once and the sum that it is
fused into once: 2^-23 + 4 * 2^-24 = 6 * 2^-24 of factor * (|x| + |y|). The order that the
step leaves out is its angle squared, (2 pi 2^-24)^2 / 2 < 2^-43; the angle is off by
position * 2^-65 turns at most, below 2^-31 radians. A bf16 result rounds once more, half a
step: 2^-8 of its magnitude."""
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


def check(got, x, positions, f, factor, near, inverse=False):
    """got: the tensor that fs_rope wrote; x: its input."""
    v = x.double().cpu().numpy()
    want = R.rotate(v, positions, f, factor, near, inverse)
    r = len(f)
    part = np.zeros_like(v)  # |x| + |y| of each value's pair
    if near:
        s = np.abs(v[..., 0:2 * r:2]) + np.abs(v[..., 1:2 * r:2])
        part[..., 0:2 * r:2], part[..., 1:2 * r:2] = s, s
    else:
        s = np.abs(v[..., :r]) + np.abs(v[..., r:2 * r])
        part[..., :r], part[..., r:2 * r] = s, s
    tol = (6 * 2.0**-24 + 2.0**-30) * abs(factor) * part
    if str(got.dtype) == "torch.bfloat16":
        tol = tol + np.where(part > 0, 2.0**-8 * (np.abs(want) + tol), 0)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err - tol).max()


SHAPES = [  # H, Hkv, hd, rot
    (9, 3, 64, 64), (32, 8, 128, 128), (16, 2, 256, 64), (4, 4, 80, 20), (3, 1, 96, 96), (2, 1, 2, 2), (5, 5, 7, 6),
    (1, 0, 128, 32), (2, 2, 1024, 512), (6, 2, 66, 66)]


@pytest.mark.parametrize("H,Hkv,hd,rot", SHAPES)
@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("panel", [False, True])
def test_rotation(H, Hkv, hd, rot, near, bf16, panel):
    """Contiguous tensors, and columns of a projection's panel; out of place."""
    import torch
    rng = np.random.default_rng(hd + rot)
    f, m = fs.fs_rope_frequencies(rot, 10000.0, dict(kind="ramp", factor=4.0, original=4096))
    for n in (1, 5, 67):
        pos = np.concatenate([[0], rng.integers(1, 100000, n)])[-n:].astype(np.int32)
        if panel:
            p = _t(rng.standard_normal((n, (H + 2 * Hkv) * hd + 3)).astype(np.float32), bf16)
            q, k = p[:, :H * hd].unflatten(1, (H, hd)), p[:, H * hd:(H + Hkv) * hd].unflatten(1, (Hkv, hd)) if Hkv else None
        else:
            q = _t(rng.standard_normal((n, H, hd)).astype(np.float32), bf16)
            k = _t(rng.standard_normal((n, Hkv, hd)).astype(np.float32), bf16) if Hkv else None
        qo, ko = torch.full((n, H, hd), 7.0, dtype=q.dtype, device="cuda"), None
        if Hkv:
            ko = torch.full((n, Hkv, hd), 7.0, dtype=q.dtype, device="cuda")
        fs.fs_rope(q, _t(pos), f, k=k, q_out=qo, k_out=ko, interleaved=near, factor=m)
        check(qo, q, pos, f, m, near)
        if Hkv:
            check(ko, k, pos, f, m, near)


@pytest.mark.parametrize("near", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_in_place_in_a_panel_leaves_the_rest(near, bf16):
    rng = np.random.default_rng(1)
    n, H, Hkv, hd, rot = 33, 6, 2, 64, 32
    f, m = fs.fs_rope_frequencies(rot)
    p = _t(rng.standard_normal((n, (H + 2 * Hkv) * hd)).astype(np.float32), bf16)
    old = p.clone()
    pos = rng.integers(0, 5000, n).astype(np.int32)
    pos[[3, 20]] = -1, -2**31  # padded rows
    fs.fs_rope(p[:, :H * hd].unflatten(1, (H, hd)), _t(pos), f, k=p[:, H * hd:(H + Hkv) * hd].unflatten(1, (Hkv, hd)),
               interleaved=near)
    some = pos >= 0
    for a, b, h in ((0, H * hd, H), (H * hd, (H + Hkv) * hd, Hkv)):
        check(p[:, a:b].unflatten(1, (h, hd))[some], old[:, a:b].unflatten(1, (h, hd))[some], pos[some], f, 1.0, near)
    assert (p[~some] == old[~some]).all() and (p[:, (H + Hkv) * hd:] == old[:, (H + Hkv) * hd:]).all()
    # what lies behind the turned part keeps its bits
    assert (p[:, :H * hd].unflatten(1, (H, hd))[..., rot:] == old[:, :H * hd].unflatten(1, (H, hd))[..., rot:]).all()


def test_padded_rows_out_of_place_are_not_written():
    import torch
    q, f = _t(np.ones((4, 2, 64), np.float32)), np.ones(16)
    out = torch.full_like(q, 5.0)
    fs.fs_rope(q, _t(np.array([-1, 3, -7, 0], np.int32)), f, q_out=out)
    assert (out[[0, 2]] == 5.0).all() and (out[3] == 1.0).all() and (out[1][:, 32:] == 1.0).all()


@pytest.mark.parametrize("near", [False, True])
def test_far_positions(near):
    """The largest positions, fast and slow frequencies, negative and above a turn; 64-bit
    angles of the reference are long doubles."""
    rng = np.random.default_rng(2)
    f = np.array([1.0, 0.1, 1e-3, 1e-9, 0.0, -0.37, 6.5, 1000.123, -2.0**20, 3.3e-5])
    pos = np.array([0, 1, 2, 4095, 131071, 1048575, 2**24 + 1, 2**31 - 1, 12345678, 2**30], np.int32)
    # 64 bits of an angle of 2^31 * 2^20: the long double reference itself is off by
    # 2^51 * 2^-64, so those pairs stay below 2^31 * 2^10
    f[-2] = -2.0**10
    x = _t(rng.standard_normal((len(pos), 3, 2 * len(f))).astype(np.float32))
    out = x.clone()
    fs.fs_rope(x, _t(pos), f, q_out=out, interleaved=near)
    check(out, x, pos, f, 1.0, near)


def test_inverse_undoes():
    rng = np.random.default_rng(3)
    f, m = fs.fs_rope_frequencies(64, 10000.0, dict(kind="ramp", factor=16.0, original=2048))
    x = _t(rng.standard_normal((50, 4, 64)).astype(np.float32))
    pos = rng.integers(0, 1 << 20, 50).astype(np.int32)
    y, z = x.clone(), x.clone()
    fs.fs_rope(x, _t(pos), f, q_out=y, factor=m)
    check(y, x, pos, f, m, False)
    fs.fs_rope(y, _t(pos), f, q_out=z, factor=1 / m, inverse=True)
    check(z, y, pos, f, 1 / m, False, inverse=True)
    assert (z - x).abs().max() < 2e-6


def test_values_that_are_no_numbers_stay_in_their_pair():
    x = np.ones((1, 1, 8), np.float32)
    x[0, 0, 1] = np.nan
    x[0, 0, 6] = np.inf
    out = _t(x)
    fs.fs_rope(out, _t(np.array([3], np.int32)), np.array([1.0, 0.5]), interleaved=False)
    got = out.cpu().numpy()[0, 0]
    assert np.isnan(got[[1, 3]]).all() and np.isfinite(got[[0, 2, 4, 5, 7]]).all() and np.isinf(got[6])


def test_misaligned_rows():
    """Rows that start anywhere and strides of any number."""
    import torch
    rng = np.random.default_rng(4)
    f, _ = fs.fs_rope_frequencies(64)
    for bf16 in (False, True):
        for off, stride in ((1, 201), (2, 202), (3, 203), (4, 204), (8, 208)):
            buf = _t(rng.standard_normal(7 * 208 + 16).astype(np.float32), bf16)
            q = torch.as_strided(buf, (7, 3, 64), (stride, 64, 1), off)
            out = torch.empty(7, 3, 64, dtype=q.dtype, device="cuda")
            pos = rng.integers(0, 9999, 7).astype(np.int32)
            for near in (False, True):
                fs.fs_rope(q, _t(pos), f, q_out=out, interleaved=near)
                check(out, q, pos, f, 1.0, near)


def test_many_heads_and_rows():
    import torch
    rng = np.random.default_rng(5)
    f, _ = fs.fs_rope_frequencies(128)
    q, k = (torch.randn(3001, h, 128, device="cuda").bfloat16() for h in (64, 8))
    pos = rng.integers(0, 1 << 20, 3001).astype(np.int32)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    fs.fs_rope(q, _t(pos), f, k=k, q_out=qo, k_out=ko)
    some = rng.integers(0, 3001, 40)
    check(qo[some], q[some], pos[some], f, 1.0, False)
    check(ko[some], k[some], pos[some], f, 1.0, False)
    # one row has the bits that it has in a batch
    one = torch.empty_like(q[:1])
    fs.fs_rope(q[77:78], _t(pos[77:78]), f, q_out=one)
    assert (one == qo[77:78]).all()
