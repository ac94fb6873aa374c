"""Argument checks of the 8-bit cache operators and of draft verification: they
come before any CUDA call, so they run without a GPU (the addresses below are
never read)."""
import ctypes as C

import pytest

from continuous_transformer_decode_gb300 import build, fs

ARG, SCRATCH = fs.CODES["FS_ERR_ARG"], fs.CODES["FS_ERR_SCRATCH"]
P = 1 << 20  # an aligned address


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def cache(**kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, page_table=P, n_pages=4, n_kv_heads=2, page_size=16,
             head_dim=64, n_lanes=2, max_pages=2)
    d.update(kw)
    return fs.fs_kv_q8(*[d[f] for f, _ in fs.fs_kv_q8._fields_])


def append(c=None, **kw):
    d = dict(k=P, v=P, ks=128, vs=128, dtype=0, lanes=P, pos=P, n=3, cos=None, sin=None, rl=0)
    d.update(kw)
    return fs.lib().fs_kv_q8_append(C.byref(c or cache()), d["k"], d["v"], d["ks"], d["vs"],
                                    d["dtype"], d["lanes"], d["pos"], d["n"], d["cos"], d["sin"],
                                    d["rl"], None)


def read(c=None, **kw):
    d = dict(k=P, v=P, ks=128, vs=128, dtype=0, lanes=P, pos=P, n=3)
    d.update(kw)
    return fs.lib().fs_kv_q8_read(C.byref(c or cache()), d["lanes"], d["pos"], d["n"], d["k"],
                                  d["v"], d["ks"], d["vs"], d["dtype"], None)


def attend(c=None, **kw):
    d = dict(q=P, qs=256, lanes=P, lens=P, n=3, H=4, max_len=32, scale=0.125, cos=None, sin=None,
             rl=0, out=P, os=256, dtype=0, split=64, ws=None, wb=0)
    d.update(kw)
    return fs.lib().fs_kv_q8_attention(
        C.byref(c or cache()), d["q"], d["qs"], d["lanes"], d["lens"], d["n"], d["H"], d["max_len"],
        d["scale"], d["cos"], d["sin"], d["rl"], d["out"], d["os"], d["dtype"], d["split"], d["ws"],
        d["wb"], None)


def verify(**kw):
    d = dict(logits=P, ld=100, rows=5, V=100, start=P, n=2, draft=P, probs=P, lp=100, temps=P, ua=P,
             us=P, acc=P, nxt=P)
    d.update(kw)
    return fs.lib().fs_verify_draft(d["logits"], d["ld"], d["rows"], d["V"], d["start"], d["n"],
                                    d["draft"], d["probs"], d["lp"], d["temps"], d["ua"], d["us"],
                                    d["acc"], d["nxt"], None)


BAD_CACHE = [dict(head_dim=32), dict(head_dim=96), dict(head_dim=0), dict(page_size=0),
             dict(n_kv_heads=0), dict(max_pages=0), dict(n_pages=0), dict(n_lanes=0),
             dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None),
             dict(page_table=None), dict(k=P + 8), dict(v=P + 1), dict(k_scale=P + 2),
             dict(page_table=P + 1), dict(max_pages=1 << 27),
             dict(n_pages=1 << 27)]


@pytest.mark.parametrize("bad", BAD_CACHE)
@pytest.mark.parametrize("call", [append, read, attend])
def test_bad_cache(call, bad):
    assert call(cache(**bad)) == ARG
    assert fs.fs_last_error(None)


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(dtype=-1), dict(n=-1), dict(k=None), dict(v=None), dict(ks=127),
    dict(vs=0), dict(k=P + 2), dict(v=P + 1, dtype=1), dict(lanes=None), dict(pos=None),
    dict(lanes=P + 2), dict(cos=P), dict(sin=P), dict(cos=P, sin=P, rl=0),
    dict(cos=P + 2, sin=P, rl=8), dict(n=(1 << 31) - 1)])
def test_append(bad):
    assert append(**bad) == ARG


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(n=-1), dict(ks=127), dict(vs=-5), dict(k=P + 2), dict(v=P + 1, dtype=1),
    dict(lanes=None), dict(pos=None), dict(pos=P + 1)])
def test_read(bad):
    assert read(**bad) == ARG


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(n=-1), dict(n=65536), dict(H=0), dict(H=3), dict(H=18), dict(max_len=-1),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(split=-64), dict(split=96),
    dict(split=(1 << 30) + 64), dict(q=None), dict(out=None), dict(qs=255), dict(os=255),
    dict(q=P + 2), dict(lanes=None), dict(lens=None), dict(lens=P + 1), dict(cos=P),
    dict(cos=P, sin=P, rl=31)])
def test_attention(bad):
    assert attend(**bad) == ARG


def test_attention_workspace():
    c = cache(max_pages=16)
    size = fs.fs_kv_q8_attention_workspace(c, 3, 4, 200, 64)
    assert size == 3 * 4 * 4 * (64 + 2) * 4  # 4 splits of 3 rows of 4 heads
    assert fs.fs_kv_q8_attention_workspace(c, 3, 4, 64, 64) == 0
    assert fs.fs_kv_q8_attention_workspace(c, 3, 4, 0, 64) == size  # 0: the capacity, 256 tokens
    assert fs.fs_kv_q8_attention_workspace(c, 3, 4, 1000, 64) == size
    assert attend(c, max_len=200) == SCRATCH
    assert attend(c, max_len=200, ws=P, wb=size - 1) == SCRATCH
    assert attend(c, max_len=200, ws=P + 8, wb=size) == ARG
    with pytest.raises(fs.FsError):
        fs.fs_kv_q8_attention_workspace(c, 3, 5, 200, 64)
    with pytest.raises(fs.FsError):
        fs.fs_kv_q8_attention_workspace(c, 3, 4, 200, 65)
    long = cache(max_pages=1 << 20)
    assert fs.fs_kv_q8_attention_workspace(long, 1, 4, 8192 * 64, 64) > 0
    with pytest.raises(fs.FsError):
        fs.fs_kv_q8_attention_workspace(long, 1, 4, 8192 * 64 + 1, 64)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(n=-1), dict(V=0), dict(logits=None), dict(ld=99), dict(lp=99),
    dict(logits=P + 2), dict(draft=None), dict(ua=None), dict(us=None), dict(start=None),
    dict(temps=None), dict(acc=None), dict(nxt=None), dict(draft=P + 2), dict(temps=P + 1),
    dict(nxt=P + 3)])
def test_verify(bad):
    assert verify(**bad) == ARG


def test_no_rows_is_no_work():
    assert append(n=0, k=None, v=None, lanes=None, pos=None) == 0
    assert read(n=0) == 0
    assert read(k=None, v=None) == 0
    assert attend(n=0, q=None) == 0
    assert verify(n=0) == 0
    assert append(n=0, dtype=5) == ARG  # still an invalid call


def test_null_cache():
    assert fs.lib().fs_kv_q8_read(None, P, P, 1, P, P, 64, 64, 0, None) == ARG


def test_binding_refuses_tensors_it_cannot_use():
    import torch
    z = torch.zeros
    codes, scale = z(2, 1, 16, 64, dtype=torch.uint8), z(2, 1, 16)
    with pytest.raises(fs.FsError):  # host tensors
        fs.fs_kv_q8_view(codes, codes, scale, scale, z(1, 1, dtype=torch.int32))
    with pytest.raises(fs.FsError):  # codes and scales of different shapes
        fs.fs_kv_q8_view(codes, codes, scale, z(2, 16, 1), z(1, 1, dtype=torch.int32))
    one = z(1, dtype=torch.int32)
    with pytest.raises(fs.FsError):
        fs.fs_kv_q8_append(cache(), z(1, 2, 64), z(1, 2, 64), one, one)
    with pytest.raises(fs.FsError):
        fs.fs_verify_draft(z(1, 8), z(2, dtype=torch.int32), one, None, z(1), z(1), z(1), one, one)


def test_no_stream_is_torchs_current_stream(monkeypatch):
    """A call that is given no stream goes to the current stream of its tensors' device,
    one that is given a stream to that."""
    import torch

    class OnDevice(torch.Tensor):  # a host tensor that says it is on device 0
        __torch_function__ = torch._C._disabled_torch_function_impl
        is_cuda = True

        def get_device(self):
            return 0

        @property
        def device(self):
            return torch.device("cuda", 0)

    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype).as_subclass(OnDevice)
    i32 = lambda *s: z(*s, dtype=torch.int32)
    got = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: got.append((name, a[-1])) or 0

    monkeypatch.setattr(fs, "lib", lambda: Lib())
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 4242 + d, raising=False)

    class Stream:
        cuda_stream = 77

    for given, want in ((None, 4242), (Stream(), 77), (55, 55)):
        got.clear()
        fs.fs_kv_q8_append(cache(), z(1, 2, 64), z(1, 2, 64), i32(1), i32(1), stream=given)
        fs.fs_kv_q8_read(cache(), i32(1), i32(1), z(1, 2, 64), stream=given)
        fs.fs_kv_q8_attention(cache(), z(1, 4, 64), i32(1), i32(1), z(1, 4, 64), stream=given)
        fs.fs_verify_draft(z(1, 8), i32(2), i32(1), None, z(1), z(1), z(1), i32(1), i32(1),
                           stream=given)
        assert got == [(n, want) for n in ("fs_kv_q8_append", "fs_kv_q8_read", "fs_kv_q8_attention",
                                           "fs_verify_draft")]


@pytest.mark.parametrize("shape", [(10, 64), (5, 64), (10, 16), (320,), (1, 10, 32), (0, 32)])
def test_rotation_tables_of_another_shape(shape):
    """Tables are [rope_len, head_dim / 2]: ones of the whole head_dim would be read as
    twice as many positions of the wrong angles, empty ones (which have no address) as
    no rotation."""
    import torch
    t = torch.zeros(shape)
    one = torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 2, 64)
    for call in (lambda: fs.fs_kv_q8_append(cache(), x, x, one, one, rope=(t, t)),
                 lambda: fs.fs_kv_q8_attention(cache(), x, one, one, x, rope=(t, t))):
        with pytest.raises(fs.FsError, match="rope"):
            call()
