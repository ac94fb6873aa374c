"""GPU: fs_sample_filtered on the logits that fs_decode_step_batch writes, on the handle's
stream without waiting in between, its tokens fed to the next step; against the rule in 64
bits on the same logits."""
import numpy as np
import pytest

from continuous_transformer_decode_gb300 import fs, synth
from tests import _step_ref as R
from tests._gpu_util import make_gpu

pytestmark = pytest.mark.gpu
SMALL = dict(name="small-bf16", L=2, d=128, H=2, Hkv=1, hd=64, F=256, V=512, rms_eps=1e-5, rope_theta=1e4, tied=True)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from continuous_transformer_decode_gb300 import build
    build.build()


@pytest.mark.parametrize("cfg,fmt,dtype", [(synth.MODEL_T, "f32", fs.FS_DTYPE_F32), (SMALL, "bf16", fs.FS_DTYPE_BF16)], ids=["f32", "bf16"])
def test_tokens_of_steps(cfg, fmt, dtype):
    import torch
    lanes, V = [0, 2, 3, 5, 6], cfg["V"]
    n = len(lanes)
    rng = np.random.default_rng(7)
    T = np.array([0.0, 0.7, 1.0, 1.3, 0.9], np.float32)
    k = np.array([0, 20, 0, 5, 0], np.int32)
    p = np.array([1.0, 0.9, 0.8, 1.0, 1.0], np.float32)
    m = np.array([0.0, 0.0, 0.05, 0.1, 0.0], np.float32)
    dev = [torch.from_numpy(a).cuda() for a in (T, k, p, m)]
    h = make_gpu(cfg, synth.make_weights(cfg, seed=3, fmt=fmt), dtype)
    stream = torch.cuda.Stream()
    try:
        fs.fs_set_stream(h, stream)
        tokens, seen = [3, 1, 4, 1, 5], set()
        for step in range(12):
            u = rng.random(n).astype(np.float32)
            with torch.cuda.stream(stream):
                buf = torch.empty((n, V), device="cuda")
                ud, tok = torch.from_numpy(u).cuda(), torch.empty(n, dtype=torch.int32, device="cuda")
                kept = torch.empty_like(tok)
                fs.fs_decode_step_batch(h, lanes, np.full(n, step, np.int32), tokens, logits_out=buf)
                fs.fs_sample_filtered(buf, dev[0], ud, tok, top_k=dev[1], top_p=dev[2], min_p=dev[3], kept=kept)
            stream.synchronize()
            z = buf.cpu().numpy()
            want = [R.sample(*r) for r in zip(z, T, u, k, p, m)]
            assert tok.tolist() == [w[0] for w in want] and kept.tolist() == [w[1] for w in want]
            tokens = tok.tolist()
            assert tokens[0] == int(np.argmax(z[0]))
            seen |= set(tokens)
        assert len(seen) > 4
    finally:
        fs.fs_destroy(h)
