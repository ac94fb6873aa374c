"""GPU: a decode handle whose KV arena is quantised as it is written (kv_dtype
FS_DTYPE_Q8_ROW): the decode and chunked steps run on the 8-bit cache operators,
export reads it back, clone and evict move its rows; and a speculative step, from
the drafted rows to the next token, on fs_step_batch_chunked, fs_verify_draft and
fs_lane_evict.

The reference is the f64 brute force of the whole model with keys and values
rounded to their 8-bit rows. With f32 weights the handle's logits are within 2e-3
of it as the f32 handle's are (the parity tests), and a projection that differs by
f32 rounding moves about one code in ten thousand by a step: of some 20000 codes
two, each a step of amax / 127 (0.024 deviations) in one of 64 elements of one
token. In a value that is at most 0.024 of one attention weight; in a key it turns
a score by 0.024 |q_d| / 8, and the weight by 1 %: both below 3e-3 of a logit of
unit deviation through weights of 0.02. So 5e-3.
"""
from unittest import mock

import numpy as np
import pytest

from continuous_transformer_decode_gb300 import fs, synth
from tests import _f64_model as F
from tests import _gpu_util as U
from tests import _q8_ref as R
from tests import test_gpu_chunked as chunked

pytestmark = pytest.mark.gpu

Q8 = fs.FS_DTYPE_Q8_ROW
SMALL = dict(name="small-q8kv", L=2, d=128, H=4, Hkv=2, hd=64, F=256, V=512, rms_eps=1e-5,
             rope_theta=1e4, tied=True)
WIDE = dict(SMALL, name="wide-q8kv", H=2, Hkv=1, hd=256)
MAX_ABS = 5e-3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from continuous_transformer_decode_gb300 import build
    build.build()


def _rows(a):
    codes, scale = R.quantise(a)
    return codes * scale[..., None]


def _reference(cfg, W, toks):
    with mock.patch.object(F, "_bf16_round", _rows):
        return F.forward_logits(cfg, W, toks, kv_bf16=True)


def _feed(h, lane, toks, V):
    import torch
    out = []
    for t in toks:
        pos = np.array([fs.fs_lane_length(h, lane)], np.int32)
        buf = torch.empty((1, V), dtype=torch.float32, device="cuda")
        fs.fs_decode_step_batch(h, [lane], pos, [int(t)], logits_out=buf)
        torch.cuda.synchronize()
        out.append(buf.cpu().numpy()[0])
    return np.stack(out)


@pytest.mark.parametrize("cfg,page_size,max_pos", [(SMALL, 16, 64), (SMALL, 7, 900), (WIDE, 24, 64)])
def test_decode_matches_the_model_with_8_bit_rows(cfg, page_size, max_pos):
    W = synth.make_weights(cfg, seed=1, fmt="f32")
    h = U.make_gpu(cfg, W, fs.FS_DTYPE_F32, Q8, max_lanes=3, max_pos=max_pos, page_size=page_size)
    try:
        assert fs.fs_attention_path(h) == "q8-mma"
        prompts = [[int(t) for t in p] for p in synth.make_prompts(3, [40, 23, 31], cfg["V"], seed=2)]
        got = U.gpu_teacher_forced(h, cfg, [0, 1, 2], prompts, cfg["V"])
        for g, p in zip(got, prompts):
            U.compare_logits(g, _reference(cfg, W, p), MAX_ABS, 0.9999)
        assert fs.fs_device_error(h) == 0
    finally:
        fs.fs_destroy(h)


@pytest.mark.parametrize("act_split", [0, 1])
def test_decode_bf16_weights(act_split):
    """The tensor-core path: within the bf16 tolerances of the parity tests of the
    model on the same weights."""
    W = synth.make_weights(SMALL, seed=3, fmt="bf16")
    Wf = {k: (synth.bf16_to_f32(v) if getattr(v, "dtype", None) == np.uint16 else v)
          for k, v in W.items() if k != "layers"}
    Wf["layers"] = [{k: (synth.bf16_to_f32(v) if v.dtype == np.uint16 else v) for k, v in ly.items()}
                    for ly in W["layers"]]
    h = U.make_gpu(SMALL, W, fs.FS_DTYPE_BF16, Q8, max_lanes=2, max_pos=300, act_split=act_split)
    try:
        toks = [int(t) for t in synth.make_prompts(1, 50, SMALL["V"], seed=4)[0]]
        U.compare_logits(_feed(h, 1, toks, SMALL["V"]), _reference(SMALL, Wf, toks), 5e-2, 0.9995)
    finally:
        fs.fs_destroy(h)


@pytest.mark.parametrize("max_pos", [200, 5000])
def test_chunked_equals_one_token_steps(max_pos):
    cfg = synth.with_layers(synth.MODEL_S, 2)
    W = synth.make_weights(cfg, seed=1, fmt="bf16")
    chunked._compare(cfg, W, fs.FS_DTYPE_BF16, Q8, max_pos, "q8-mma")


def test_import_export_clone_and_evict():
    cfg = SMALL
    W = synth.make_weights(cfg, seed=1, fmt="f32")
    h = U.make_gpu(cfg, W, fs.FS_DTYPE_F32, Q8, max_lanes=5, max_pos=96, page_size=16)
    n = 45
    kv = [synth.make_kv(n, cfg["Hkv"], cfg["hd"], seed=5, path=(l,)) for l in range(cfg["L"])]
    K, V = (np.stack([x[i] for x in kv]) for i in range(2))
    try:
        fs.fs_lane_import_kv(h, 0, K, V)
        old = []
        for l in range(cfg["L"]):
            k, v = fs.fs_lane_export_kv(h, 0, l, cfg["Hkv"], cfg["hd"])
            # one f32 product of the code and the f32 scale
            assert np.allclose(k, _rows(K[l]), rtol=2.0 ** -22, atol=0)
            assert np.allclose(v, _rows(V[l]), rtol=2.0 ** -22, atol=0)
            old.append((k, v))
        fs.fs_lane_clone(h, 0, 2)
        for l in range(cfg["L"]):
            k, v = fs.fs_lane_export_kv(h, 2, l, cfg["Hkv"], cfg["hd"])
            assert np.array_equal(k, old[l][0]) and np.array_equal(v, old[l][1])
        # both go on alike, and apart from a third lane
        fs.fs_lane_import_kv(h, 3, K[:, :20], V[:, :20])
        a, b = _feed(h, 0, [5, 6, 7, 8], cfg["V"]), _feed(h, 2, [5, 6, 7, 8], cfg["V"])
        assert np.array_equal(a, b)
        # evict: values move as they are, keys are turned back and quantised anew
        cut, end = 11, 30
        fs.fs_lane_evict(h, 2, cut, end)
        m = n + 4 - (end - cut)
        assert fs.fs_lane_length(h, 2) == m
        cos, sin = R.rope_tables(end, cfg["hd"])
        for l in range(cfg["L"]):
            k0, v0 = fs.fs_lane_export_kv(h, 0, l, cfg["Hkv"], cfg["hd"])
            k, v = fs.fs_lane_export_kv(h, 2, l, cfg["Hkv"], cfg["hd"])
            assert np.array_equal(v, np.concatenate([v0[:cut], v0[end:]]))
            assert np.array_equal(k[:cut], k0[:cut])
            moved = R.rotate(k0[end:], cos[[end - cut]], -sin[[end - cut]])
            amax = np.abs(moved).max(-1, keepdims=True)
            # half a step of 1 / 127, and f32 arithmetic
            assert (np.abs(k[cut:] - moved) <= amax * (0.5 / 127 + 2.0 ** -18)).all()
        # lane 0, which shares pages with the clone, is as it was
        for l in range(cfg["L"]):
            k, v = fs.fs_lane_export_kv(h, 0, l, cfg["Hkv"], cfg["hd"])
            assert np.array_equal(k[:n], old[l][0]) and np.array_equal(v[:n], old[l][1])
        fs.fs_lane_evict(h, 0, n, n + 4)  # a suffix: nothing moves
        assert np.array_equal(_feed(h, 0, [5, 6, 7, 8], cfg["V"]), a)
        fs.fs_lane_fill_random_kv(h, 4, 33, 9)
        k, v = fs.fs_lane_export_kv(h, 4, 1, cfg["Hkv"], cfg["hd"])
        assert abs(k.std() - 1) < 0.05 and abs(v.std() - 1) < 0.05 and not np.array_equal(k, v)
    finally:
        fs.fs_destroy(h)


def test_evict_of_keys_near_the_largest_value():
    """A key turned back past the largest f32 is stored as an infinity is by the
    append: as the largest value, in a row with a finite scale."""
    cfg, n, cut, end = SMALL, 24, 3, 9
    h = U.make_gpu(cfg, synth.make_weights(cfg, seed=1, fmt="f32"), fs.FS_DTYPE_F32, Q8,
                   max_lanes=1, max_pos=64, page_size=16)
    rng = np.random.default_rng(12)
    shape = (cfg["L"], n, cfg["Hkv"], cfg["hd"])
    K = (3.2e38 * rng.choice([-1.0, 1.0], shape)).astype(np.float32)
    V = rng.standard_normal(shape).astype(np.float32)
    big = float(np.finfo(np.float32).max)
    cos, sin = R.rope_tables(end, cfg["hd"])
    try:
        fs.fs_lane_import_kv(h, 0, K, V)
        old = [fs.fs_lane_export_kv(h, 0, l, cfg["Hkv"], cfg["hd"])[0] for l in range(cfg["L"])]
        fs.fs_lane_evict(h, 0, cut, end)
        for l in range(cfg["L"]):
            k = fs.fs_lane_export_kv(h, 0, l, cfg["Hkv"], cfg["hd"])[0].astype(np.float64)
            moved = R.rotate(old[l][end:], cos[[end - cut]], -sin[[end - cut]]).astype(np.float64)
            assert (np.abs(moved) > big).any()
            moved = np.clip(moved, -big, big)
            amax = np.abs(moved).max(-1, keepdims=True)
            assert np.isfinite(k).all()
            assert (np.abs(k[cut:] - moved) <= amax * (0.5 / 127 + 2.0 ** -18)).all()
    finally:
        fs.fs_destroy(h)


def test_speculative_step_end_to_end():
    """Three lanes, drafts of 4, 2 and 0 tokens: one chunked step scores them, the
    verification accepts a prefix, the rejected suffix leaves the cache; the lane
    then goes on, bit for bit, as one fed the accepted tokens one by one."""
    import torch
    cfg, V = SMALL, SMALL["V"]
    W = synth.make_weights(cfg, seed=1, fmt="f32")
    h = U.make_gpu(cfg, W, fs.FS_DTYPE_F32, Q8, max_lanes=16, max_pos=128, page_size=16)
    rng = np.random.default_rng(6)
    try:
        prompts = [[int(t) for t in p] for p in synth.make_prompts(3, [15, 31, 7], V, seed=7)]
        for k, p in enumerate(prompts):
            _feed(h, k, p[:-1], V)
        drafts = [4, 2, 0]
        # the draft model: the target's own logits over the first rows, sharpened
        lanes, pos, toks, start, draft, q = [], [], [], [0], [], []
        for k, p in enumerate(prompts):
            n = fs.fs_lane_length(h, k)
            z = _reference(cfg, W, p)[-1]
            prob = np.exp(2 * (z - z.max()))
            prob = (prob / prob.sum()).astype(np.float32)
            cand = rng.choice(V, size=drafts[k], p=prob.astype(np.float64) / prob.astype(np.float64).sum())
            row_toks = [p[-1]] + [int(c) for c in cand]
            lanes += [k] * len(row_toks)
            pos += list(range(n, n + len(row_toks)))
            toks += row_toks
            draft += row_toks[1:] + [-1]
            q += [prob] * len(row_toks)
            start.append(start[-1] + len(row_toks))
        rows = start[-1]
        logits = torch.empty(rows, V, device="cuda")
        fs.fs_step_batch_chunked(h, lanes, np.array(pos, np.int32), toks, logits_out=logits)
        c = dict(row_start=np.int32(start), draft=np.int32(draft), probs=np.stack(q),
                 temps=np.float32([0.7, 1.0, 0.0]), u_accept=rng.random(rows).astype(np.float32),
                 u_sample=rng.random(3).astype(np.float32))
        dev = {k: torch.from_numpy(v).cuda() for k, v in c.items()}
        acc, nxt = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
        fs.fs_verify_draft(logits, dev["row_start"], dev["draft"], dev["probs"], dev["temps"],
                           dev["u_accept"], dev["u_sample"], acc, nxt)
        torch.cuda.synchronize()
        # the logits of the step are the model's, and the answer is the rule's on them
        for k, p in enumerate(prompts):
            ref = _reference(cfg, W, p + toks[start[k] + 1:start[k + 1]])
            U.compare_logits(logits[start[k]:start[k + 1]].cpu().numpy(), ref[len(p) - 1:], MAX_ABS, 0.9999)
        want = R.verify(logits=logits.cpu().numpy(), **c)
        assert np.array_equal(acc.cpu().numpy(), want[0])
        assert np.array_equal(nxt.cpu().numpy(), want[1])
        for k, p in enumerate(prompts):
            a = int(want[0][k])
            fs.fs_lane_evict(h, k, len(p) + a, len(p) + drafts[k])
            fed = p + toks[start[k] + 1:start[k] + 1 + a]
            assert fs.fs_lane_length(h, k) == len(fed)
            _feed(h, 4 + k, fed, V)
            t = int(want[1][k])
            assert np.array_equal(_feed(h, k, [t], V), _feed(h, 4 + k, [t], V))
    finally:
        fs.fs_destroy(h)


def test_traced_steps_give_one_launch_per_kernel():
    import torch
    from continuous_transformer_decode_gb300 import trace as tr
    W = synth.make_weights(SMALL, seed=1, fmt="bf16")
    h = U.make_gpu(SMALL, W, fs.FS_DTYPE_BF16, Q8, max_lanes=4, max_pos=9000)
    try:
        lanes, pos = [0, 1, 2, 3], np.zeros(4, np.int32)
        out = torch.empty(4, dtype=torch.int32, device="cuda")
        for _ in range(3):
            fs.fs_decode_step_greedy(h, lanes, pos, [1, 2, 3, 4], out)
        torch.cuda.synchronize()
        fs.fs_trace_enable(h, 1 << 16)
        l0 = fs.fs_kernel_launches(h)
        for _ in range(2):
            fs.fs_decode_step_greedy(h, lanes, pos, [1, 2, 3, 4], out)
        recs, n = fs.fs_trace_read(h)
        launched = fs.fs_kernel_launches(h) - l0
        names = [x["name"] for x in tr.launches(recs)]
        assert len(names) == launched
        assert names.count("kv_q8_append") == names.count("attn_q8") == names.count("attn_q8_join") == 4
    finally:
        fs.fs_destroy(h)


def test_refused_shapes():
    cfg = dict(SMALL, hd=32)
    W = synth.make_weights(cfg, seed=1, fmt="f32")
    with pytest.raises(fs.FsError):
        U.make_gpu(cfg, W, fs.FS_DTYPE_F32, Q8, max_lanes=2, max_pos=64)


def test_operators_leave_no_marks_in_a_handles_trace():
    """The trace holds the handle's steps: a call on the caller's own cache, whatever
    its stream, neither fills it nor holds its buffer."""
    from tests.test_gpu_kv_q8 import Pages, _attend, _cuda
    h = U.make_gpu(SMALL, synth.make_weights(SMALL, seed=1, fmt="f32"), fs.FS_DTYPE_F32, Q8,
                   max_lanes=2, max_pos=64)
    rng = np.random.default_rng(13)
    pg = Pages(rng, [300], 2, 64, 16)
    q = rng.standard_normal((1, 4, 64)).astype(np.float32)
    try:
        fs.fs_trace_enable(h, 1 << 12)
        _attend(pg, _cuda(q), [0], [300], split_len=64)   # split, so joined too
        recs, n = fs.fs_trace_read(h)
        assert n == 0 and len(recs) == 0
    finally:
        fs.fs_destroy(h)
