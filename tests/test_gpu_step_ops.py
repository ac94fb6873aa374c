"""GPU: the operators for what differs from request to request, run together as a batched
step does: pages and rows, the projection with each row's adapter, rotary positions, the
8-bit cache and attention over it, and a token a row; then a draft's rejected tokens leave.
Each stage is compared with 64 bits from the stage's own inputs."""
import numpy as np
import pytest

from continuous_transformer_decode_gb300 import fs
from tests import _q8_ref as Q
from tests import _step_ref as R

pytestmark = pytest.mark.gpu
D, H, HKV, HD, PAGE, LANES, WIDE, RANK, ADAPTERS, VOCAB = 256, 4, 2, 64, 8, 6, 12, 16, 3, 500
N = (H + 2 * HKV) * HD


@pytest.fixture(scope="module", autouse=True)
def _built():
    from continuous_transformer_decode_gb300 import build
    build.build()


def _np(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


class Step:
    """Weights, a cache, a pool, and buffers for up to `rows` rows."""

    def __init__(self, rows, seed=0):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        f = lambda *s: torch.randn(*s, generator=g, device="cuda")
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
        self.rows, self.gen = rows, g
        self.W = (f(N, D) * D**-0.5).bfloat16()
        self.A, self.B = (f(ADAPTERS, RANK, D) * D**-0.5).bfloat16(), (f(ADAPTERS, N, RANK) * RANK**-0.5).bfloat16()
        self.scale = torch.rand(ADAPTERS, generator=g, device="cuda") + 0.5
        self.adapter_of_lane = torch.tensor([0, 2, -1, 1, 1, 0], dtype=torch.int32, device="cuda")
        self.head = f(VOCAB, H * HD) * (H * HD)**-0.5
        self.freq, self.factor = fs.fs_rope_frequencies(HD, 10000.0, dict(kind="bands", factor=4.0, original=64))
        n_pages = 50
        self.holders, self.table, self.lengths = i32(n_pages), i32(LANES, WIDE) - 1, i32(LANES)
        self.holders[::7] = 1  # somebody else's
        u8 = lambda: torch.full((n_pages, HKV, PAGE, HD), 128, dtype=torch.uint8, device="cuda")
        sc = lambda: torch.zeros(n_pages, HKV, PAGE, device="cuda")
        self.cache = fs.fs_kv_q8_view(u8(), u8(), sc(), sc(), self.table)
        self.grow, self.keep = i32(LANES), i32(LANES) + 1000
        self.row_start, self.lane, self.pos, self.len = i32(LANES + 1), i32(rows), i32(rows), i32(rows)
        self.slot, self.status = torch.zeros(rows, dtype=torch.int64, device="cuda"), i32(4)
        self.x = f(rows, D).bfloat16()
        self.y, self.out, self.tok, self.kept = f(rows, N), f(rows, H, HD), i32(rows), i32(rows)
        self.temps, self.u = torch.rand(rows, generator=g, device="cuda") + 0.3, torch.rand(rows, generator=g, device="cuda")
        self.top_k, self.top_p = i32(rows) + 40, torch.full((rows,), 0.9, device="cuda")
        ws = fs.fs_kv_q8_attention_workspace(self.cache, rows, H, WIDE * PAGE, 64)
        self.ws = torch.empty(max(ws, 16), dtype=torch.uint8, device="cuda")

    def pages(self):
        fs.fs_pages_update(self.holders, self.table, self.lengths, self.grow, PAGE, self.status, keep=self.keep,
                           row_start=self.row_start, row_lane=self.lane, row_position=self.pos, row_length=self.len,
                           row_slot=self.slot)

    def heads(self):
        return (self.y[:, :H * HD].unflatten(1, (H, HD)), self.y[:, H * HD:(H + HKV) * HD].unflatten(1, (HKV, HD)),
                self.y[:, (H + HKV) * HD:].unflatten(1, (HKV, HD)))

    def adapters(self):
        import torch
        mine = torch.where(self.lane >= 0, self.adapter_of_lane[self.lane.clamp(min=0)], -1).to(torch.int32)
        fs.fs_lora_add(self.x, mine, self.A, self.B, self.scale, self.y, base=self.y)
        return mine

    def rope(self):
        q, k, _ = self.heads()
        fs.fs_rope(q, self.pos, self.freq, k=k, factor=self.factor)

    def attend(self):
        q, k, v = self.heads()
        fs.fs_kv_q8_append(self.cache, k, v, self.lane, self.pos)
        fs.fs_kv_q8_attention(self.cache, q, self.lane, self.len, self.out, max_len=WIDE * PAGE, split_len=64, workspace=self.ws)

    def sample(self):
        import torch
        self.logits = torch.matmul(self.out.flatten(1), self.head.T) * 4
        fs.fs_sample_filtered(self.logits, self.temps, self.u, self.tok, top_k=self.top_k, top_p=self.top_p, kept=self.kept)


def test_steps_of_a_batch():
    import torch
    s = Step(rows=64)
    host = dict(holders=_np(s.holders), table=_np(s.table), lengths=_np(s.lengths))
    for step, (grow, keep) in enumerate([([9, 3, 0, 17, 1, 8], None), ([1] * 6, None), ([4, 4, 1, 4, 1, 1], None),
                                         ([1, 1, 1, 1, 0, 12], [11, 9, 3, 20, 0, 0]), ([1] * 6, None)]):
        s.grow.copy_(torch.tensor(grow))
        s.keep.copy_(torch.tensor(keep if keep else [1000] * LANES))
        s.x.copy_(torch.randn(s.rows, D, generator=s.gen, device="cuda"))
        s.pages()
        want = R.pages_update(**host, grow=np.array(grow), page=PAGE, keep=None if keep is None else np.array(keep), max_rows=s.rows)
        torch.cuda.synchronize()
        host = {k: want[k] for k in host}
        assert s.status.tolist() == list(want["status"]) and want["status"][0] == 0
        for k, t in (("holders", s.holders), ("table", s.table), ("lengths", s.lengths), ("row_lane", s.lane),
                     ("row_position", s.pos), ("row_length", s.len), ("row_slot", s.slot)):
            assert np.array_equal(_np(t), want[k]), k
        n = int(want["status"][1])
        # the shared projection, then each row's adapter in place
        fs.fs_gemm_bf16_noalloc(s.W, s.x, s.y)
        base = s.y.clone()
        mine = s.adapters()
        ref, terms, _ = R.lora(_np(s.x), _np(mine), _np(s.A), _np(s.B), _np(s.scale), _np(base))
        tol = (D / 16 + RANK / 8 + 40) * 2.0**-23 * terms + 2.0**-24 * (np.abs(ref) + np.abs(_np(base)) + terms)
        assert (np.abs(_np(s.y) - ref) <= tol).all()
        assert torch.equal(s.y[n:], base[n:])  # padding
        # rotary positions of the row's own place
        q0, k0, _ = (_np(t) for t in s.heads())
        s.rope()
        q, k, v = s.heads()
        pos = _np(s.pos)
        for got, x in ((q, q0), (k, k0)):
            ref = R.rotate(x[:n], pos[:n], s.freq, s.factor)
            pair = np.abs(x[:n]) + np.abs(np.roll(x[:n], HD // 2, -1))
            assert (np.abs(_np(got)[:n] - ref) <= (6 * 2.0**-24 + 2.0**-30) * s.factor * pair).all()
            assert np.array_equal(_np(got)[n:], x[n:])
        # the cache: a row is where row_slot says, half a code off at most
        s.attend()
        codes, scales = s.cache.tensors[0], s.cache.tensors[2]
        at = s.slot[:n]
        kept = (codes.transpose(1, 2).flatten(0, 1)[at].double() - 128) * scales.transpose(1, 2).flatten(0, 1)[at].double()[..., None]
        amax = k[:n].double().abs().amax(-1, keepdim=True)
        assert ((kept - k[:n].double()).abs() <= amax * (0.5 / 127 + 2.0**-22)).all()
        c = Q.Cache(*(t.cpu().numpy() for t in s.cache.tensors[:2]), *(t.cpu().numpy() for t in s.cache.tensors[2:4]), s.table.cpu().numpy())
        ref, tol = Q.attention(c, _np(q)[:n], _np(s.lane)[:n], _np(s.len)[:n], HD**-0.5)
        assert (np.abs(_np(s.out)[:n] - ref) <= tol + 2.0**-24 * np.abs(ref)).all()
        assert (s.out[n:] == 0).all()
        s.sample()
        zs, ts, us = s.logits.cpu().numpy(), s.temps.cpu().numpy(), s.u.cpu().numpy()
        ref = [R.sample(zs[i], ts[i], us[i], 40, np.float32(0.9)) for i in range(s.rows)]
        assert s.tok.tolist() == [r[0] for r in ref] and s.kept.tolist() == [r[1] for r in ref]


def test_a_captured_step_replayed_is_the_eager_one():
    """Pages to tokens in one graph, on a stream of its own, beside the same calls made one
    by one; two graphs of two batches at once."""
    import torch
    eager, graphed = [Step(24, seed) for seed in (3, 4)], [Step(24, seed) for seed in (3, 4)]

    def calls(s):
        s.pages()
        s.adapters()
        s.rope()
        s.attend()
        s.sample()

    graphs, streams = [], [torch.cuda.Stream() for _ in graphed]
    for s, st in zip(graphed, streams):
        start = {k: v.clone() for k, v in vars(s).items() if hasattr(v, "clone")}
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            calls(s)  # once before the capture: the product's workspace
        st.synchronize()
        for k, v in start.items():
            getattr(s, k).copy_(v)
        for t in s.cache.tensors[:2]:
            t.fill_(128)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            calls(s)
        graphs.append(g)
    rng = np.random.default_rng(5)
    for step in range(6):
        grow = torch.tensor(rng.integers(0, 4, LANES), dtype=torch.int32)
        keep = torch.tensor(np.where(rng.random(LANES) < 0.2, 0, rng.integers(3, 60, LANES)), dtype=torch.int32)
        y = torch.randn(24, N, device="cuda")
        for s in eager + graphed:
            s.grow.copy_(grow), s.keep.copy_(keep), s.y.copy_(y)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        for s in eager:
            calls(s)
        torch.cuda.synchronize()
        for a, b in zip(eager, graphed):
            for k in ("status", "holders", "table", "lengths", "lane", "pos", "slot", "y", "out", "tok", "kept"):
                assert torch.equal(getattr(a, k), getattr(b, k)), (step, k)


def test_calls_without_a_stream_run_on_torchs_current_one():
    """Inputs made on a side stream by slow work, the operators called inside it without a
    stream of their own."""
    import torch
    side = torch.cuda.Stream()
    want = Step(16, 9)
    want.grow.fill_(2)
    want.pages(), want.adapters(), want.rope(), want.attend(), want.sample()
    s = Step(16, 9)
    torch.cuda.synchronize()
    big = torch.randn(4096, 4096, device="cuda")
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        for _ in range(20):
            big = big @ big * 1e-3
        s.grow.fill_(2)  # behind the products
        s.pages(), s.adapters(), s.rope(), s.attend(), s.sample()
    side.synchronize()
    for k in ("status", "y", "out", "tok", "kept"):
        assert torch.equal(getattr(s, k), getattr(want, k)), k
