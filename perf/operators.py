"""Operators of a decode step over an 8-bit paged KV cache, and of speculative decoding: the cases that are
measured, their inputs, and their plain forms.

Three operators, told apart by a case's "op":
  cache   keys (rotated by their position) and values of some tokens are quantised into the pages of their
          lanes, one f32 scale and head_dim 8-bit codes a (token, KV head), and read back
  attend  attention of one new token a lane over the lane's quantised pages, rows of every length at once
  verify  drafted tokens against the target's probabilities from given random numbers: how many are
          accepted, and the token that follows

The cache: codes k, v uint8 [pages, Hkv, page_size, hd], each a whole number in -127 .. 127 plus 128; scales f32
[pages, Hkv, page_size]; page_table int32 [lanes, max_pages]; token t of a lane is in slot t % page_size of the
lane's page t // page_size. A value stands for code * scale, with scale = amax / 127 and code = x * 127 / amax
rounded to the nearest whole number (ties to even), amax the row's largest magnitude (a row of zeros: scale 0).
"""
import math

import torch

own = False


def listed():
    """Shapes: 9 / 3 heads of 64 with a vocabulary of 49152 and 32 / 8 heads of 128 with one of 32000 are the two
    models that the tests and the benchmark run; the other shapes are generic."""
    return [
        # one lane's next token: the smallest call of the cache, where latency counts
        dict(name="cache-1-row", op="cache", rows=1, lanes=1, heads=9, kv=3, hd=64, page=16, io="f32"),
        # a decode step of 256 lanes, each at its own position
        dict(name="cache-256-lanes", op="cache", rows=256, lanes=256, heads=32, kv=8, hd=128, page=16, io="bf16"),
        # a prompt's chunk, an odd number of rows out of the f32 projection panel (rows of q, k and v side by side)
        dict(name="cache-4099-chunk", op="cache", rows=4099, lanes=3, heads=32, kv=8, hd=128, page=16, io="f32"),
        # whole prompts of many lanes
        dict(name="cache-65536-prompts", op="cache", rows=65536, lanes=16, heads=32, kv=8, hd=128, page=64, io="bf16"),
        # one short lane: latency
        dict(name="attend-1-short", op="attend", lanes=1, lo=17, hi=17, heads=9, kv=3, hd=64, page=16, empty=0, io="f32"),
        # full serving of the small model: many lanes, short contexts, a few lanes without tokens
        dict(name="attend-256-lanes", op="attend", lanes=256, lo=1, hi=512, heads=9, kv=3, hd=64, page=16, empty=5, io="f32"),
        # the larger model at 128 lanes, ragged contexts
        dict(name="attend-128-ragged", op="attend", lanes=128, lo=128, hi=4096, heads=32, kv=8, hd=128, page=16, empty=0, io="bf16"),
        # one lane with a very long context of odd length
        dict(name="attend-1-long", op="attend", lanes=1, lo=131071, hi=131071, heads=32, kv=8, hd=128, page=16, empty=0, io="bf16"),
        # wide heads, eight query heads a KV head, pages of 24 that end inside every tile
        dict(name="attend-33-wide", op="attend", lanes=33, lo=1, hi=3001, heads=16, kv=2, hd=256, page=24, empty=2, io="f32"),
        # one sequence with four drafted tokens
        dict(name="verify-1", op="verify", seqs=1, lo=4, hi=4, vocab=32000, probs=True, greedy=0.0),
        # 64 sequences with 0 to 7 drafted tokens each, a quarter of them greedy
        dict(name="verify-64-ragged", op="verify", seqs=64, lo=0, hi=7, vocab=49152, probs=True, greedy=0.25),
        # 256 sequences with four tokens each from a lookup in the prompt (no draft probabilities)
        dict(name="verify-256-lookup", op="verify", seqs=256, lo=4, hi=4, vocab=49152, probs=False, greedy=0.25),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cache", "attend", "attend", "verify"])
    if op == "verify":
        vocab = _spread(rng, 257, 49152)
        hi = rng.randint(0, 7)
        most = max(1, min(256, 256 * 5 * 49152 // ((hi + 1) * vocab) // (2 if hi > 4 else 1)))
        return dict(op=op, seqs=_spread(rng, 1, most), lo=rng.randint(0, hi), hi=hi, vocab=vocab, probs=rng.random() < 0.6,
                    greedy=rng.choice([0.0, 0.25, 1.0]))
    hd, kv = rng.choice([64, 128, 128, 256]), rng.randint(1, 8)
    group = rng.randint(1, 8)
    page = rng.choice([8, 16, 16, 24, 32, 64, rng.randint(1, 128)])
    io = rng.choice(["f32", "bf16"])
    if op == "cache":
        rows = _spread(rng, 1, 65536 * 1024 // (kv * hd) // (2 if io == "f32" else 1) // 2)
        return dict(op=op, rows=rows, lanes=min(rows, _spread(rng, 1, 256)), heads=kv * group, kv=kv, hd=hd, page=page, io=io)
    lanes = _spread(rng, 1, 256)
    hi = _spread(rng, 1, min(131072, 128 * 4096 * 1024 // (lanes * kv * hd) // 2))
    return dict(op=op, lanes=lanes, lo=rng.randint(1, hi), hi=hi, heads=kv * group, kv=kv, hd=hd, page=page, empty=rng.choice([0, 0, lanes // 5]), io=io)


# ------------------------------------------------------------------------------------------------ inputs
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _rope(positions, hd):
    """cos and sin f32 [positions, hd / 2] of p * 10000^(-2i / hd), from 64 bits."""
    inv = 10000.0 ** (-2.0 * torch.arange(hd // 2, dtype=torch.float64, device="cuda") / hd)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return a.cos().float(), a.sin().float()


def _codes(x):
    """Codes (uint8) and scales (f32) of the rows of x [..., hd]: the plain form of the quantiser. The quotient is
    taken in 64 bits, as a code lies next to the border of two whole numbers now and then."""
    amax = x.abs().amax(-1)
    scale = (amax.double() / 127.0).float()
    q = (x.double() * 127.0) / amax.double().clamp(min=1e-300)[..., None]
    return (q.round() + 128.0).to(torch.uint8), scale


def _pages(lens, page, gen):
    """A page table int32 [lanes, max_pages] that gives every lane room for lens + 1 tokens in scattered pages, and the number of pages."""
    need = [n // page + 1 for n in lens]
    total = sum(need)
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    width = max(need)
    count = torch.tensor(need, device="cuda")
    first = torch.cumsum(count, 0) - count
    at = (first[:, None] + torch.arange(width, device="cuda")).clamp(max=total - 1)
    inside = torch.arange(width, device="cuda") < count[:, None]
    return torch.where(inside, order[at], 0).to(torch.int32).contiguous(), total


def _prepare_cache(c, gen):
    rows, lanes, heads, kv, hd = c["rows"], c["lanes"], c["heads"], c["kv"], c["hd"]
    lane = torch.arange(rows, dtype=torch.int64, device="cuda") % lanes
    base = torch.randint(0, 200, (lanes,), generator=gen, device="cuda")  # tokens that a lane holds already
    pos = base[lane] + torch.arange(rows, device="cuda") // lanes
    lens = (base + rows // lanes + 1).tolist()
    table, total = _pages(lens, c["page"], gen)
    t = _TYPES[c["io"]]
    # one row of the projection: q, then k, then v
    panel = torch.randn(rows, (heads + 2 * kv) * hd, generator=gen, device="cuda").to(t)
    k = panel[:, heads * hd:(heads + kv) * hd].unflatten(1, (kv, hd))
    v = panel[:, (heads + kv) * hd:].unflatten(1, (kv, hd))
    shape = (total, kv, c["page"], hd)
    s = dict(op="cache", panel=panel, k=k, v=v, lanes=lane.to(torch.int32), positions=pos.to(torch.int32), rope=_rope(max(lens) + 1, hd),
             kc=torch.full(shape, 128, dtype=torch.uint8, device="cuda"), vc=torch.full(shape, 128, dtype=torch.uint8, device="cuda"),
             ks=torch.zeros(shape[:3], device="cuda"), vs=torch.zeros(shape[:3], device="cuda"), table=table,
             k_out=torch.empty(rows, kv, hd, dtype=t, device="cuda"), v_out=torch.empty(rows, kv, hd, dtype=t, device="cuda"))
    return s


def _prepare_attend(c, gen):
    n, heads, kv, hd, page = c["lanes"], c["heads"], c["kv"], c["hd"], c["page"]
    lens = torch.randint(c["lo"], c["hi"] + 1, (n,), generator=gen, device="cuda")
    if c["empty"]:
        lens[torch.randperm(n, generator=gen, device="cuda")[:c["empty"]]] = 0
    longest = int(lens.max())
    table, total = _pages(lens.tolist(), page, gen)
    shape = (total, kv, page, hd)
    kc, vc = torch.empty(shape, dtype=torch.uint8, device="cuda"), torch.empty(shape, dtype=torch.uint8, device="cuda")
    ks, vs = torch.empty(shape[:3], device="cuda"), torch.empty(shape[:3], device="cuda")
    step = max(1, (1 << 26) // (kv * page * hd))  # pages at a time
    for codes, scales in ((kc, ks), (vc, vs)):
        for p in range(0, total, step):
            codes[p:p + step], scales[p:p + step] = _codes(torch.randn(min(step, total - p), kv, page, hd, generator=gen, device="cuda"))
    t = _TYPES[c["io"]]
    return dict(op="attend", q=torch.randn(n, heads, hd, generator=gen, device="cuda").to(t), lanes=torch.randperm(n, generator=gen, device="cuda").to(torch.int32),
                lens=lens.to(torch.int32), longest=longest, kc=kc, vc=vc, ks=ks, vs=vs, table=table, rope=_rope(longest + 1, hd),
                out=torch.empty(n, heads, hd, dtype=t, device="cuda"))


def _prepare_verify(c, gen):
    n, vocab = c["seqs"], c["vocab"]
    drafts = torch.randint(c["lo"], c["hi"] + 1, (n,), generator=gen, device="cuda")
    start = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    start[1:] = torch.cumsum(drafts + 1, 0)
    rows = int(start[-1])
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), drafts + 1, output_size=rows)
    logits = torch.randn(rows, vocab, generator=gen, device="cuda") * 2.5
    greedy = torch.rand(n, generator=gen, device="cuda") < c["greedy"]
    temps = torch.where(greedy, 0.0, 0.6 + 0.6 * torch.rand(n, generator=gen, device="cuda"))
    other = logits + 0.7 * torch.randn(rows, vocab, generator=gen, device="cuda")  # the draft model's logits
    if c["probs"]:
        probs = torch.softmax(other / torch.where(temps > 0, temps, 1.0)[seq][:, None], -1)
        # a draw from probs: the largest of log(probs) + Gumbel noise; the greedy ones take the draft's largest
        noise = -torch.log(-torch.log(torch.rand(rows, vocab, generator=gen, device="cuda").clamp(1e-7, 1 - 1e-7)))
        draft = torch.where(greedy[seq], other.argmax(-1), (probs.log() + noise).argmax(-1))
    else:
        probs = None
        draft = torch.where(torch.rand(rows, generator=gen, device="cuda") < 0.7, other.argmax(-1), torch.randint(0, vocab, (rows,), generator=gen, device="cuda"))
    return dict(op="verify", logits=logits, start=start.to(torch.int32), draft=draft.to(torch.int32), probs=probs, temps=temps,
                u_accept=torch.rand(rows, generator=gen, device="cuda"), u_sample=torch.rand(n, generator=gen, device="cuda"),
                n_accepted=torch.empty(n, dtype=torch.int32, device="cuda"), next_token=torch.empty(n, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = {"cache": _prepare_cache, "attend": _prepare_attend, "verify": _prepare_verify}[case["op"]](case, gen)
    if own:
        from continuous_transformer_decode_gb300 import fs
        s["fs"] = fs
        if s["op"] != "verify":
            s["view"] = fs.fs_kv_q8_view(s["kc"], s["vc"], s["ks"], s["vs"], s["table"])
        if s["op"] == "attend":
            size = fs.fs_kv_q8_attention_workspace(s["view"], case["lanes"], case["heads"], s["longest"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _rotate(x, cos, sin):
    """The rotary positions of x [rows, heads, hd]: pairs (i, i + hd / 2), cos and sin [rows, hd / 2]."""
    half = x.shape[-1] // 2
    a, b = x[..., :half], x[..., half:]
    c, s = cos[:, None], sin[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _cache_plain(s):
    pos, lane = s["positions"].long(), s["lanes"].long()
    page = s["kc"].shape[2]
    where = s["table"][lane, pos // page].long()
    slot = pos % page
    cos, sin = s["rope"]
    k, ks = _codes(_rotate(s["k"].double(), cos[pos].double(), sin[pos].double()))  # 64 bits: see _codes
    v, vs = _codes(s["v"].float())
    s["kc"][where, :, slot], s["vc"][where, :, slot] = k, v
    s["ks"][where, :, slot], s["vs"][where, :, slot] = ks, vs
    for codes, scales, out in ((s["kc"], s["ks"], s["k_out"]), (s["vc"], s["vs"], s["v_out"])):
        out.copy_((codes[where, :, slot].float() - 128.0) * scales[where, :, slot][..., None])
    return {"k": s["k_out"], "v": s["v_out"]}


def _attend_plain(s):
    n, heads, hd = s["q"].shape
    kv, page = s["kc"].shape[1:3]
    lens = s["lens"].long()
    cos, sin = s["rope"]
    at = (lens - 1).clamp(min=0)
    q = _rotate(s["q"].float(), cos[at], sin[at]).view(n, kv, heads // kv, hd)
    wide = -(-s["longest"] // page)
    pages = s["table"][s["lanes"].long(), :wide].long()

    def values(codes, scales):
        x = (codes[pages].float() - 128.0) * scales[pages][..., None]
        return x.transpose(1, 2).reshape(n, kv, wide * page, hd)

    seen = (torch.arange(wide * page, device="cuda") < lens[:, None])[:, None, None]
    z = torch.matmul(q, values(s["kc"], s["ks"]).transpose(-1, -2)) * hd ** -0.5
    z = torch.where(seen, z, -math.inf)
    top = z.amax(-1, keepdim=True)
    w = torch.where(seen, (z - torch.where(top > -math.inf, top, 0.0)).exp(), 0.0)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, values(s["vc"], s["vs"])) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(o.view(n, heads, hd))
    return s["out"]


def _verify_plain(s):
    logits, start, probs, temps = s["logits"], s["start"].long(), s["probs"], s["temps"]
    rows, vocab = logits.shape
    n = temps.numel()
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), start.diff(), output_size=rows)
    place = torch.arange(rows, device="cuda") - start[seq]  # a row's place in its sequence
    drafts = start.diff() - 1
    index = torch.arange(vocab, device="cuda")
    draft = s["draft"].long()[:, None]
    t = torch.where(temps > 0, temps, 1.0)[seq][:, None]
    top = logits.amax(-1, keepdim=True)
    best = torch.where(logits == top, index, vocab).amin(-1)
    # the chance of the drafted token; the sum in 64 bits
    p = ((logits.gather(1, draft) - top).double() / t.double()).exp() / ((logits - top) / t).exp().sum(-1, keepdim=True, dtype=torch.float64)
    q = probs.gather(1, draft).double() if probs is not None else 1.0
    fine = torch.where(temps[seq] > 0, (s["u_accept"].double()[:, None] * q < p)[:, 0], best == draft[:, 0])
    stop = torch.where(fine | (place == drafts[seq]), vocab, place)
    accepted = drafts.scatter_reduce(0, seq, stop, "amin")
    # the next token, from what is left of the target's probabilities: running sums in 64 bits, as a
    # number may lie next to the border of two tokens
    row = start[:-1] + accepted
    e = ((logits[row].double() - top[row].double()) / t[row].double()).exp()
    p = e / e.sum(-1, keepdim=True)
    taken = probs[row].double() if probs is not None else torch.where(index == draft[row], p, 0.0)
    left = torch.where((accepted < drafts)[:, None], (p - taken).clamp(min=0.0), p)
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, p)
    run_sum = left.cumsum(-1)
    target = s["u_sample"].double()[:, None] * run_sum[:, -1:]
    token = torch.where((run_sum >= target) & (left > 0), index, vocab).amin(-1)
    last = torch.where(left > 0, index, -1).amax(-1)
    token = torch.where(temps > 0, torch.where(token < vocab, token, last), best[row])
    s["n_accepted"].copy_(accepted)
    s["next_token"].copy_(token)
    return {"accepted": s["n_accepted"], "next": s["next_token"]}


def run(state):
    s = state
    if not own:
        return {"cache": _cache_plain, "attend": _attend_plain, "verify": _verify_plain}[s["op"]](s)
    fs = s["fs"]
    if s["op"] == "cache":
        fs.fs_kv_q8_append(s["view"], s["k"], s["v"], s["lanes"], s["positions"], rope=s["rope"])
        fs.fs_kv_q8_read(s["view"], s["lanes"], s["positions"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if s["op"] == "attend":
        fs.fs_kv_q8_attention(s["view"], s["q"], s["lanes"], s["lens"], s["out"], max_len=s["longest"], rope=s["rope"], workspace=s["workspace"])
        return s["out"]
    fs.fs_verify_draft(s["logits"], s["start"], s["draft"], s["probs"], s["temps"], s["u_accept"], s["u_sample"], s["n_accepted"], s["next_token"])
    return {"accepted": s["n_accepted"], "next": s["next_token"]}


# ------------------------------------------------------------------------------------------------ floors
def _mean_len(c):
    return (c["lo"] + c["hi"]) / 2 * (c["lanes"] - c["empty"])


def work(case):
    c = case
    if c["op"] == "cache":  # k and v in, codes and scales out, the values that they stand for out
        size = {"f32": 4, "bf16": 2}[c["io"]]
        return {"bytes": c["rows"] * 2 * c["kv"] * (c["hd"] * (2 * size + 1) + 4), "flops": c["rows"] * 2 * c["kv"] * c["hd"] * 4}
    if c["op"] == "attend":  # every key and value of every lane once
        size = {"f32": 4, "bf16": 2}[c["io"]]
        return {"bytes": _mean_len(c) * 2 * c["kv"] * (c["hd"] + 4) + c["lanes"] * 2 * c["heads"] * c["hd"] * size,
                "flops": _mean_len(c) * 4 * c["heads"] * c["hd"]}
    rows = c["seqs"] * ((c["lo"] + c["hi"]) / 2 + 1)  # every row of logits, and one row of the draft's probabilities a sequence
    return {"bytes": (rows + (c["seqs"] if c["probs"] else 0)) * c["vocab"] * 4, "flops": rows * c["vocab"] * 3}


# ------------------------------------------------------------------------------------------------ 64 bits
def _exact_cache(s):
    """The definition, in 64 bits: a value is the nearest multiple of its row's amax / 127 (this says nothing of pages)."""
    half = s["k"].shape[2] // 2
    angle = s["positions"].long()
    cos, sin = (t.double()[angle].unsqueeze(1) for t in s["rope"])
    k, v = s["k"].double(), s["v"].double()
    k = torch.stack([k[:, :, :half] * cos - k[:, :, half:] * sin, k[:, :, :half] * sin + k[:, :, half:] * cos], 2).flatten(2)
    unit = [x.abs().max(2, keepdim=True)[0] / 127 for x in (k, v)]
    return {"k": torch.round(k / unit[0]) * unit[0], "v": torch.round(v / unit[1]) * unit[1]}


def _exact_attend(s):
    """Lane by lane over its own tokens, as the sum of exp(q k) v over the sum of exp(q k)."""
    n, heads, hd = s["q"].shape
    kv, page = s["kc"].shape[1:3]
    out = torch.zeros(n, heads, hd, dtype=torch.float64, device="cuda")
    lens, lanes = s["lens"].tolist(), s["lanes"].tolist()
    for i in range(n):
        m = lens[i]
        if m == 0:
            continue
        own_pages = s["table"][lanes[i], :(m + page - 1) // page].long()
        k, v = [((c[own_pages].double() - 128) * f[own_pages].double()[..., None]).permute(1, 0, 2, 3).flatten(1, 2)[:, :m] for c, f in ((s["kc"], s["ks"]), (s["vc"], s["vs"]))]
        c, f = (t[m - 1].double() for t in s["rope"])
        q = s["q"][i].double()
        turned = torch.cat([q[:, :hd // 2] * c - q[:, hd // 2:] * f, q[:, :hd // 2] * f + q[:, hd // 2:] * c], 1)
        for g in range(kv):
            mine = slice(g * (heads // kv), (g + 1) * (heads // kv))
            out[i, mine] = torch.softmax(turned[mine] @ k[g].T / math.sqrt(hd), 1) @ v[g]
    return out


def _exact_verify(s):
    """Sequence by sequence, the rule as it is written down."""
    starts, draft, temps = s["start"].tolist(), s["draft"].tolist(), s["temps"].tolist()
    u = s["u_accept"].tolist()
    got, following = [], []
    for i, t in enumerate(temps):
        first, last = starts[i], starts[i + 1] - 1
        x = s["logits"][first:last + 1].double()
        p = torch.softmax(x / t, 1) if t else (torch.arange(x.shape[1], device="cuda") == x.max(1)[1][:, None]).double()
        r, token = first, None
        while r < last:
            d = draft[r]
            limit = 1.0 if s["probs"] is None or not t else float(s["probs"][r, d])
            here = float(p[r - first, d])
            if (here == 0.0) if not t else not (u[r] * limit < here):
                break
            r += 1
        w = p[r - first].clone()
        if r < last and t:
            if s["probs"] is None:
                w[draft[r]] = 0
            else:
                w = torch.relu(w - s["probs"][r].double())
            if float(w.sum()) <= 0:
                w = p[r - first]
        total = torch.cumsum(w, 0)
        token = int(torch.searchsorted(total, float(s["u_sample"][i]) * total[-1:])[0]) if t else int(w.argmax())
        got.append(r - first)
        following.append(token)
    return {"accepted": torch.tensor(got, dtype=torch.int32), "next": torch.tensor(following, dtype=torch.int32)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"cache": _exact_cache, "attend": _exact_attend, "verify": _exact_verify}[case["op"]](s)
