"""Operators for what differs from request to request in a batched step: the cases that are measured, their inputs,
and their plain forms.

Four operators, told apart by a case's "op":
  pages   lanes keep part of their tokens and take new ones: pages are let go and taken on the GPU, and every new token
          gets its row (lane, position, length, slot of the cache)
  rope    rotary positions of queries and keys: pairs of halves or neighbours, the whole head or its first part, angles
          of far positions with frequencies scaled for long contexts
  lora    each row's own low-rank adapter, added to what a shared projection gave
  sample  one token a row from given random numbers, with the row's temperature, top-k, top-p and min-p
"""
import math

import torch

own = False


def listed():
    """Shapes: 9 / 3 heads of 64 with a width of 576 and a vocabulary of 49152, and 32 / 8 heads of 128 with widths of
    4096 and 14336 and a vocabulary of 32000 are the two models that the tests and the benchmark run; the others are generic."""
    return [
        # one lane's next token: the smallest call, where latency counts
        dict(name="pages-1-lane", op="pages", lanes=1, page=16, lo=200, hi=200, cut=0, grow_lo=1, grow=1, pad=0, others=0.0, room=1.5),
        # a step of 256 decoding lanes after a draft's rejected tokens have left, rows padded to the captured step's
        dict(name="pages-256-decode", op="pages", lanes=256, page=16, lo=1, hi=4096, cut=4, grow_lo=1, grow=5, pad=256, others=0.1, room=1.3),
        # prompts' chunks of many lanes, an odd page size
        dict(name="pages-1021-prompts", op="pages", lanes=1021, page=24, lo=0, hi=3001, cut=7, grow_lo=0, grow=257, pad=0, others=0.1, room=1.3),
        # one token of the small model: latency
        dict(name="rope-1-token", op="rope", n=1, heads=9, kv=3, hd=64, rot=64, near=False, far=2048, scaling="none", io="f32"),
        # a chunk of odd length out of the projection's panel, neighbours paired, a quarter of a wide head turned
        dict(name="rope-4099-part", op="rope", n=4099, heads=16, kv=2, hd=256, rot=64, near=True, far=32768, scaling="base", io="f32"),
        # whole prompts, far positions, frequencies scaled by a ramp over the dimensions
        dict(name="rope-65536-far", op="rope", n=65536, heads=32, kv=8, hd=128, rot=128, near=False, far=1048576, scaling="ramp", io="bf16"),
        # one token of the small model's projections: latency
        dict(name="lora-1-token", op="lora", n=1, adapters=4, rank=8, k=576, width=960, runs=False, without=0.0, x="bf16", y="f32"),
        # a decode step of 256 lanes with 64 adapters among them, a tenth of the lanes without one
        dict(name="lora-256-lanes", op="lora", n=256, adapters=64, rank=16, k=4096, width=4096, runs=False, without=0.1, x="bf16", y="f32"),
        # prompts of requests with eight adapters, into the widest projection
        dict(name="lora-8192-prompts", op="lora", n=8192, adapters=8, rank=64, k=4096, width=14336, runs=True, without=0.0, x="bf16", y="bf16"),
        # one row with the usual top-k and top-p: latency
        dict(name="sample-1-row", op="sample", n=1, vocab=32000, greedy=0.0, topk=1.0, klo=50, khi=50, topp=1.0, plo=0.9, minp=0.0),
        # 64 rows, each with its own mix: without filters, top-k, top-p, min-p, greedy
        dict(name="sample-64-mixed", op="sample", n=64, vocab=49152, greedy=0.15, topk=0.5, klo=1, khi=2000, topp=0.5, plo=0.5, minp=0.3),
        # full serving: 256 rows with top-p
        dict(name="sample-256-topp", op="sample", n=256, vocab=49152, greedy=0.0, topk=0.0, klo=1, khi=1, topp=1.0, plo=0.8, minp=0.1),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "rope", "lora", "sample"])
    if op == "pages":
        lanes = _spread(rng, 1, 1024)
        grow = rng.choice([1, 5, _spread(rng, 1, 100000 // lanes)])
        hi = _spread(rng, 1, min(131072, 3000000 // lanes))
        return dict(op=op, lanes=lanes, page=rng.choice([8, 16, 16, 24, 64, rng.randint(1, 128)]), lo=rng.randint(0, hi), hi=hi,
                    cut=rng.choice([0, 4, 100]), grow_lo=rng.randint(0, grow), grow=grow, pad=rng.choice([0, 0, 100]),
                    others=rng.choice([0.0, 0.1, 0.5]), room=rng.choice([1.3, 2.0, 0.9]))
    if op == "rope":
        hd, kv = rng.choice([64, 128, 128, 256, 80, 96]), rng.randint(1, 8)
        heads = kv * rng.randint(1, 8)
        io = rng.choice(["f32", "bf16"])
        most = 65536 * 40 * 128 // ((heads + kv) * hd) // (2 if io == "f32" else 1)
        return dict(op=op, n=_spread(rng, 1, min(65536, most)), heads=heads, kv=kv, hd=hd, rot=rng.choice([hd, hd, hd // 2, hd // 4 // 2 * 2, 2 * rng.randint(1, hd // 2)]),
                    near=rng.random() < 0.4, far=_spread(rng, 1, 1048576), scaling=rng.choice(["none", "linear", "base", "ramp", "bands"]), io=io)
    if op == "lora":
        adapters, rank = _spread(rng, 1, 256), rng.choice([8, 16, 16, 24, 32, 64, 128])
        k, width = 8 * _spread(rng, 8, 1792), _spread(rng, 1, 14336)
        most = 8192 * 8 * 64 * (4096 + 14336) // (adapters * rank * (k + width))
        return dict(op=op, n=_spread(rng, 1, max(1, min(8192, most))), adapters=adapters, rank=rank, k=k, width=width, runs=rng.random() < 0.5,
                    without=rng.choice([0.0, 0.1, 0.9]), x=rng.choice(["bf16", "bf16", "f32"]), y=rng.choice(["bf16", "f32"]))
    vocab = _spread(rng, 2, 131072)
    klo = _spread(rng, 1, vocab)
    return dict(op=op, n=_spread(rng, 1, min(256, max(1, 256 * 49152 // vocab))), vocab=vocab, greedy=rng.choice([0.0, 0.2]), topk=rng.choice([0.0, 0.5, 1.0]), klo=klo,
                khi=rng.randint(klo, vocab), topp=rng.choice([0.0, 0.5, 1.0]), plo=rng.uniform(0.05, 0.99), minp=rng.choice([0.0, 0.0, 0.5]))


# ------------------------------------------------------------------------------------------------ inputs
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _ints(lo, hi, size, gen):
    return torch.randint(lo, hi + 1, size, generator=gen, device="cuda", dtype=torch.int32)


def _evenly(lo, hi, n, gen):
    """n whole numbers spread evenly over lo .. hi, in any order: their sum, and so every size, does not depend on the seed."""
    at = (torch.arange(n, dtype=torch.float64) + 0.5) / n * (hi - lo)
    return (lo + at.round().to(torch.int32)).cuda()[torch.randperm(n, generator=gen, device="cuda")]


def _prepare_pages(c, gen):
    n, page = c["lanes"], c["page"]
    lengths, grow = _evenly(c["lo"], c["hi"], n, gen), _evenly(c["grow_lo"], c["grow"], n, gen)
    keep = (lengths - _ints(0, c["cut"], (n,), gen)).clamp(min=0)
    if c["cut"]:  # a few lanes are done
        keep = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.05, 0, keep).to(torch.int32)
    held = (lengths + page - 1) // page
    held_n = int(held.sum())
    most = (c["hi"] + c["grow"] + page - 1) // page
    total = int((held_n + int(grow.sum()) // page + n) * c["room"])
    n_pages = max(held_n, 1, int(total / (1.0 - c["others"])))
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    first = torch.cumsum(held, 0) - held
    col = torch.arange(most, device="cuda")
    table = torch.where(col < held[:, None], order[(first[:, None] + col).clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous()
    holders = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    holders[order[:held_n].long()] = 1
    others = order[held_n:held_n + int((n_pages - held_n) * c["others"])]  # pages of somebody else
    holders[others.long()] = 2
    rows = int(grow.sum()) + c["pad"]
    s = dict(op="pages", page=page, holders=holders, table=table, lengths=lengths, keep=keep, grow=grow)
    s["row_start"] = torch.empty(n + 1, dtype=torch.int32, device="cuda")
    for name in ("row_lane", "row_position", "row_length"):
        s[name] = torch.empty(rows, dtype=torch.int32, device="cuda")
    s["row_slot"] = torch.empty(rows, dtype=torch.int64, device="cuda")
    s["status"] = torch.empty(4, dtype=torch.int32, device="cuda")
    return s


def _scaling(c):
    """The scaling's numbers as a model's configuration holds them: contexts of 8192 stretched by 8."""
    return {"none": None, "linear": dict(kind="linear", factor=8.0), "base": dict(kind="base", factor=8.0),
            "ramp": dict(kind="ramp", factor=8.0, original=8192, beta_fast=32.0, beta_slow=1.0),
            "bands": dict(kind="bands", factor=8.0, original=8192, low=1.0, high=4.0)}[c["scaling"]]


def _frequencies(rot, theta, s):
    """Angle a position of each pair (64 bits), and the factor of the turned values."""
    j = torch.arange(rot // 2, dtype=torch.float64)
    f = theta ** (-2.0 * j / rot)
    if s is None:
        return f, 1.0
    if s["kind"] == "linear":
        return f / s["factor"], 1.0
    if s["kind"] == "base":
        return (theta * s["factor"] ** (rot / (rot - 2.0)) if rot > 2 else theta) ** (-2.0 * j / rot), 1.0
    turns = s["original"] * f / (2 * math.pi)  # of a pair over the original context
    if s["kind"] == "bands":
        part = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0.0, 1.0)
        return f / s["factor"] * (1 - part) + f * part, 1.0
    at = [rot * math.log(s["original"] / (2 * math.pi * b)) / (2 * math.log(theta)) for b in (s["beta_fast"], s["beta_slow"])]
    low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    ramp = ((j - low) / (high - low if high > low else 0.001)).clamp(0.0, 1.0)
    return f / s["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(s["factor"]) + 1.0


def _prepare_rope(c, gen):
    n, heads, kv, hd = c["n"], c["heads"], c["kv"], c["hd"]
    t = _TYPES[c["io"]]
    panel = torch.randn(n, (heads + 2 * kv) * hd, generator=gen, device="cuda").to(t)  # one row of the projection: q, k, v
    s = dict(op="rope", q=panel[:, :heads * hd].unflatten(1, (heads, hd)), k=panel[:, heads * hd:(heads + kv) * hd].unflatten(1, (kv, hd)),
             positions=_ints(0, c["far"] - 1, (n,), gen), near=c["near"], rot=c["rot"],
             q_out=torch.empty(n, heads, hd, dtype=t, device="cuda"), k_out=torch.empty(n, kv, hd, dtype=t, device="cuda"))
    if own:
        from continuous_transformer_decode_gb300 import fs
        s["freq"], s["factor"] = fs.fs_rope_frequencies(c["rot"], 10000.0, _scaling(c))
    else:
        f, s["factor"] = _frequencies(c["rot"], 10000.0, _scaling(c))
        s["freq"] = f.cuda()
    return s


def _prepare_lora(c, gen):
    n, a, r, k, width = c["n"], c["adapters"], c["rank"], c["k"], c["width"]
    if c["runs"]:  # rows of a request side by side, about eight requests an adapter
        edges = torch.rand(n, generator=gen, device="cuda") < min(1.0, 8.0 * a / n)
        run = torch.cumsum(edges, 0)
        which = _ints(0, a - 1, (n + 1,), gen)[run]
        gone = (torch.rand(n + 1, generator=gen, device="cuda") < c["without"])[run]
    else:
        which, gone = _ints(0, a - 1, (n,), gen), torch.rand(n, generator=gen, device="cuda") < c["without"]
    y = _TYPES[c["y"]]
    return dict(op="lora", x=torch.randn(n, k, generator=gen, device="cuda").to(_TYPES[c["x"]]), adapter=torch.where(gone, -1, which).to(torch.int32),
                a=(torch.randn(a, r, k, generator=gen, device="cuda") * k ** -0.5).to(torch.bfloat16),
                b=(torch.randn(a, width, r, generator=gen, device="cuda") * r ** -0.5).to(torch.bfloat16),
                scale=0.25 + torch.rand(a, generator=gen, device="cuda"), base=torch.randn(n, width, generator=gen, device="cuda").to(y),
                out=torch.empty(n, width, dtype=y, device="cuda"))


def _prepare_sample(c, gen):
    n, vocab = c["n"], c["vocab"]
    rand = lambda: torch.rand(n, generator=gen, device="cuda")
    temps = torch.where(rand() < c["greedy"], 0.0, 0.6 + 0.6 * rand())
    k = torch.where(rand() < c["topk"], _ints(c["klo"], c["khi"], (n,), gen), 0).to(torch.int32)
    p = torch.where(rand() < c["topp"], c["plo"] + (1.0 - c["plo"]) * rand() * 0.99, 1.0)
    m = torch.where(rand() < c["minp"], 0.01 + 0.2 * rand(), 0.0)
    return dict(op="sample", logits=torch.randn(n, vocab, generator=gen, device="cuda") * 2.5, temps=temps, top_k=k, top_p=p, min_p=m, u=rand(),
                tokens=torch.empty(n, dtype=torch.int32, device="cuda"), kept=torch.empty(n, dtype=torch.int32, device="cuda"))


_PREPARE = {"pages": _prepare_pages, "rope": _prepare_rope, "lora": _prepare_lora, "sample": _prepare_sample}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    s = _PREPARE[case["op"]](case, gen)
    if own:
        from continuous_transformer_decode_gb300 import fs
        s["fs"] = fs
    return s


# ------------------------------------------------------------------------------------------------ plain forms
_STATE = ("holders", "table", "lengths", "row_start", "row_lane", "row_position", "row_length", "row_slot", "status")


def _pages_plain(s):
    page, table, holders = s["page"], s["table"], s["holders"]
    n, wide = table.shape
    n_pages, rows = holders.numel(), s["row_lane"].numel()
    col = torch.arange(wide, device="cuda")
    up = lambda x: (x + page - 1) // page
    # what lanes do not keep goes
    had = s["lengths"].long().clamp(0, wide * page)
    held = torch.minimum(had, s["keep"].long().clamp(min=0))
    after = up(held)
    gone = (col >= after[:, None]) & (col < up(had)[:, None])
    where = torch.where(gone & (table >= 0) & (table < n_pages), table.long(), n_pages)
    less = torch.zeros(n_pages + 1, dtype=torch.int32, device="cuda").scatter_add_(0, where.flatten(), torch.ones_like(where, dtype=torch.int32).flatten())
    holders.copy_((holders - less[:n_pages]).clamp(min=0))
    # the lowest free pages, lanes in order
    grow = s["grow"].long().clamp(min=0)
    want = up(held + grow) - after
    first = torch.cumsum(want, 0) - want
    free = holders == 0
    place = torch.cumsum(free, 0) - 1
    found = torch.zeros(n_pages + 1, dtype=torch.int32, device="cuda").scatter_(0, torch.where(free, place, n_pages), torch.arange(n_pages, dtype=torch.int32, device="cuda"))
    n_free, n_want, n_rows = free.sum(), want.sum(), grow.sum()
    fits = (n_want <= n_free) & ((held + grow) <= wide * page).all()
    ok = fits & (n_rows <= rows)
    code = torch.where(fits, torch.where(n_rows <= rows, 0, -11), -6)
    new = (col >= after[:, None]) & (col < (after + want)[:, None]) & ok
    page_of = found[(first[:, None] + col - after[:, None]).clamp(0, n_pages)]
    table.copy_(torch.where(new, page_of, torch.where(gone, -1, table)))
    holders.copy_(torch.where(free & (place < n_want) & ok, 1, holders))
    s["lengths"].copy_(torch.where(ok, held + grow, held))
    end = torch.cumsum(torch.where(ok, grow, 0), 0)
    s["row_start"][0] = 0
    s["row_start"][1:] = end
    r = torch.arange(rows, device="cuda")
    inside = r < end[-1]
    lane = torch.searchsorted(end, r, right=True).clamp(max=n - 1)
    pos = (held[lane] + r - (end - torch.where(ok, grow, 0))[lane]).clamp(0, wide * page - 1)
    s["row_lane"].copy_(torch.where(inside, lane, -1))
    s["row_position"].copy_(torch.where(inside, pos, -1))
    s["row_length"].copy_(torch.where(inside, pos + 1, 0))
    s["row_slot"].copy_(torch.where(inside, table[lane, pos // page].long() * page + pos % page, -1))
    s["status"].copy_(torch.stack([code, n_rows, n_want, n_free]))
    return {k: s[k] for k in _STATE}


def _rope_plain(s):
    angle = s["positions"].double()[:, None] * s["freq"]  # 64 bits: far positions
    c, n = ((x() * s["factor"]).float()[:, None] for x in (angle.cos, angle.sin))
    rot = s["rot"]
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        v = x[..., :rot].float()
        a, b = (v[..., 0::2], v[..., 1::2]) if s["near"] else (v[..., :rot // 2], v[..., rot // 2:])
        turned = (a * c - b * n, b * c + a * n)
        out[..., :rot] = torch.stack(turned, -1).flatten(-2) if s["near"] else torch.cat(turned, -1)
        out[..., rot:] = x[..., rot:]
    return {"q": s["q_out"], "k": s["k_out"]}


def _lora_plain(s):
    """Every row against all adapters, the others' parts then taken as 0: no row is looked for."""
    adapters, r, k = s["a"].shape
    low = torch.matmul(s["x"].float(), s["a"].float().view(adapters * r, k).T).view(-1, adapters, r)
    mine = s["adapter"][:, None] == torch.arange(adapters, device="cuda")
    low = torch.where(mine[..., None], low * s["scale"][:, None], 0.0)
    delta = torch.matmul(low.flatten(1), s["b"].float().transpose(1, 2).reshape(adapters * r, -1))
    s["out"].copy_(s["base"].float() + delta)
    return s["out"]


def _sample_plain(s):
    """In 64 bits: running sums lie next to a border now and then."""
    z = s["logits"]
    n, vocab = z.shape
    index = torch.arange(vocab, device="cuda")
    temps = s["temps"].double()[:, None]
    top = z.amax(-1, keepdim=True)
    best = torch.where(z == top, index, vocab).amin(-1)
    ranked, order = torch.sort(z, dim=-1, descending=True, stable=True)  # equal ones by their index
    w = ((ranked - top).double() / torch.where(temps > 0, temps, 1.0)).exp()
    k = s["top_k"].long()[:, None]
    inside = (index < k) | (k <= 0)
    w_in = torch.where(inside, w, 0.0)
    upto = w_in.cumsum(-1)
    p = s["top_p"].double()[:, None]
    inside &= (p >= 1.0) | (upto - w_in < p * upto[:, -1:]) | (index == 0)
    inside &= (w >= s["min_p"].double()[:, None]) | (index == 0)
    kept = inside.sum(-1)
    left = torch.zeros_like(w).scatter_(-1, order, torch.where(inside, w, 0.0))  # in the order of the vocabulary
    run_sum = left.cumsum(-1)
    target = s["u"].double()[:, None] * run_sum[:, -1:]
    token = torch.where((run_sum >= target) & (left > 0), index, vocab).amin(-1)
    last = torch.where(left > 0, index, -1).amax(-1)
    greedy = s["temps"] <= 0
    s["tokens"].copy_(torch.where(greedy, best, torch.where(token < vocab, token, last)))
    s["kept"].copy_(torch.where(greedy, 1, kept))
    return {"tokens": s["tokens"], "kept": s["kept"]}


_PLAIN = {"pages": _pages_plain, "rope": _rope_plain, "lora": _lora_plain, "sample": _sample_plain}


def run(state):
    s = state
    if not own:
        return _PLAIN[s["op"]](s)
    fs = s["fs"]
    if s["op"] == "pages":
        fs.fs_pages_update(s["holders"], s["table"], s["lengths"], s["grow"], s["page"], s["status"], keep=s["keep"], row_start=s["row_start"], row_lane=s["row_lane"],
                           row_position=s["row_position"], row_length=s["row_length"], row_slot=s["row_slot"])
        return {k: s[k] for k in _STATE}
    if s["op"] == "rope":
        fs.fs_rope(s["q"], s["positions"], s["freq"], k=s["k"], q_out=s["q_out"], k_out=s["k_out"], interleaved=s["near"], factor=s["factor"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if s["op"] == "lora":
        fs.fs_lora_add(s["x"], s["adapter"], s["a"], s["b"], s["scale"], s["out"], base=s["base"])
        return s["out"]
    fs.fs_sample_filtered(s["logits"], s["temps"], s["u"], s["tokens"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], kept=s["kept"])
    return {"tokens": s["tokens"], "kept": s["kept"]}


# ------------------------------------------------------------------------------------------------ floors
def work(case):
    c = case
    if c["op"] == "pages":  # the holders, the lanes' numbers, the table's new entries, the rows
        rows, pages = c["lanes"] * (c["grow_lo"] + c["grow"]) / 2, c["lanes"] * (c["lo"] + c["hi"]) / 2 / c["page"]
        return {"bytes": pages * c["room"] / (1 - c["others"]) * 4 + c["lanes"] * 20 + rows / c["page"] * 8 + (rows + c["pad"]) * 20, "flops": 0}
    if c["op"] == "rope":  # q and k in and out
        size = {"f32": 4, "bf16": 2}[c["io"]]
        values = c["n"] * (c["heads"] + c["kv"])
        return {"bytes": values * c["hd"] * 2 * size + c["n"] * 4, "flops": values * c["rot"] * 3}
    if c["op"] == "lora":  # x, base, out, and the adapters that occur
        sx, sy = ({"f32": 4, "bf16": 2}[c[t]] for t in ("x", "y"))
        rows = c["n"] * (1 - c["without"])
        met = c["adapters"] * (1 - (1 - 1 / c["adapters"]) ** rows)
        return {"bytes": rows * c["k"] * sx + 2 * c["n"] * c["width"] * sy + met * c["rank"] * (c["k"] + c["width"]) * 2, "flops": 2 * rows * c["rank"] * (c["k"] + c["width"])}
    return {"bytes": c["n"] * c["vocab"] * 4, "flops": c["n"] * c["vocab"] * 3}


# ------------------------------------------------------------------------------------------------ 64 bits
def _exact_pages(s):
    """Lane by lane, as a host's allocator does it."""
    page = s["page"]
    holders, table, lengths, keep, grow = (s[k].tolist() for k in ("holders", "table", "lengths", "keep", "grow"))
    wide, rows = s["table"].shape[1], s["row_lane"].numel()
    for i, pages in enumerate(table):
        left = min(lengths[i], keep[i])
        for j in range(-(-left // page), -(-lengths[i] // page)):
            holders[pages[j]] -= 1
            pages[j] = -1
        lengths[i] = left
    free = [p for p, h in enumerate(holders) if h == 0]
    want = [-(-(a + g) // page) - -(-a // page) for a, g in zip(lengths, grow)]
    full = sum(want) > len(free) or any(a + g > wide * page for a, g in zip(lengths, grow))
    code = -6 if full else -11 if sum(grow) > rows else 0
    out = {"holders": holders, "status": [code, sum(grow), sum(want), len(free)], "row_start": [0]}
    lane, position, length, slot = [], [], [], []
    fresh = iter(free)
    for i, pages in enumerate(table):
        if code == 0:
            at = -(-lengths[i] // page)
            for j in range(at, at + want[i]):
                pages[j] = next(fresh)
                holders[pages[j]] = 1
            for t in range(lengths[i], lengths[i] + grow[i]):
                lane.append(i)
                position.append(t)
                length.append(t + 1)
                slot.append(pages[t // page] * page + t % page)
            lengths[i] += grow[i]
        out["row_start"].append(len(lane))
    rest = rows - len(lane)
    out.update(table=table, lengths=lengths, row_lane=lane + [-1] * rest, row_position=position + [-1] * rest, row_length=length + [0] * rest, row_slot=slot + [-1] * rest)
    return {k: torch.tensor(out[k], dtype=torch.int64 if k == "row_slot" else torch.int32) for k in _STATE}


def _exact_rope(s, case):
    """As products of complex numbers, a head at a time."""
    f, factor = _frequencies(case["rot"], 10000.0, _scaling(case))
    angle = s["positions"].double().unsqueeze(1) * f.cuda()
    turn = torch.polar(torch.full_like(angle, factor), angle)
    out = {}
    half = case["rot"] // 2
    for name in ("q", "k"):
        y = s[name].double()
        for h in range(y.shape[1]):
            v = y[:, h, :2 * half].clone()
            z = torch.view_as_complex(v.view(-1, half, 2)) if case["near"] else torch.complex(v[:, :half].contiguous(), v[:, half:].contiguous())
            z = z * turn
            y[:, h, :2 * half] = torch.view_as_real(z).flatten(1) if case["near"] else torch.cat([z.real, z.imag], 1)
        out[name] = y
    return out


def _exact_lora(s):
    """Adapter by adapter over the rows that have it."""
    out = s["base"].double()
    for a in range(s["a"].shape[0]):
        rows = (s["adapter"] == a).nonzero()[:, 0]
        if rows.numel():
            product = s["x"][rows].double() @ s["a"][a].double().T @ s["b"][a].double().T
            out[rows] += float(s["scale"][a]) * product
    return out


def _exact_sample(s):
    """Row by row, the rule as it is written down."""
    tokens, kept = [], []
    for z, t, k, p, m, u in zip(s["logits"], *(s[x].tolist() for x in ("temps", "top_k", "top_p", "min_p", "u"))):
        if t <= 0:
            tokens.append(int(torch.nonzero(z == z.max())[0]))
            kept.append(1)
            continue
        w = torch.exp((z.double() - z.max().double()) / t)
        order = torch.argsort(z, descending=True, stable=True)
        if k > 0:
            order = order[:k]
        if p < 1:
            mass = torch.cumsum(w[order], 0)
            ahead = torch.cat([mass.new_zeros(1), mass[:-1]])
            order = order[:max(1, int((ahead < p * mass[-1]).sum()))]
        order = order[:max(1, int((w[order] >= m).sum()))]
        places = torch.sort(order)[0]
        total = torch.cumsum(w[places], 0)
        tokens.append(int(places[min(int(torch.searchsorted(total, u * total[-1:])[0]), len(places) - 1)]))
        kept.append(len(order))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32), "kept": torch.tensor(kept, dtype=torch.int32)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s, case)
    return {"pages": _exact_pages, "lora": _exact_lora, "sample": _exact_sample}[case["op"]](s)
