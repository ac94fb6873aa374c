"""The operators for what differs from request to request (pages, rotary positions,
adapters, filtered sampling) in 64 bits on the CPU, from their definitions in
include/fs.h: what the GPU tests compare with."""
from __future__ import annotations

import numpy as np

OK, KV_FULL, SCRATCH = 0, -6, -11


def pages_update(holders, table, lengths, grow, page, keep=None, max_rows=0):
    """New holders, table, lengths, and row_start, row_lane, row_position, row_length,
    row_slot, status, as a host's allocator would do it."""
    holders, table, lengths = holders.copy(), table.copy(), lengths.astype(np.int64)
    n, wide = table.shape
    cap = wide * page
    up = lambda t: -(-int(t) // page)
    lengths = np.clip(lengths, 0, cap)
    for i in range(n):
        left = lengths[i] if keep is None else min(lengths[i], max(0, int(keep[i])))
        for j in range(up(left), up(lengths[i])):
            p, table[i, j] = table[i, j], -1
            if 0 <= p < len(holders) and holders[p] > 0:
                holders[p] -= 1
        lengths[i] = left
    g = np.maximum(grow.astype(np.int64), 0)
    free = [p for p in range(len(holders)) if holders[p] == 0]
    want = [up(lengths[i] + g[i]) - up(lengths[i]) for i in range(n)]
    code = OK
    if sum(want) > len(free) or any(lengths + g > cap):
        code = KV_FULL
    elif g.sum() > max_rows:
        code = SCRATCH
    most = 2**31 - 1
    status = [code, min(int(g.sum()), most), min(sum(want), most), len(free)]
    start, rows = [0], []
    fresh = iter(free)
    for i in range(n):
        if code == OK:
            first = up(lengths[i])
            for j in range(first, first + want[i]):
                table[i, j] = next(fresh)
                holders[table[i, j]] = 1
            for t in range(lengths[i], lengths[i] + g[i]):
                rows.append((i, t, t + 1, int(table[i, t // page]) * page + t % page))
            lengths[i] += g[i]
        start.append(len(rows))
    rows += [(-1, -1, 0, -1)] * (max_rows - len(rows))
    lane, pos, length, slot = (np.array([r[c] for r in rows], np.int64) for c in range(4))
    return dict(holders=holders, table=table, lengths=lengths.astype(np.int32), row_start=np.array(start),
                row_lane=lane, row_position=pos, row_length=length, row_slot=slot, status=np.array(status))


def rotate(x, positions, inv_freq, factor=1.0, interleaved=False, inverse=False):
    """x [n, heads, hd] f64, turned; angles in long doubles."""
    out = x.astype(np.float64).copy()
    a = positions.astype(np.longdouble)[:, None] * inv_freq.astype(np.longdouble)
    a = (-a if inverse else a)
    z = (np.cos(a) + 1j * np.sin(a)).astype(np.complex128)[:, None] * factor
    half = len(inv_freq)
    if interleaved:
        v = (out[..., 0:2 * half:2] + 1j * out[..., 1:2 * half:2]) * z
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = v.real, v.imag
    else:
        v = (out[..., :half] + 1j * out[..., half:2 * half]) * z
        out[..., :half], out[..., half:2 * half] = v.real, v.imag
    return out


def lora(x, adapter, A, B, scale, base):
    """(out, sum of the terms' magnitudes, |B| |s A x|), f64."""
    x, A, B, s = (t.astype(np.float64) for t in (x, A, B, scale))
    out = base.astype(np.float64).copy()
    terms, low = np.zeros_like(out), np.zeros_like(out)
    for i, a in enumerate(adapter):
        if 0 <= a < len(A):
            t = A[a] @ x[i] * s[a]
            out[i] += B[a] @ t
            terms[i] = np.abs(B[a]) @ (np.abs(A[a]) @ np.abs(x[i])) * abs(s[a])
            low[i] = np.abs(B[a]) @ np.abs(t)
    return out, terms, low


def kept_ranks(z, T, top_k, top_p, min_p):
    """(indices that stay, in rank order; all tokens' weights) of one row in 64 bits."""
    z = np.where(np.isnan(z), -np.inf, z.astype(np.float64)) + 0.0
    order = np.argsort(-z, kind="stable")
    order = order[z[order] > -np.inf]
    if len(order) == 0:
        return order, np.zeros_like(z)
    m = z[order[0]]
    with np.errstate(invalid="ignore"):
        w = np.where(z == m, 1.0, np.exp((z - m) / T))
    w = np.nan_to_num(w, nan=0.0)
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        c = np.cumsum(w[order].astype(np.longdouble))
        ahead = np.concatenate([[0], c[:-1]])
        order = order[:max(1, int((ahead < np.longdouble(np.float32(top_p)) * c[-1]).sum()))]
    if min_p > 0:
        order = order[:max(1, int((w[order] >= np.float64(np.float32(min_p))).sum()))]
    return order, w


def sample(z, T, u, top_k=0, top_p=1.0, min_p=0.0):
    """(token, kept) of one row."""
    zz = np.where(np.isnan(z), -np.inf, z)
    if not (zz > -np.inf).any():
        return 0, 0
    if not T > 0:
        return int(np.argmax(zz)), 1
    order, w = kept_ranks(z, float(np.clip(np.float64(np.float32(T)), 1e-30, 1e30)), top_k, top_p, min_p)
    places = np.sort(order)
    c = np.cumsum(w[places].astype(np.longdouble))
    ok = (c >= np.longdouble(np.float32(min(u, 1.0))) * c[-1]) & (w[places] > 0)
    t = places[np.argmax(ok)] if ok.any() else places[w[places] > 0][-1]
    return int(t), len(order)
