"""The 8-bit paged cache, the attention over it and draft verification in 64
bits on the CPU, from their definitions in include/fs.h: what the GPU tests
compare with."""
from __future__ import annotations

import numpy as np


def bf16(x):
    """Nearest bf16 values (as f32)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    u = (u + np.uint32(0x7FFF) + ((u >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xFFFF0000)
    return u.view(np.float32)


def rope_tables(n, hd, theta=1e4):
    inv = theta ** (-2.0 * np.arange(hd // 2) / hd)
    a = np.arange(n)[:, None] * inv
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def rotate(x, cos, sin):
    """x [rows, heads, hd], cos / sin [rows, hd / 2]; 64 bits."""
    x, c, s = x.astype(np.float64), cos.astype(np.float64)[:, None], sin.astype(np.float64)[:, None]
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def quantise(x):
    """Codes (signed) and 64-bit scales of the rows of x."""
    big = float(np.finfo(np.float32).max)
    x = np.clip(np.nan_to_num(x.astype(np.float64), nan=0.0, posinf=big, neginf=-big), -big, big)
    amax = np.abs(x).max(-1)
    q = np.rint(x * 127.0 / np.where(amax > 0, amax, 1.0)[..., None])
    return np.where(amax[..., None] > 0, q, 0).astype(np.int64), amax / 127.0


class Cache:
    """Values that the cache stands for, f64, by (lane, token); absent tokens are not in the dict."""

    def __init__(self, codes_k, codes_v, ks, vs, table):
        self.k = (codes_k.astype(np.float64) - 128) * ks.astype(np.float64)[..., None]
        self.v = (codes_v.astype(np.float64) - 128) * vs.astype(np.float64)[..., None]
        self.table = table
        self.n_pages, self.Hkv, self.ps, self.hd = codes_k.shape

    def rows(self, lane, n):
        """(tokens present, K [m, Hkv, hd], V) of the first n tokens of a lane."""
        if not 0 <= lane < self.table.shape[0]:
            return np.zeros(0, int), np.zeros((0, self.Hkv, self.hd)), np.zeros((0, self.Hkv, self.hd))
        n = max(0, min(n, self.table.shape[1] * self.ps))
        t = np.arange(n)
        page = self.table[lane][t // self.ps]
        ok = (page >= 0) & (page < self.n_pages)
        t, page = t[ok], page[ok]
        return t, self.k[page, :, t % self.ps], self.v[page, :, t % self.ps]


def attention(cache, q, lanes, lengths, scale, rope=None):
    """Outputs f64 [n, H, hd] and, per output, a bound of the error of f32
    arithmetic.

    The bound, with A = sum p |v| of the output: a score is off by at most
    dz = 2^-20 scale max_t sum |q_d k_d| (the rotation 4 roundings, the two-part
    f16 query 2^-22, the f32 dot product and its two scalings, a dozen roundings
    along a path of the tensor core's sum), which turns a weight by 2 dz; the
    exponential of token t is good to a relative 2^-22 (1 + |z_t - max|), as its
    argument is rounded, so it moves the output by at most
    2^-22 sum p |v| (1 + |z - max|). (The values' scales may differ by any factor,
    so a token with a small p and a large |z - max| can carry the output: the
    distance stays inside the sum.) The join and the division add a few 2^-24,
    and the f32 sums over n tokens at most n 2^-24 of A. Together
    A (2 dz + 2^-18 + n 2^-24) + 2^-22 sum p |v| |z - max|; the sum of the weights,
    which divides, is off by the same expression with |v| = 1, its distances
    included: A sum p |z - max| 2^-22. Small weights have an absolute error too: in
    f32 those below 2^-126 of the largest are lost (2^-126 sum |v|), and as two f16
    parts of p_t scale_t, scaled so that the largest is 2^14, each is off by at
    most half of f16's smallest step, 2^-25, that is 2^-39 max p amax of it for codes
    up to 127: n 2^-39 max_t(p_t amax_t). (It shows where the token that carries
    all the weight has a zero in this place.)"""
    n, H, hd = q.shape
    out = np.zeros((n, H, hd))
    tol = np.zeros((n, H, hd))
    G = H // cache.Hkv
    for i in range(n):
        _, K, V = cache.rows(int(lanes[i]), int(lengths[i]))
        if len(K) == 0:
            continue
        x = q[i:i + 1].astype(np.float64)
        if rope is not None:
            at = [int(lengths[i]) - 1]
            x = rotate(x, rope[0][at], rope[1][at])
        for h in range(H):
            k, v = K[:, h // G], V[:, h // G]
            z = scale * (k @ x[0, h])
            dz = 2.0 ** -20 * abs(scale) * (np.abs(k) @ np.abs(x[0, h])).max()
            far = z.max() - z
            p = np.exp(-far)
            p /= p.sum()
            out[i, h] = p @ v
            A = p @ np.abs(v)
            tol[i, h] = (A * (2 * dz + 2.0 ** -18 + len(K) * 2.0 ** -24 + 2.0 ** -22 * (p @ far))
                         + 2.0 ** -22 * ((p * far) @ np.abs(v)) + 2.0 ** -126 * np.abs(v).sum(0)
                         + len(K) * 2.0 ** -39 * (p * np.abs(v).max(-1)).max())
    return out, tol


def verify(logits, row_start, draft, probs, temps, u_accept, u_sample):
    """(n_accepted, next_token) by the rule, in 64 bits."""
    acc, nxt = [], []
    n_rows = logits.shape[0]
    for s in range(len(temps)):
        r0 = min(max(int(row_start[s]), 0), n_rows)
        r1 = max(r0, min(int(row_start[s + 1]), n_rows))
        if r0 == r1:
            acc.append(0)
            nxt.append(-1)
            continue
        for r in range(r0, r1):
            z = logits[r].astype(np.float64)
            z = np.where(np.isnan(z), -np.inf, z)
            x, last, m = int(draft[r]), r == r1 - 1, z.max()
            known = 0 <= x < len(z)
            if m == -np.inf:
                token = 0
                break
            if not temps[s] > 0:
                token = int(np.argmax(z))
                if not last and x == token:
                    continue
                break
            with np.errstate(invalid="ignore"):
                e = np.where(z == m, 1.0, np.exp((z - m) / float(temps[s])))
            p = e / e.sum()
            q = probs[r].astype(np.float64) if probs is not None else None
            if not last and known and float(u_accept[r]) * (q[x] if q is not None else 1.0) < p[x]:
                continue
            w = p.copy()
            if not last:
                if q is not None:
                    w = np.maximum(p - q, 0.0)
                elif known:
                    w[x] = 0.0
            if not w.sum() > 0:
                w = p
            c = np.cumsum(w)
            ok = np.nonzero((c >= float(u_sample[s]) * c[-1]) & (w > 0))[0]
            token = int(ok[0]) if len(ok) else int(np.nonzero(w > 0)[0][-1])
            break
        acc.append(r - r0)
        nxt.append(token)
    return np.array(acc, np.int32), np.array(nxt, np.int32)
