"""Plain references of the operators that serve prompts and shared pages (numpy, 64 bits, loops)."""
from __future__ import annotations

import math

import numpy as np
import torch

from lm_reference import ceil_div


# -------------------------------------------------------------- attention
def gather(K, V, ks, vs, row, t, page, h, D):
    """Keys and values [len(t), D] in 64 bits of tokens t of a request whose row of the table this is."""
    p = np.asarray(row)[t // page]
    p = np.where((p >= 0) & (p < K.shape[0]), p, 0)              # (an index outside the pool reads page 0)
    k = K[p, h, t % page, :D].double().numpy()
    v = V[p, h, t % page // 8, :D, t % page % 8].double().numpy()
    if ks is not None:
        k = k * ks[p, h, t % page].double().numpy()[:, None]
        v = v * vs[p, h, t % page].double().numpy()[:, None]
    return k, v


def row_attention(q, k, v, scale, terms):
    """out [D], log-sum, and bounds of their errors, of one query row over keys k and values v [n, D].

    A score is a sum of D products in fp32 and its scaling: off by (D + 16) 2^-24 sum |q k|.  The weights then err by
    that much relatively, in the numerator and in the sum; sums over n tokens add n 2^-24.  A weight held in `terms` bf16
    terms is off by 2^-8 of what the terms before it leave: 2^-(8 terms)."""
    n, D = k.shape
    x = k @ q * scale
    m = x.max()
    w = np.exp(x - m)
    z = w.sum()
    most = (np.abs(k) @ np.abs(q)).max() * abs(scale)
    eps = 2.0 ** -24 * (2 * (D + 16) * most + 64 + n)
    lse = m + math.log(z)
    return w @ v / z, lse, (eps + 2.0 ** (-8 * terms)) * (w @ np.abs(v)) / z, eps + 2.0 ** -22 * abs(lse)


def visible(x, window, sinks):
    """Tokens that the row at position x sees."""
    t = np.arange(x + 1)
    return t[(t > x - window) | (t < sinks)] if window else t


def prompt(q, sections, table, start, lens, page, scale, window, sinks, max_len, terms):
    """fp64 results of every row that belongs to a request; rows outside keep NaN (left as they were).  q [T, A, D]."""
    K, V, ks, vs = sections
    T, A, D = q.shape
    H = K.shape[1]
    out, tol = np.full((T, A, D), np.nan), np.zeros((T, A, D))
    lse, ltol = np.full((T, A), np.nan), np.zeros((T, A))
    for r in range(len(lens)):
        s0, s1 = (min(max(int(start[i]), 0), T) for i in (r, r + 1))
        n = s1 - s0
        length = min(max(int(lens[r]), 0), max_len)
        for i in range(max(n, 0)):
            x = length - n + i
            t = visible(x, window, sinks) if x >= 0 else np.arange(0)
            for h in range(H):
                if len(t):
                    k, v = gather(K, V, ks, vs, table[r], t, page, h, D)
                for a in range(h * (A // H), (h + 1) * (A // H)):
                    if len(t):
                        out[s0 + i, a], lse[s0 + i, a], tol[s0 + i, a], ltol[s0 + i, a] = row_attention(q[s0 + i, a], k, v, scale, terms)
                    else:
                        out[s0 + i, a], lse[s0 + i, a] = 0, -np.inf
    return out, lse, tol, ltol


def groups_of(start, R):
    """The group of each request (-1: none)."""
    of = np.full(R, -1)
    for g in range(len(start) - 1):
        of[max(0, start[g]):max(0, min(R, start[g + 1]))] = g
    return of


def shared(q, sections, table, lens, start, prefix, page, scale, max_len, max_prefix, terms):
    """fp64 results of one token per request; a prefix is read from the pages of its group's first request."""
    K, V, ks, vs = sections
    R, A, D = q.shape
    H = K.shape[1]
    out, tol = np.zeros((R, A, D)), np.zeros((R, A, D))
    lse, ltol = np.full((R, A), -np.inf), np.zeros((R, A))
    of = groups_of(start, R)
    clip = lambda n: min(max(int(n), 0), max_len)  # noqa: E731
    for r in range(R):
        n, g = clip(lens[r]), of[r]
        first = max(0, start[g]) if g >= 0 else r
        pre = min(min(max(int(prefix[g]), 0), max_prefix), clip(lens[first])) if g >= 0 else 0
        if n == 0:
            continue
        for h in range(H):
            parts = [gather(K, V, ks, vs, table[first], np.arange(min(pre, n)), page, h, D),
                     gather(K, V, ks, vs, table[r], np.arange(min(pre, n), n), page, h, D)]
            k, v = (np.concatenate(x) for x in zip(*parts))
            for a in range(h * (A // H), (h + 1) * (A // H)):
                out[r, a], lse[r, a], tol[r, a], ltol[r, a] = row_attention(q[r, a], k, v, scale, terms)
    return out, lse, tol, ltol


# ------------------------------------------------------------------ pages
def fork(src, keep, lens, ring, head, count, table, page, pool):
    """Request by request.  ring is changed in place; returns the tables (entries past a request's pages: None), lengths,
    the copies, and the state."""
    R, S = table.shape
    first_ring = ring.copy()
    most = S * page
    lens = [min(max(int(n), 0), most) for n in lens]
    want, refused = [], 0
    for r in range(R):
        s, k = int(src[r]), int(keep[r])
        if not 0 <= s < R or not 0 <= k <= lens[s]:
            s, k = r, lens[r]
            refused += 1
        want.append((s, k))
    ok = lambda p: 0 <= p < pool  # noqa: E731
    before = {int(table[r, j]) for r in range(R) for j in range(ceil_div(lens[r], page))}
    whole = {int(table[s, j]) for s, k in want for j in range(k // page)}
    ends = {}                                        # page -> the requests that end inside it
    for r, (s, k) in enumerate(want):
        if k % page:
            ends.setdefault(int(table[s, k // page]), []).append((s != r, r))
    out, now, copies = [], [], []
    for r, (s, k) in enumerate(want):
        rows = [int(table[s, j]) for j in range(ceil_div(k, page))]
        last = rows[-1] if k % page else -1
        if k % page and ok(last) and (last in whole or min(ends[last])[1] != r):
            if len(copies) < count:
                rows[-1] = int(first_ring[(head + len(copies)) % pool])
                copies.append((last, rows[-1]))
            else:
                rows.pop()
                k -= k % page
                refused += 1
        out.append(rows + [None] * (S - len(rows)))
        now.append(k)
    freed = sorted(p for p in before if ok(p) and p not in whole and p not in ends)
    for i, p in enumerate(freed[:pool - count]):
        ring[(head + count + i) % pool] = p
    return out, now, copies, [(head + len(copies)) % pool, count - len(copies) + len(freed[:pool - count]), len(copies), refused]


def compact(lens, table, page, pool, places):
    """The tables, copies, free pages in order, and the state."""
    R, S = table.shape
    held = [ceil_div(min(max(int(n), 0), S * page), page) for n in lens]
    used = {int(table[r, j]) for r in range(R) for j in range(held[r])} & set(range(pool))
    free = sorted(set(range(pool)) - used)
    moves = []
    for f, t in zip(sorted(used, reverse=True), free):
        if f > t and len(moves) < places:
            moves.append((f, t))
    to = dict(moves)
    out = [[to.get(int(table[r, j]), int(table[r, j])) if j < held[r] else None for j in range(S)] for r in range(R)]
    after = {to.get(p, p) for p in used}
    free = sorted(set(range(pool)) - after)
    return out, moves, free, [0, len(free), len(moves), max(after) + 1 if after else 0]


# --------------------------------------------------------------- rotation
def frequencies(rot, base, kind="plain", factor=1.0, trained=0.0, keep=0.0, scale=0.0):
    f = []
    for i in range(rot // 2):
        w = base ** (-2 * i / rot)
        if kind == "linear":
            w /= factor
        elif kind == "ramp":
            d = lambda turns: rot * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(d(keep)), 0), min(math.ceil(d(scale)), rot - 1)
            t = min(max((i - lo) / max(hi - lo, 0.001), 0), 1)
            w = w * (1 - t) + w / factor * t
        elif kind == "band":
            t = min(max((trained * w / (2 * math.pi) - scale) / (keep - scale), 0), 1)
            w = w * t + w / factor * (1 - t)
        f.append(w)
    return np.array(f)


def rope(x, w, pos, table, rot, pairs, eps, mscale):
    """fp64 norms and rotation of x [T, H, D], angles from the table's 64-bit fractions; and the size of the terms of each
    output (its error is a small multiple of 2^-24 of that)."""
    T, H, D = x.shape
    y = x.astype(np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
    out, mag = y.copy(), np.abs(y)
    if rot:
        turns = np.array([[int(p) * int(f) % 2 ** 64 / 2.0 ** 64 for f in table[:rot // 2]] for p in pos])
        c, s = (mscale * g(2 * np.pi * turns)[:, None] for g in (np.cos, np.sin))
        i = np.arange(rot // 2)
        iu, iv = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
        u, v = y[..., iu], y[..., iv]
        out[..., iu], out[..., iv] = u * c - v * s, v * c + u * s
        mag[..., iu] = mag[..., iv] = (np.abs(u) + np.abs(v)) * abs(mscale)
    return out, mag


def half_step(dtype):
    """Most that rounding to the type moves a value, relative to it."""
    return torch.finfo(dtype).eps / 2
