"""Plain references of the operators of include/bitq_lm.h (numpy and torch on the CPU, 64 bits, loops),
and input builders shared by their tests."""
from __future__ import annotations

import math

import numpy as np
import torch


def ceil_div(a, b):
    return -(-a // b)


# ------------------------------------------------------------------- plan
def plan(old, new, page, table, ring, head, count, tokens):
    """One scheduling step, request by request.  table, ring: int32 arrays, changed in place."""
    R, stride = table.shape
    cap = len(ring)
    most = stride * page
    first_ring, first_table = ring.copy(), table.copy()
    length, start, slot, req, pos = list(old), [0], [], [], []
    taken = given_tokens = back = refused = 0
    closed = False
    for r in range(R):
        o, n = int(old[r]), int(new[r])
        start.append(given_tokens)
        if o < 0 or n < 0 or o > most or n > most:
            refused += 1
            continue
        held, need = ceil_div(o, page), ceil_div(n, page)
        if n > o:
            if closed or taken + need - held > count or given_tokens + n - o > tokens:
                closed = True
                refused += 1
                continue
            for j in range(held, need):
                table[r, j] = first_ring[(head + taken) % cap]
                taken += 1
            for p in range(o, n):
                slot.append(int(table[r, p // page]) * page + p % page)
                req.append(r)
                pos.append(p)
            given_tokens += n - o
            start[-1] = given_tokens
        else:
            for j in range(need, held):
                if back < cap - count:
                    ring[(head + count + back) % cap] = first_table[r, j]
                    back += 1
        length[r] = n
    pad = [-1] * (tokens - len(slot))
    i32 = lambda v: np.array(v, dtype=np.int64).astype(np.int32)  # noqa: E731
    return dict(len=i32(length), start=i32(start), slot=i32(slot + pad), req=i32(req + pad), pos=i32(pos + pad),
                state=i32([(head + taken) % cap, count - taken + back, given_tokens, refused]))


# ------------------------------------------------------------------ cache
def codes(x):
    """int8 codes and fp32 scales of rows (last dimension), in the quantizer's fp32 arithmetic."""
    x = np.asarray(x, dtype=np.float32)
    amax = np.abs(x).max(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        s = np.where(amax > 0, np.float32(127) / amax, np.float32(0)).astype(np.float32)
    q = np.clip(np.rint(x * s), -127, 127).astype(np.int8)
    return q, (amax / np.float32(127)).astype(np.float32)[..., 0]


def write(K, V, ks, vs, k, v, slots, page):
    """New rows into the sections of a cache (torch CPU tensors, in place).  k, v: fp32 [T, H, D]."""
    D = k.shape[2]
    nslots = K.shape[0] * page
    for t, s in enumerate(slots.tolist()):
        if not 0 <= s < nslots:
            continue
        p, off = divmod(s, page)
        for rows, vals, scale in ((K, k, ks), (V, v, vs)):
            if scale is None:
                w = vals[t].to(torch.bfloat16)
            else:
                q, d = codes(vals[t].numpy())
                w = torch.from_numpy(q)
                scale[p, :, off] = torch.from_numpy(d)
            if rows is K:
                K[p, :, off, :] = 0
                K[p, :, off, :D] = w
            else:
                V[p, :, off // 8, :, off % 8] = 0
                V[p, :, off // 8, :D, off % 8] = w


# -------------------------------------------------------------- attention
def attention(q, K, V, ks, vs, table, lens, page, scale, window, max_len):
    """fp64 attention, and a bound on the fp32 error of each output and of the log-sum.

    K, V (and ks, vs): sections of a cache on the CPU.  A score is a sum of D products in fp32 (error at most
    (D + 8) 2^-24 sum |q k|, with the scaling); the weights then err by that much relatively, each way; sums over
    n tokens add n 2^-24."""
    R, A, D = q.shape
    H = K.shape[1]
    G = A // H
    out = np.zeros((R, A, D))
    lse = np.full((R, A), -np.inf)
    tol, ltol = np.zeros((R, A, D)), np.zeros((R, A))
    for r in range(R):
        n = min(max(int(lens[r]), 0), max_len)
        lo = max(0, n - window) if window else 0
        if n <= lo:
            continue
        t = np.arange(lo, n)
        p = table[r][t // page]
        for h in range(H):
            k = K[p, h, t % page, :D].double().numpy()
            v = V[p, h, t % page // 8, :D, t % page % 8].double().numpy()
            if ks is not None:
                k = k * ks[p, h, t % page].double().numpy()[:, None]
                v = v * vs[p, h, t % page].double().numpy()[:, None]
            for a in range(h * G, (h + 1) * G):
                x = k @ q[r, a] * scale
                m = x.max()
                w = np.exp(x - m)
                out[r, a] = w @ v / w.sum()
                lse[r, a] = m + math.log(w.sum())
                most = (np.abs(k) @ np.abs(q[r, a])).max() * abs(scale)
                eps = 2.0 ** -24 * (2 * (D + 16) * most + 64 + len(t))
                tol[r, a] = eps * (w @ np.abs(v)) / w.sum()
                ltol[r, a] = eps + 2.0 ** -22 * abs(lse[r, a])
    return out, lse, tol, ltol


def cache_sections(pages, H, P, D, int8, rng, fill=1.0):
    """Random sections of a cache on the CPU: K, V, ks, vs (None for bf16); padding elements zero in K."""
    Dp = (D + 31) // 32 * 32
    g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
    k, v = (torch.randn((pages, H, P, D), generator=g) * fill for _ in range(2))
    K = torch.zeros(pages, H, P, Dp, dtype=torch.int8 if int8 else torch.bfloat16)
    V = torch.zeros(pages, H, P // 8, Dp, 8, dtype=K.dtype)
    ks = vs = None
    if int8:
        q, d = codes(k.numpy())
        k, ks = torch.from_numpy(q), torch.from_numpy(d)
        q, d = codes(v.numpy())
        v, vs = torch.from_numpy(q), torch.from_numpy(d)
    K[..., :D] = k.to(K.dtype)
    V[..., :D, :] = v.to(V.dtype).view(pages, H, P // 8, 8, D).transpose(-1, -2)
    return K, V, ks, vs


# ------------------------------------------------------------------- norm
def norm(u, r, post, gate, pre, alpha, beta, eps_post, eps_pre):
    """fp64 residual update: r', h, and the fp32 error scale of each (terms' magnitudes)."""
    y = u
    if post is not None:
        y = u / np.sqrt((u * u).mean(1, keepdims=True) + eps_post) * post
    y = beta * y * (1 if gate is None else gate)
    ro = y if r is None else alpha * r + y
    mag = np.abs(y) + (0 if r is None else np.abs(alpha * r))
    if pre is None:
        return ro, ro, mag, mag
    f = pre / np.sqrt((ro * ro).mean(1, keepdims=True) + eps_pre)
    return ro, ro * f, mag, mag * np.abs(f) + np.abs(ro * f)
