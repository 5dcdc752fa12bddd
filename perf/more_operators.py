"""Cases, plain forms and work counts of the operators that serve prompts and shared pages beside the paged cache.

Five operators, named by a case's "op":

  rope     norms of queries and keys for each head and their rotation by position, in one pass (bq.qk_rope)
  prompt   attention of a request's new tokens, one or many, over the paged cache, with a window and first tokens that
           stay visible (bq.prompt_attn)
  shared   attention of one new token per request for groups of requests that share a prefix (bq.shared_attn)
  fork     requests continued from other requests, cut or freed, with pages shared and copied (bq.kv_fork, bq.kv_copy)
  compact  the pages in use moved to the low end of the pool (bq.kv_compact, bq.kv_copy)

With own = False `run` computes them with elementary torch operations in 32 bits (angles in 64); with own = True it
calls the library.  `exact` computes them once more in 64 bits.
"""
import math

import torch

own = False

BF16, F32, I8 = "bf16", "f32", "int8"
TORCH = {BF16: torch.bfloat16, F32: torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of 64 requests at far positions: norms, halves rotated, frequencies stretched for long contexts
        dict(name="rope_decode_64", op="rope", tokens=64, q_heads=64, k_heads=8, head_dim=128, rot=128, layout="half",
             norm=True, scaling="ramp", max_pos=131072, x=F32, out=BF16, idle=3),
        # a prompt's tokens: half of each head rotated, neighbouring pairs, no norms
        dict(name="rope_prompt_4096", op="rope", tokens=4096, q_heads=64, k_heads=8, head_dim=128, rot=64,
             layout="pairs", norm=False, scaling="none", max_pos=8192, x=BF16, out=BF16, idle=0),
        # a whole prompt of a 4096-wide layer (32 heads of 128 on 8)
        dict(name="prompt_1x4096", op="prompt", requests=1, chunk=4096, fill="full", heads=32, kv_heads=8, head_dim=128,
             page=64, max_len=4096, cache=BF16, q=BF16, out=BF16, window=0, sinks=0),
        # continuous batching: chunks of up to 512 tokens behind contexts of up to 16384, in a window with 4 first tokens
        dict(name="prompt_8x512_window_int8", op="prompt", requests=8, chunk=512, fill="ragged", heads=32, kv_heads=8,
             head_dim=128, page=32, max_len=16384, cache=I8, q=BF16, out=BF16, window=4096, sinks=4),
        # a decode step in a window with first tokens, 64 requests (8192 wide: 64 heads on 8)
        dict(name="prompt_64x1_window", op="prompt", requests=64, chunk=1, fill="full", heads=64, kv_heads=8,
             head_dim=128, page=16, max_len=8192, cache=BF16, q=BF16, out=BF16, window=2048, sinks=4),
        # one request checks 5 drafted tokens: latency, fp32 from the projections
        dict(name="prompt_1x5", op="prompt", requests=1, chunk=5, fill="full", heads=32, kv_heads=8, head_dim=128,
             page=16, max_len=2053, cache=BF16, q=F32, out=F32, window=0, sinks=0),
        # 64 conversations on one long document
        dict(name="shared_64x16384", op="shared", requests=64, groups=1, prefix=16384, own_len=1024, heads=64, kv_heads=8,
             head_dim=128, page=32, cache=BF16, q=BF16, out=BF16),
        # a few system prompts, 40 requests of 32 heads, int8 cache, fp32 in and out
        dict(name="shared_40_of_5_int8", op="shared", requests=40, groups=5, prefix=2000, own_len=700, heads=32,
             kv_heads=32, head_dim=64, page=16, cache=I8, q=F32, out=F32),
        # a step of beam search: 16 prompts of 4 beams
        dict(name="fork_beams_64", op="fork", requests=64, page=16, max_len=1024, mix="beams", kv_heads=8, head_dim=128,
             cache=BF16),
        # a serving batch: samples begun from one prompt, drafts taken back, requests ended
        dict(name="fork_mixed_256", op="fork", requests=256, page=64, max_len=8192, mix="mixed", kv_heads=2,
             head_dim=128, cache=BF16),
        # a small pool after some requests ended
        dict(name="compact_8", op="compact", requests=8, page=16, max_len=512, used=0.6, kv_heads=8, head_dim=128,
             cache=BF16),
        # a large pool at a third of its pages, before its upper part is given away
        dict(name="compact_256", op="compact", requests=256, page=16, max_len=1024, used=0.35, kv_heads=8, head_dim=128,
             cache=BF16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "prompt", "prompt", "shared", "shared", "fork", "compact"])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 128, 256])
        H = rng.choice([1, 2, 5, 8, 32])
        G = rng.choice([1, 2, 4, 7, 8]) if H < 32 else 1
        T = _log(rng, 1, max(1, min(8192, 2048 * 72 * 128 // (H * (G + 1) * D))))
        return dict(op=op, tokens=T, q_heads=H * G, k_heads=H, head_dim=D, rot=rng.choice([D, D, D // 2, D // 4]),
                    layout=rng.choice(["half", "pairs"]), norm=rng.random() < 0.6,
                    scaling=rng.choice(["none", "linear", "ramp", "band"]), max_pos=rng.choice([4096, 131072, 1000000]),
                    x=rng.choice([BF16, F32]), out=rng.choice([BF16, F32]), idle=rng.choice([0, 0, T // 5]))
    if op == "prompt":
        D = rng.choice([64, 64, 80, 96, 128, 128, 256])
        H = rng.choice([1, 2, 5, 8, 32])
        G = rng.choice([1, 1, 2, 4, 7, 8, 16, 20]) if H < 32 else 1
        R = _log(rng, 1, 64)
        N = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 16, 2048), _log(rng, 16, 2048)])
        N = max(1, min(N, 32768 * 128 // (R * H * G * D)))
        # (no more products than the whole prompt of 4096 tokens, no more keys than 64 windows of 2048)
        L = min(131072, 4096 * 4096 * 32 * 128 // (2 * R * N * H * G * D), 64 * 2048 * 8 * 128 // (R * H * D))
        L = _log(rng, N, max(N, L))
        w = rng.choice([0, 0, max(1, L // 3), min(L, 1024)])
        f32 = rng.choice([F32, BF16, BF16])
        return dict(op=op, requests=R, chunk=N, fill=rng.choice(["full", "ragged"]), heads=H * G, kv_heads=H, head_dim=D,
                    page=rng.choice([8, 16, 32, 64, 128]), max_len=L, cache=rng.choice([BF16, BF16, I8]), q=f32,
                    out=f32, window=w, sinks=rng.choice([0, 1, 4, 64]) if w else 0)
    if op == "shared":
        D = rng.choice([64, 80, 128, 128, 256])
        H = rng.choice([1, 2, 5, 8, 32])
        G = rng.choice([1, 2, 4, 7, 8]) if H < 32 else 1
        R = _log(rng, 2, 128)
        n = rng.choice([1, 1, 2, 5]) if R >= 5 else 1
        L = _log(rng, 16, max(16, min(32768, 64 * 16384 * 64 * 128 // (R * H * G * D), 256 * 1024 * 1024 // (R * H * D))))
        f32 = rng.choice([F32, BF16, BF16])
        return dict(op=op, requests=R, groups=n, prefix=L, own_len=_log(rng, 1, max(1, min(2048, L))), heads=H * G,
                    kv_heads=H, head_dim=D, page=rng.choice([8, 16, 32, 64, 128]), cache=rng.choice([BF16, BF16, I8]),
                    q=f32, out=f32)
    R = _log(rng, 2, 256)
    H, D = rng.choice([(1, 64), (2, 80), (8, 128), (5, 64)])
    P = rng.choice([8, 16, 32, 64])
    most = max(2 * P, min(8192, 256 * 1024 * 8 * 128 // (R * H * D)))
    L = _log(rng, 2 * P, most)
    c = dict(op=op, requests=R, page=P, max_len=L, kv_heads=H, head_dim=D, cache=BF16)
    return c | (dict(mix=rng.choice(["beams", "mixed"])) if op == "fork" else dict(used=round(rng.uniform(0.1, 0.9), 2)))


# --------------------------------------------------------- cache geometry
def _dp(D):
    """Elements of a cache row: the head dimension rounded up to 32, zero beyond it."""
    return (D + 31) // 32 * 32


def _a256(n):
    return (n + 255) // 256 * 256


def _cache(c, pages):
    """A cache of `pages` pages as one byte buffer, and its sections as views: K [page][head][token][Dp],
    V [page][head][token / 8][Dp][8] (and for int8 a scale per row of each)."""
    H, P, D = c["kv_heads"], c["page"], _dp(c["head_dim"])
    e = 2 if c["cache"] == BF16 else 1
    n = pages * H * P * D
    at = [0, _a256(n * e)]
    at.append(at[1] + _a256(n * e))
    at.append(at[2] + _a256(pages * H * P * 4))
    total = at[2] if c["cache"] == BF16 else at[3] + _a256(pages * H * P * 4)
    blob = torch.zeros(total, dtype=torch.uint8, device="cuda")
    t = torch.bfloat16 if c["cache"] == BF16 else torch.int8
    s = dict(cache=blob, pages=pages, K=blob[:n * e].view(t).view(pages, H, P, D),
             V=blob[at[1]:at[1] + n * e].view(t).view(pages, H, P // 8, D, 8))
    if c["cache"] == I8:
        s["ks"] = blob[at[2]:at[2] + pages * H * P * 4].view(torch.float32).view(pages, H, P)
        s["vs"] = blob[at[3]:at[3] + pages * H * P * 4].view(torch.float32).view(pages, H, P)
    return s


def _q8(x):
    """Codes and scale of rows (amax / 127, ties to even)."""
    amax = x.abs().amax(-1, keepdim=True)
    most = torch.full_like(amax, 127.0)
    s = torch.where(amax > 0, most / amax, 0.0)
    return torch.clamp(torch.round(x * s), -127, 127).to(torch.int8), (amax / most).squeeze(-1)


def _fill(c, s, g):
    """Random keys and values in every slot (what is past a request's length is another request's old data)."""
    K, V, D = s["K"], s["V"], c["head_dim"]
    step = max(1, (1 << 26) // K[0].numel())
    for k in range(0, K.shape[0], step):
        b = slice(k, k + step)
        for name in ("K", "V"):
            x = torch.randn((*K[b].shape[:3], D), generator=g, device="cuda")
            if c["cache"] == I8:
                x, sc = _q8(x)
                s["ks" if name == "K" else "vs"][b] = sc
            if name == "K":
                K[b, ..., :D] = x.to(K.dtype)
            else:
                V[b, ..., :D, :] = x.to(V.dtype).view(*V[b].shape[:3], 8, D).transpose(-1, -2)


def _tables(lens, page, stride, g, pages=None):
    """A table [R][stride] of pages in random order for requests of the given lengths (-1 elsewhere), and the pool's size
    (by default no more pages than they hold)."""
    held = (lens + page - 1) // page
    pages = max(1, int(held.sum())) if pages is None else pages
    order = torch.randperm(pages, generator=g, device="cuda")
    j = torch.arange(stride, device="cuda")
    at = (held.cumsum(0) - held)[:, None] + j
    return torch.where(j < held[:, None], order[at.clamp(max=pages - 1)], -1).to(torch.int32), pages


# ----------------------------------------------------------------- prepare
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return _PREPARE[c["op"]](c, g, int(seed)) | dict(op=c["op"], c=c)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _ints(g, lo, hi, n):
    return torch.randint(lo, hi, (n,), generator=g, device="cuda")


def _prepare_rope(c, g, seed):
    T, A, H, D = c["tokens"], c["q_heads"], c["k_heads"], c["head_dim"]
    x = _randn(g, T, A + 2 * H, D).to(TORCH[c["x"]])             # the rows of one projection: queries, keys, values
    pos = _ints(g, 0, c["max_pos"], T)
    if T > 256:                                                  # prompts: runs of positions
        t = torch.arange(T, device="cuda")
        pos = (pos[t // 1024] + t) % c["max_pos"]
    pos[T - c["idle"]:] = -1                                     # places of the list that hold no token
    o = TORCH[c["out"]]
    w = [(1 + 0.1 * _randn(g, D)) for _ in range(2)] if c["norm"] else [None, None]
    return dict(q=x[:, :A], k=x[:, A:A + H], qw=w[0], kw=w[1], pos=pos.to(torch.int32),
                qo=torch.zeros(T, A, D, dtype=o, device="cuda"), ko=torch.zeros(T, H, D, dtype=o, device="cuda"))


def _prepare_prompt(c, g, seed):
    R, N, P, L = c["requests"], c["chunk"], c["page"], c["max_len"]
    new = torch.full((R,), N, device="cuda")
    lens = torch.full((R,), L, device="cuda")
    if c["fill"] == "ragged":
        new = _ints(g, 0, N + 1, R)
        lens = torch.maximum(new, (torch.rand(R, generator=g, device="cuda") * (L + 1)).long().clamp(max=L))
        lens[seed % R], new[seed % R] = L, N                     # someone has the longest
    table, pages = _tables(lens, P, (L + P - 1) // P, g)
    s = _cache(c, pages)
    _fill(c, s, g)
    start = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), new.cumsum(0)])
    T = R * N                                                    # (rows past the last new token hold nothing)
    return s | dict(q=_randn(g, T, c["heads"], c["head_dim"]).to(TORCH[c["q"]]), table=table, lens=lens.to(torch.int32),
                    start=start.to(torch.int32),
                    res=torch.zeros(T, c["heads"], c["head_dim"], dtype=TORCH[c["out"]], device="cuda"),
                    lse=torch.zeros(T, c["heads"], dtype=torch.float32, device="cuda"))


def _prepare_shared(c, g, seed):
    R, n, P = c["requests"], c["groups"], c["page"]
    # group sizes as even as they go, prefixes from half of the longest on (the longest exists)
    start = torch.tensor([R * i // n for i in range(n + 1)], device="cuda")
    prefix = (c["prefix"] * (0.5 + 0.5 * torch.rand(n, generator=g, device="cuda"))).long().clamp(min=1)
    prefix[seed % n] = c["prefix"]
    own_len = 1 + (torch.rand(R, generator=g, device="cuda") * c["own_len"]).long().clamp(max=c["own_len"] - 1)
    of = torch.bucketize(torch.arange(R, device="cuda"), start[1:], right=True)
    lens = prefix[of] + own_len
    L = c["prefix"] + c["own_len"]
    stride = (L + P - 1) // P
    # whole pages of the prefix are the group's, the others each request's own (with the prefix's last tokens in them)
    whole = prefix // P
    held = (lens + P - 1) // P
    mine = held - whole[of]
    pages = int(whole.sum() + mine.sum())
    order = torch.randperm(pages, generator=g, device="cuda")
    j = torch.arange(stride, device="cuda")
    shared_at = (whole.cumsum(0) - whole)[of][:, None] + j
    own_at = whole.sum() + (mine.cumsum(0) - mine)[:, None] + j - whole[of][:, None]
    at = torch.where(j < whole[of][:, None], shared_at, own_at).clamp(0, pages - 1)
    table = torch.where(j < held[:, None], order[at], -1)
    s = _cache(c, pages)
    _fill(c, s, g)
    # the copies of the page that the prefix ends in agree in its tokens
    first = start[:-1][of]
    tail = (prefix % P)[of]
    last = whole[of].clamp(max=stride - 1)
    r = torch.arange(R, device="cuda")
    page, frm = table[r, last], table[first, last]
    o = torch.arange(P, device="cuda")
    take = (o < tail[:, None])                                   # [R][P]
    for name in ("K", "V", "ks", "vs"):
        if name not in s:
            continue
        x = s[name]
        if name == "V":
            m = take.view(R, 1, P // 8, 1, 8)
        else:
            m = take.view(R, 1, P, *([1] * (x.dim() - 3)))
        x[page] = torch.where(m, x[frm], x[page])
    return s | dict(q=_randn(g, R, c["heads"], c["head_dim"]).to(TORCH[c["q"]]), table=table.to(torch.int32),
                    lens=lens.to(torch.int32), start=start.to(torch.int32), prefix=prefix.to(torch.int32))


def _prepare_fork(c, g, seed):
    R, P, L = c["requests"], c["page"], c["max_len"]
    r = torch.arange(R, device="cuda")
    stride = (L + P - 1) // P
    if c["mix"] == "beams":                                      # 4 beams a prompt: whole pages shared, each its last page
        lens = (_ints(g, L // 2, L, R) // 4 * 4 + 1).clamp(max=L)[r // 4]
        src = r // 4 * 4 + _ints(g, 0, 4, R)
        src = src.clamp(max=R - 1)
        keep = lens[src]
    else:
        lens = _ints(g, 1, L + 1, R)
        kind = _ints(g, 0, 100, R)
        src = torch.where(kind < 40, _ints(g, 0, R, R), r)       # a sample begun from another request's tokens
        keep = torch.where(kind < 40, lens[src] - lens[src] // 8 * (kind % 2), lens)
        keep = torch.where((kind >= 40) & (kind < 60), lens - lens // 5, keep)      # drafts taken back
        keep = torch.where((kind >= 60) & (kind < 75), 0, keep)                     # ended
    table, pages = _tables(lens, P, stride, g, R * stride + R + 5)
    table = table.long()
    if c["mix"] == "beams":
        j = torch.arange(stride, device="cuda")
        same = j < (lens // P)[:, None]
        table = torch.where(same, table[r // 4 * 4], table)
    used = torch.zeros(pages + 1, dtype=torch.bool, device="cuda")
    used[torch.where(table >= 0, table, pages)] = True
    free = torch.nonzero(~used[:pages]).squeeze(1)
    free = free[torch.randperm(free.numel(), generator=g, device="cuda")]
    head = int(_ints(g, 0, pages, 1))
    ring = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(free.numel(), device="cuda")) % pages] = free.to(torch.int32)
    s = _cache(c, pages)
    _fill(c, s, g)
    return s | dict(src=src.to(torch.int32), keep=keep.to(torch.int32), lens=lens.to(torch.int32),
                    table=table.to(torch.int32), table_out=torch.full((R, stride), -1, dtype=torch.int32, device="cuda"),
                    ring=ring, state=torch.tensor([head, free.numel()], dtype=torch.int32, device="cuda"))


def _prepare_compact(c, g, seed):
    R, P, L = c["requests"], c["page"], c["max_len"]
    stride = (L + P - 1) // P
    some = (torch.rand(R, generator=g, device="cuda") * 2 * min(c["used"], 1 - c["used"]) * (L + 1)).long().clamp(max=L)
    lens = some if c["used"] < 0.5 else L - some                 # about `used` of the pool's pages together
    table, pages = _tables(lens, P, stride, g, R * stride + 1)
    s = _cache(c, pages)
    _fill(c, s, g)
    return s | dict(lens=lens.to(torch.int32), table=table,
                    table_out=torch.full((R, stride), -1, dtype=torch.int32, device="cuda"),
                    ring=torch.full((pages,), -1, dtype=torch.int32, device="cuda"))


_PREPARE = dict(rope=_prepare_rope, prompt=_prepare_prompt, shared=_prepare_shared, fork=_prepare_fork,
                compact=_prepare_compact)


# --------------------------------------------------------------------- run
def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


BASE, EPS, MSCALE = 500000.0, 1e-6, 1.1    # of the rotation's frequencies, of the norms, of the stretched rotation's length
FACTOR, TRAINED = 8.0, 8192                # contexts stretched by FACTOR over TRAINED positions
RAMP, BAND = (32.0, 1.0), (4.0, 1.0)       # turns over TRAINED from which a frequency stays, to which it is divided


def _freqs(c):
    """Radians per position of the rotated pairs, in 64 bits."""
    rot = c["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = BASE ** (-2 * i / rot)
    if c["scaling"] == "linear":
        return f / FACTOR
    if c["scaling"] == "ramp":                                   # a ramp over the pairs' numbers
        at = lambda turns: rot * math.log(TRAINED / (turns * 2 * math.pi)) / (2 * math.log(BASE))  # noqa: E731
        lo, hi = max(math.floor(at(RAMP[0])), 0), min(math.ceil(at(RAMP[1])), rot - 1)
        t = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / FACTOR * t + f * (1 - t)
    if c["scaling"] == "band":                                   # a ramp over the turns themselves
        turns = TRAINED * f / (2 * math.pi)
        t = ((turns - BAND[1]) / (BAND[0] - BAND[1])).clamp(0, 1)
        return f / FACTOR * (1 - t) + f * t
    return f


def _mscale(c):
    return MSCALE if c["scaling"] in ("ramp", "band") else 1.0


def _plain_rope(s):
    c, rot = s["c"], s["c"]["rot"]
    a = s["pos"].double()[:, None] * _freqs(c)
    cos, sin = (torch.cos(a) * _mscale(c)).float()[:, None], (torch.sin(a) * _mscale(c)).float()[:, None]
    out = {}
    for name, x, w, old in (("q", s["q"], s["qw"], s["qo"]), ("k", s["k"], s["kw"], s["ko"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        if c["layout"] == "half":
            u, v = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([u * cos - v * sin, v * cos + u * sin, x[..., rot:]], -1)
        else:
            u, v = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.cat([torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2), x[..., rot:]], -1)
        out[name] = torch.where(s["pos"][:, None, None] >= 0, y.to(old.dtype), old)
    return out


def _rows(s, page, off):
    """Keys and values [.., H, D] in 32 bits of the tokens at the given pages and offsets."""
    D = s["c"]["head_dim"]
    k, v = s["K"][page, :, off, :D].float(), s["V"][page, :, off // 8, :D, off % 8].float()
    if s["c"]["cache"] == I8:
        k, v = k * s["ks"][page, :, off][..., None], v * s["vs"][page, :, off][..., None]
    return k, v


def _softmax(x):
    """Weights' numerators, their sum and its logarithm; rows without a finite score have none."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    return p, torch.where(z > 0, z, 1.0), (m + torch.log(z)).squeeze(-1)


def _plain_prompt(s):
    c = s["c"]
    R, N, A, H, D, P = c["requests"], c["chunk"], c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    G, T, dev = A // H, R * N, s["q"].device
    lens, start = s["lens"].long(), s["start"].long()
    new = start[1:] - start[:-1]
    # the tokens that some new token sees: the first ones, then the last ones
    span = min(c["max_len"], c["window"] + N - 1) if c["window"] else c["max_len"]
    base = (lens - span).clamp(min=0)[:, None]
    few = torch.arange(c["sinks"], device=dev)[None].expand(R, -1)
    t = torch.cat([few, base + torch.arange(span, device=dev)], 1)                    # [R][n]
    once = torch.cat([few < base, torch.ones(R, span, dtype=torch.bool, device=dev)], 1) & (t < lens[:, None])
    page = torch.gather(s["table"].long(), 1, (t // P).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    k, v = _rows(s, page, t % P)                                                      # [R][n][H][D]
    i = torch.arange(N, device=dev)
    rows = torch.where(i < new[:, None], start[:-1, None] + i, T)                     # [R][N], T: none
    q = s["q"][rows.clamp(max=T - 1)].float().view(R, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(R, H, N * G, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))                 # [R][H][N G][n]
    pos = (lens - new)[:, None] + i                                                   # [R][N]
    keep = once[:, None] & (t[:, None] <= pos[..., None])
    if c["window"]:
        keep = keep & ((t[:, None] > pos[..., None] - c["window"]) | (t[:, None] < c["sinks"]))
    x = torch.where(keep[:, None, :, None].expand(R, H, N, G, -1).reshape(x.shape), x, -math.inf)
    p, z, lse = _softmax(x)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / z
    o = o.view(R, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(R * N, A, D)
    lse = lse.view(R, H, N, G).permute(0, 2, 1, 3).reshape(R * N, A)
    wide, lwide = torch.cat([s["res"], s["res"][:1]]), torch.cat([s["lse"], s["lse"][:1]])
    wide[rows.reshape(-1)] = o.to(wide.dtype)
    lwide[rows.reshape(-1)] = lse
    return dict(out=wide[:T], lse=lwide[:T])


def _plain_shared(s):
    c = s["c"]
    R, A, H, D, P = c["requests"], c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    t = torch.arange(c["prefix"] + c["own_len"], device=s["q"].device)
    page = s["table"].long()[:, t // P].clamp(min=0)
    k, v = _rows(s, page, (t % P)[None].expand(R, -1))
    q = s["q"].float().view(R, H, A // H, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    p, z, lse = _softmax(torch.where((t < s["lens"][:, None])[:, None, None], x, -math.inf))
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / z
    return dict(out=o.reshape(R, A, D).to(TORCH[c["out"]]), lse=lse.reshape(R, A))


def _copy_pages(s, frm, to, valid):
    """Pages `to` of the cache become copies of pages `frm`, where valid (elsewhere the first copy is made once more)."""
    frm, to = torch.where(valid, frm, frm[0]), torch.where(valid, to, to[0])
    frm, to = frm.clamp(min=0), torch.where(to < 0, frm, to)     # (no copy at all: a page onto itself)
    for x in (s["K"], s["V"]):
        x[to] = x[frm]
    return dict(K=s["K"], V=s["V"])


def _plain_fork(s):
    R, P = s["c"]["requests"], s["c"]["page"]
    table, ring, n = s["table"].long(), s["ring"], s["pages"]
    src, keep, lens = s["src"].long(), s["keep"].long(), s["lens"].long()
    r, j = torch.arange(R, device=src.device), torch.arange(table.shape[1], device=src.device)
    bad = (src < 0) | (src >= R) | (keep < 0) | (keep > lens[src.clamp(0, R - 1)])
    src, keep = torch.where(bad, r, src), torch.where(bad, lens, keep)
    rows = table[src]
    before = torch.zeros(n + 1, dtype=torch.bool, device=src.device)
    before[torch.where(j < ((lens + P - 1) // P)[:, None], table, n)] = True
    whole = torch.zeros(n + 1, dtype=torch.bool, device=src.device)
    whole[torch.where(j < (keep // P)[:, None], rows, n)] = True
    # of the requests that end inside a page the one that had it, or else the first, keeps it; unless it is another's whole page
    part = keep % P > 0
    last = torch.where(part, rows[r, (keep // P).clamp(max=table.shape[1] - 1)], n)
    key = torch.where(src == r, 0, R) + r
    first = torch.full((n + 1,), 2 * R, device=src.device).scatter_reduce(0, last, key, "amin")
    whole[n] = False
    copy = part & (whole[last] | (first[last] != key))
    want = copy.long().cumsum(0)
    given = copy & (want <= s["state"][1])
    cut = copy & ~given
    fresh = ring[(s["state"][0] + want - 1) % n].long()
    after = whole | (first < 2 * R)
    freed = (before & ~after)[:n]
    rank = freed.long().cumsum(0) - 1
    to = (s["state"][0] + s["state"][1] + rank) % n
    wide = torch.cat([ring, ring[:1]])
    wide[torch.where(freed, to, n)] = torch.arange(n, device=src.device, dtype=torch.int32)
    ring.copy_(wide[:n])
    now = torch.where(cut, keep - keep % P, keep)
    rows = torch.where((j == (keep // P)[:, None]) & given[:, None], fresh[:, None], rows)
    s["table_out"].copy_(torch.where(j < ((now + P - 1) // P)[:, None], rows, s["table_out"].long()))
    used = given.sum()
    at = torch.where(given, want - 1, R)
    pairs = torch.full((2, R + 1), -1, device=src.device)
    pairs[0, at], pairs[1, at] = last, fresh
    frm, to = pairs[0, :R], pairs[1, :R]
    after = torch.stack([(s["state"][0] + used) % n, s["state"][1] - used + freed.sum(), used, (bad | cut).sum()])
    return dict(table=s["table_out"], ring=ring, len=now.to(torch.int32), frm=frm.to(torch.int32), to=to.to(torch.int32),
                state=after.to(torch.int32), **_copy_pages(s, frm, to, frm >= 0))


def _plain_compact(s):
    P, n, table = s["c"]["page"], s["pages"], s["table"].long()
    lens, j = s["lens"].long(), torch.arange(table.shape[1], device=table.device)
    held = j < ((lens + P - 1) // P)[:, None]
    used = torch.zeros(n + 1, dtype=torch.bool, device=table.device)
    used[torch.where(held, table, n)] = True
    used = used[:n]
    p = torch.arange(n, device=table.device)
    place = lambda flags: torch.sort(torch.where(flags, p, n + p))[0]  # noqa: E731  (ascending, then the others)
    count = used.sum()
    top = torch.sort(torch.where(used, p, -1), descending=True)[0]      # used pages from the highest down
    low = place(~used)
    move = (top > low) & (top >= 0) & (low < n)
    frm, to = torch.where(move, top, -1), torch.where(move, low, -1)
    new = torch.cat([p, p[:1]])
    new[torch.where(move, top, n)] = low
    s["table_out"].copy_(torch.where(held, new[table.clamp(min=0)], s["table_out"].long()))
    free = p + count
    wide = torch.cat([s["ring"], s["ring"][:1]])
    wide[torch.where(free < n, p, n)] = free.clamp(max=n - 1).to(torch.int32)
    s["ring"].copy_(wide[:n])
    state = torch.stack([torch.zeros_like(count), n - count, move.sum(), count])
    return dict(table=s["table_out"], ring=s["ring"], frm=frm.to(torch.int32), to=to.to(torch.int32),
                state=state.to(torch.int32), **_copy_pages(s, frm, to, move))


_PLAIN = dict(rope=_plain_rope, prompt=_plain_prompt, shared=_plain_shared, fork=_plain_fork, compact=_plain_compact)


# ------------------------------------------------- the library's operators
def _dt(bq, name):
    return bq.DT_BF16 if name == BF16 else bq.DT_F32


def _kvdesc(bq, s):
    c = s["c"]
    return bq.kvdesc(c["kv_heads"], c["head_dim"], c["page"], s["pages"], bq.KV_BF16 if c["cache"] == BF16 else bq.KV_INT8)


def _own_rope(s):
    import bit_plane_gemv_amd as bq
    c = s["c"]
    if "h" not in s:
        kind = dict(none=bq.ROPE_PLAIN, linear=bq.ROPE_LINEAR, ramp=bq.ROPE_RAMP, band=bq.ROPE_BAND)[c["scaling"]]
        turns = dict(ramp=RAMP, band=BAND).get(c["scaling"], (0.0, 0.0))
        table = bq.rope_table(c["rot"], base=BASE, kind=kind, factor=FACTOR, trained=TRAINED, turns_keep=turns[0],
                              turns_scale=turns[1])
        d = bq.rope_desc(c["tokens"], c["q_heads"], c["k_heads"], c["head_dim"], rot=c["rot"],
                         layout=bq.ROPE_HALF if c["layout"] == "half" else bq.ROPE_PAIRS, x_dtype=_dt(bq, c["x"]),
                         out_dtype=_dt(bq, c["out"]), w_dtype=bq.DT_F32, eps=EPS, mscale=_mscale(c))
        s["h"] = (d, torch.from_numpy(table).cuda())
    d, table = s["h"]
    bq.qk_rope(d, s["q"], s["k"], s["qw"], s["kw"], table, s["pos"], s["qo"], s["ko"])
    return dict(q=s["qo"], k=s["ko"])


def _own_prompt(s):
    import bit_plane_gemv_amd as bq
    c = s["c"]
    if "h" not in s:
        d = bq.prompt_desc(_kvdesc(bq, s), c["heads"], c["requests"], s["q"].shape[0], s["table"].shape[1], c["max_len"],
                           window=c["window"], sinks=c["sinks"], q_dtype=_dt(bq, c["q"]), out_dtype=_dt(bq, c["out"]))
        s["h"] = (d, torch.empty(max(1, bq.prompt_attn_workspace(d)), dtype=torch.uint8, device="cuda"))
    d, ws = s["h"]
    bq.prompt_attn(d, s["q"], s["cache"], s["table"], s["start"], s["lens"], s["res"], ws, lse=s["lse"])
    return dict(out=s["res"], lse=s["lse"])


def _own_shared(s):
    import bit_plane_gemv_amd as bq
    c = s["c"]
    if "h" not in s:
        d = bq.shared_desc(bq.attn_desc(_kvdesc(bq, s), c["heads"], c["requests"], s["table"].shape[1],
                                        c["prefix"] + c["own_len"], q_dtype=_dt(bq, c["q"]), out_dtype=_dt(bq, c["out"])),
                           c["groups"], c["prefix"])
        s["h"] = (d, torch.empty(max(1, bq.shared_attn_workspace(d)), dtype=torch.uint8, device="cuda"),
                  torch.empty(s["q"].shape, dtype=TORCH[c["out"]], device="cuda"),
                  torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda"))
    d, ws, out, lse = s["h"]
    bq.shared_attn(d, s["q"], s["cache"], s["table"], s["lens"], s["start"], s["prefix"], out, ws, lse=lse)
    return dict(out=out, lse=lse)


def _pages_handle(bq, s, moves):
    if "h" not in s:
        d = bq.kv_pages_desc(s["c"]["requests"], s["c"]["page"], s["table"].shape[1], s["pages"], moves)
        buf = torch.empty(bq.kv_pages_size(d), dtype=torch.uint8, device="cuda")
        s["h"] = (d, _kvdesc(bq, s), buf, bq.kv_pages_views(d, buf),
                  torch.empty(bq.kv_pages_workspace(d), dtype=torch.uint8, device="cuda"))
    return s["h"]


def _own_fork(s):
    import bit_plane_gemv_amd as bq
    d, kv, buf, v, ws = _pages_handle(bq, s, s["c"]["requests"])
    bq.kv_fork(d, s["src"], s["keep"], s["lens"], s["ring"], s["state"], s["table"], s["table_out"], buf, ws)
    bq.kv_copy(kv, v["frm"], v["to"], s["cache"])
    return dict(table=s["table_out"], ring=s["ring"], len=v["len"], frm=v["frm"], to=v["to"], state=v["state"],
                K=s["K"], V=s["V"])


def _own_compact(s):
    import bit_plane_gemv_amd as bq
    d, kv, buf, v, ws = _pages_handle(bq, s, s["pages"])
    bq.kv_compact(d, s["lens"], s["table"], s["table_out"], s["ring"], buf, ws)
    bq.kv_copy(kv, v["frm"], v["to"], s["cache"])
    return dict(table=s["table_out"], ring=s["ring"], frm=v["frm"], to=v["to"], state=v["state"], K=s["K"], V=s["V"])


_OWN = dict(rope=_own_rope, prompt=_own_prompt, shared=_own_shared, fork=_own_fork, compact=_own_compact)


# -------------------------------------------------------------------- work
def _size(t):
    return {BF16: 2, F32: 4, I8: 1}[t]


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["tokens"] * (c["q_heads"] + c["k_heads"]) * c["head_dim"]
        return dict(bytes=n * (_size(c["x"]) + _size(c["out"])) + 4 * c["tokens"], flops=(8.0 if c["norm"] else 4.0) * n)
    if c["op"] == "prompt":
        R, N, L = c["requests"], c["chunk"], c["max_len"]
        full = c["fill"] == "full"
        n = N if full else (N + 1) / 2                           # means over the drawn lengths
        L = L if full else max(n, L / 2)
        w = min(L, c["window"] + c["sinks"]) if c["window"] else L
        seen = min(w, L - (n - 1) / 2) if L > n else min(w, (n + 1) / 2)                   # keys of a new token
        keys = min(L, c["window"] + c["sinks"] + n - 1) if c["window"] else L             # keys of a request
        row = 2 * c["head_dim"] * _size(c["cache"]) + (8 if c["cache"] == I8 else 0)
        io = c["head_dim"] * (_size(c["q"]) + _size(c["out"])) + 4
        return dict(bytes=R * (keys * c["kv_heads"] * row + n * c["heads"] * io),
                    flops=4.0 * R * n * seen * c["heads"] * c["head_dim"])
    if c["op"] == "shared":
        mean = c["prefix"] if c["groups"] == 1 else c["prefix"] * (0.75 + 0.25 / c["groups"])
        keys = c["groups"] * mean + c["requests"] * (c["own_len"] + 1) / 2
        row = 2 * c["head_dim"] * _size(c["cache"]) + (8 if c["cache"] == I8 else 0)
        io = c["head_dim"] * (_size(c["q"]) + _size(c["out"])) + 4
        return dict(bytes=keys * c["kv_heads"] * row + c["requests"] * c["heads"] * io,
                    flops=4.0 * c["requests"] * c["heads"] * c["head_dim"] * (mean + (c["own_len"] + 1) / 2))
    row = 2 * c["kv_heads"] * _dp(c["head_dim"]) * _size(c["cache"])
    per = c["max_len"] / c["page"]                               # most pages of a request
    if c["op"] == "fork":
        copies = 0.4 * c["requests"]
        return dict(bytes=2 * copies * c["page"] * row + 4 * c["requests"] * per, flops=0)
    used = c["requests"] * per * c["used"]
    moves = used * max(0.05, 1 - c["used"])
    return dict(bytes=2 * moves * c["page"] * row + 2 * 4 * used + 4 * c["requests"] * per, flops=0)


# ------------------------------------------------------------------- exact
def exact(case, seed):
    c = case
    if c["op"] in ("fork", "compact"):
        return None                                              # whole numbers and copies only
    s = prepare(case, seed)
    D = c["head_dim"]
    if c["op"] == "rope":
        half = c["rot"] // 2
        turn = torch.outer(s["pos"].double(), _exact_freqs(c)).unsqueeze(1)
        z = torch.polar(torch.full_like(turn, _mscale(c)), turn)                     # e^(i angle)
        res = {}
        for name, x, w in (("q", s["q"].double(), s["qw"]), ("k", s["k"].double(), s["kw"])):
            if w is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * w.double()
            y = x.clone()
            if c["layout"] == "half":
                p = torch.complex(x[..., :half].contiguous(), x[..., half:c["rot"]].contiguous()) * z
                y[..., :half], y[..., half:c["rot"]] = p.real, p.imag
            else:
                p = torch.view_as_complex(x[..., :c["rot"]].reshape(*x.shape[:-1], half, 2).contiguous()) * z
                y[..., :c["rot"]] = torch.view_as_real(p).flatten(-2)
            y[s["pos"] < 0] = 0
            res[name] = y
        return res
    A, H, P = c["heads"], c["kv_heads"], c["page"]
    G = A // H
    rows = s["q"].shape[0]
    out = torch.zeros(rows, A, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(rows, A, dtype=torch.float64, device="cuda")
    start = s["start"].tolist() if c["op"] == "prompt" else list(range(c["requests"] + 1))
    for i, n in enumerate(s["lens"].tolist()):
        a, b = start[i], start[i + 1]
        if a == b:
            continue
        first = max(0, n - (b - a) + 1 - c["window"]) if c.get("window") else 0      # of the first new token's window
        see = torch.arange(n, device="cuda")
        see = see[(see >= first) | (see < c.get("sinks", 0))]
        page, off = s["table"][i].long()[see // P], see % P
        at = torch.arange(n - (b - a), n, device="cuda")[:, None]
        hide = see > at
        if c.get("window"):
            hide = hide | ((see <= at - c["window"]) & (see >= c["sinks"]))
        for h in range(H):
            k, v = s["K"][page, h, off, :D].double(), s["V"][page, h, off // 8, :D, off % 8].double()
            if c["cache"] == I8:
                k, v = k * s["ks"][page, h, off].double()[:, None], v * s["vs"][page, h, off].double()[:, None]
            for g in range(h * G, (h + 1) * G):
                x = (s["q"][a:b, g].double() @ k.t()).div_(math.sqrt(D)).masked_fill_(hide, -math.inf)
                lse[a:b, g] = torch.logsumexp(x, 1)
                out[a:b, g] = torch.softmax(x, 1) @ v
    return dict(out=out, lse=lse)


def _exact_freqs(c):
    """Radians per position, pair by pair, from the definition."""
    rot, f = c["rot"], []
    for i in range(rot // 2):
        x = math.exp(-2 * i / rot * math.log(BASE))
        keep = 1.0
        if c["scaling"] == "linear":
            keep = 0.0
        elif c["scaling"] == "ramp":
            lo, hi = (rot * math.log(TRAINED / (2 * math.pi * t)) / (2 * math.log(BASE)) for t in RAMP)
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
            keep = 1 - min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        elif c["scaling"] == "band":
            keep = min(max((TRAINED * x / (2 * math.pi) - BAND[1]) / (BAND[0] - BAND[1]), 0.0), 1.0)
        f.append(x * keep + x / FACTOR * (1 - keep))
    return torch.tensor(f, dtype=torch.float64, device="cuda")
