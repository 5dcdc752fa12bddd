"""Cases, plain forms and work counts of the operators around the packed linear layers of a decoder.

Five operators, named by a case's "op":

  plan   block tables and slot maps of a paged cache, from the requests' lengths (bq.kv_plan)
  write  new key and value rows into the paged cache (bq.kv_write)
  attn   attention of one new token per request over the paged cache (bq.paged_attn)
  norm   residual update of a block with its gate, scale and two RMS norms (bq.block_norm)
  w8a8   int8 x int8 matrix product with a scale per token and channel (bq.gemm_w8a8)

With own = False `run` computes them with elementary torch operations in 32 bits; with own = True it
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
        # one decode step of 64 requests: every request gains one token
        dict(name="plan_decode_64", op="plan", requests=64, page=16, max_len=4096, mix="decode", tokens=64, short=False),
        # continuous batching: prefills, decodes, finished and idle requests in one step
        dict(name="plan_mixed_1024", op="plan", requests=1024, page=32, max_len=16384, mix="mixed", tokens=65536,
             short=False),
        # the 64 new rows of that decode step, fp32 as the GEMVs write them (8 key-value heads)
        dict(name="write_decode_64", op="write", tokens=64, kv_heads=8, head_dim=128, page=16, cache=BF16, x=F32,
             run=1),
        # prompts of 1365 and fewer tokens, 4096 together, at the 32 heads of a 4096-wide layer
        dict(name="write_prefill_4096", op="write", tokens=4096, kv_heads=32, head_dim=128, page=64, cache=BF16,
             x=BF16, run=1365),
        # one conversation, 32 heads of 128 (4096 wide): the latency of a step
        dict(name="attn_1x2049", op="attn", requests=1, heads=32, kv_heads=32, head_dim=128, page=16, max_len=2049,
             fill="full", cache=BF16, q=F32, out=F32, window=0),
        # a serving batch of ragged lengths, 64 query heads on 8 key-value heads (8192 wide), int8 cache
        dict(name="attn_64_ragged_int8", op="attn", requests=64, heads=64, kv_heads=8, head_dim=128, page=32,
             max_len=8192, fill="ragged", cache=I8, q=BF16, out=BF16, window=0),
        # few requests with very long contexts: the length is split over the whole GPU
        dict(name="attn_3x131072", op="attn", requests=3, heads=64, kv_heads=8, head_dim=128, page=64, max_len=131072,
             fill="full", cache=BF16, q=BF16, out=BF16, window=0),
        # one token through a block's residual update, fp32 stream
        dict(name="norm_1x4096", op="norm", rows=1, width=4096, u=F32, r=F32, out=BF16, post=True, gate="channel",
             w=F32),
        # a prefill's residual update, bf16, gate per token
        dict(name="norm_4096x8192", op="norm", rows=4096, width=8192, u=BF16, r=BF16, out=BF16, post=True,
             gate="token", w=BF16),
        # decode of one token through an 8-bit layer (11008 x 4096)
        dict(name="w8a8_1_11008x4096", op="w8a8", M=1, N=11008, K=4096, y=F32),
        # a decode batch through the down projection (4096 x 11008)
        dict(name="w8a8_64_4096x11008", op="w8a8", M=64, N=4096, K=11008, y=F32),
        # a prefill of 4096 tokens
        dict(name="w8a8_4096_11008x4096", op="w8a8", M=4096, N=11008, K=4096, y=BF16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write", "attn", "attn", "norm", "w8a8", "w8a8"])
    if op == "plan":
        mix = rng.choice(["decode", "mixed"])
        R = _log(rng, 1, 1024)
        max_len = _log(rng, 64, 16384)
        T = R if mix == "decode" else min(65536, R * max(1, max_len // 4))
        return dict(op=op, requests=R, page=rng.choice([8, 16, 32, 64, 128, 256]), max_len=max_len, mix=mix, tokens=T,
                    short=rng.random() < 0.25)
    if op == "write":
        T = _log(rng, 1, 4096)
        D = rng.choice([40, 64, 80, 96, 128, 256])
        H = rng.choice([h for h in (1, 2, 5, 8, 32) if T * h * D <= 4096 * 32 * 128])
        return dict(op=op, tokens=T, kv_heads=H, head_dim=D, page=rng.choice([8, 16, 32, 64, 128]),
                    cache=rng.choice([BF16, I8]), x=rng.choice([BF16, F32]), run=min(T, _log(rng, 1, 2048)))
    if op == "attn":
        D = rng.choice([64, 64, 80, 96, 128, 128, 256])
        H = rng.choice([1, 2, 5, 8, 32])
        G = rng.choice([1, 1, 2, 4, 7, 8, 16, 20]) if H < 32 else 1
        R = _log(rng, 1, 256)
        most = max(1, min(131072, (64 * 8192 * 8 * 128) // (R * H * D)))
        L = _log(rng, 1, most)
        return dict(op=op, requests=R, heads=H * G, kv_heads=H, head_dim=D, page=rng.choice([8, 16, 32, 64, 128]),
                    max_len=L, fill=rng.choice(["full", "ragged", "ragged"]), cache=rng.choice([BF16, BF16, I8]),
                    q=rng.choice([BF16, F32]), out=rng.choice([BF16, F32]),
                    window=rng.choice([0, 0, 0, max(1, L // 3)]))
    if op == "norm":
        C = _log(rng, 64, 28672)
        C = C if rng.random() < 0.25 else max(64, C // 64 * 64)
        M = _log(rng, 1, max(1, min(8192, 4096 * 8192 // C)))
        return dict(op=op, rows=M, width=C, u=rng.choice([BF16, F32]), r=rng.choice([BF16, F32]),
                    out=rng.choice([BF16, F32]), post=rng.random() < 0.7,
                    gate=rng.choice(["none", "channel", "token"]), w=rng.choice([BF16, F32]))
    K = max(64, _log(rng, 64, 28672) // 16 * 16)
    N = _log(rng, 16, 28672)
    M = _log(rng, 1, max(1, min(8192, 4096 * 11008 * 4096 // (N * K))))
    return dict(op=op, M=M, N=N, K=K, y=rng.choice([BF16, F32]))


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
    s = dict(cache=blob, K=blob[:n * e].view(t).view(pages, H, P, D),
             V=blob[at[1]:at[1] + n * e].view(t).view(pages, H, P // 8, D, 8))
    if c["cache"] == I8:
        s["ks"] = blob[at[2]:at[2] + pages * H * P * 4].view(torch.float32).view(pages, H, P)
        s["vs"] = blob[at[3]:at[3] + pages * H * P * 4].view(torch.float32).view(pages, H, P)
    return s


def _q8(x):
    """Codes and scale of rows: the activation quantizer's arithmetic (amax / 127, ties to even)."""
    amax = x.abs().amax(-1, keepdim=True)
    most = torch.full_like(amax, 127.0)                          # (a tensor: division by a number is rounded twice)
    s = torch.where(amax > 0, most / amax, 0.0)
    return torch.clamp(torch.round(x * s), -127, 127).to(torch.int8), (amax / most).squeeze(-1)


def _fill(c, s, g):
    """Random keys and values in every slot (what is past a request's length is another request's old data)."""
    K, V, D = s["K"], s["V"], c["head_dim"]
    for k in range(0, K.shape[0], max(1, (1 << 26) // K[0].numel())):
        b = slice(k, k + max(1, (1 << 26) // K[0].numel()))
        for name in ("K", "V"):
            x = torch.randn((*K[b].shape[:3], D), generator=g, device="cuda")
            if c["cache"] == I8:
                x, sc = _q8(x)
                s["ks" if name == "K" else "vs"][b] = sc
            if name == "K":
                K[b, ..., :D] = x.to(K.dtype)
            else:
                V[b, ..., :D, :] = x.to(V.dtype).view(*V[b].shape[:3], 8, D).transpose(-1, -2)


# ----------------------------------------------------------------- prepare
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    f = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    ints = lambda lo, hi, n: torch.randint(lo, hi, (n,), generator=g, device="cuda")  # noqa: E731
    if c["op"] == "plan":
        return _prepare_plan(c, g, ints)
    if c["op"] == "write":
        T, P = c["tokens"], c["page"]
        runs = (T + c["run"] - 1) // c["run"]                    # runs of consecutive positions, one per request
        per = (c["run"] + P - 1) // P + 1
        s = _cache(c, runs * per + 3)
        first = ints(0, P, runs)
        table = torch.randperm(runs * per + 3, generator=g, device="cuda")[:runs * per].view(runs, per)
        t = torch.arange(T, device="cuda")
        r, pos = t // c["run"], first[t // c["run"]] + t % c["run"]
        s["slots"] = (table[r, pos // P] * P + pos % P).to(torch.int32)
        kv = f(T, 2, c["kv_heads"], c["head_dim"]).to(TORCH[c["x"]])   # the rows of one K/V projection, side by side
        s |= dict(op="write", c=c, k=kv[:, 0], v=kv[:, 1])
        return s
    if c["op"] == "attn":
        R, P, L = c["requests"], c["page"], c["max_len"]
        lens = torch.full((R,), L, device="cuda")
        if c["fill"] == "ragged":
            lens = (torch.rand(R, generator=g, device="cuda") ** 2 * (L + 1)).long().clamp(max=L)
            lens[int(seed) % R] = L                              # someone has the longest
        per = (L + P - 1) // P
        held = (lens + P - 1) // P
        pages = R * per if c["fill"] == "full" else max(1, int(held.sum())) + 1
        s = _cache(c, pages)
        _fill(c, s, g)
        order = torch.randperm(pages, generator=g, device="cuda")
        j = torch.arange(per, device="cuda")
        at = (held.cumsum(0) - held)[:, None] + j
        s["table"] = torch.where(j < held[:, None], order[at.clamp(max=pages - 1)], 0).to(torch.int32)
        s |= dict(op="attn", c=c, q=f(R, c["heads"], c["head_dim"]).to(TORCH[c["q"]]), lens=lens.to(torch.int32))
        return s
    if c["op"] == "norm":
        M, C, w = c["rows"], c["width"], TORCH[c["w"]]
        s = dict(op="norm", c=c, u=(3 * f(M, C)).to(TORCH[c["u"]]), r=(2 * f(M, C)).to(TORCH[c["r"]]),
                 pre=(1 + 0.1 * f(C)).to(w), post=(1 + 0.1 * f(C)).to(w) if c["post"] else None)
        s["gate"] = None if c["gate"] == "none" else f(*((C,) if c["gate"] == "channel" else (M, C))).to(w)
        return s
    M, N, K = c["M"], c["N"], c["K"]
    a, sa = _q8(f(M, K))
    w, sw = _q8(f(N, K) * 0.02)
    return dict(op="w8a8", c=c, a=a, sa=sa, w=w, sw=sw)


def _prepare_plan(c, g, ints):
    R, P, L, T = c["requests"], c["page"], c["max_len"], c["tokens"]
    old, new = ints(0, L, R), None
    if c["mix"] == "decode":
        new = old + 1
    else:
        kind = ints(0, 100, R)
        old = torch.where(kind < 15, torch.zeros_like(old), old)                 # a new prompt
        prompt = ints(1, L + 1, R)
        grown = torch.minimum(old + 1 + ints(0, 4, R), torch.full_like(old, L))  # a token, or a few accepted drafts
        new = torch.where(kind < 15, prompt, grown)
        new = torch.where((kind >= 85) & (kind < 92), torch.zeros_like(old), new)       # finished
        new = torch.where((kind >= 92) & (kind < 95), old - old // 3, new)              # drafts taken back
        new = torch.where(kind >= 95, old, new)                                         # idle
    per = (L + P - 1) // P
    held, need = (old + P - 1) // P, (new + P - 1) // P
    cap = R * per + 7                                                                   # pages of the pool
    free = int((need - held).clamp(min=0).sum()) // 2 if c["short"] else cap - int(held.sum())
    ids = torch.randperm(cap, generator=g, device="cuda").to(torch.int32)
    j = torch.arange(per, device="cuda")
    at = (held.cumsum(0) - held)[:, None] + j
    table = torch.where(j < held[:, None], ids[at.clamp(max=cap - 1)], -1).to(torch.int32)
    ring = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    head = int(ints(0, cap, 1))
    k = torch.arange(free, device="cuda")
    ring[(head + k) % cap] = ids[cap - free:]
    return dict(op="plan", c=c, old=old.to(torch.int32), new=new.to(torch.int32), table=table, ring=ring,
                state=torch.tensor([head, free], dtype=torch.int32, device="cuda"))


# --------------------------------------------------------------------- run
def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _plain_plan(s):
    c, table, ring = s["c"], s["table"], s["ring"]
    P, T, cap, per = c["page"], c["tokens"], ring.numel(), table.shape[1]
    old, new = s["old"], s["new"]
    fits = (old >= 0) & (new >= 0) & (torch.maximum(old, new) <= per * P)
    held, need = (old + P - 1) // P, (new + P - 1) // P
    grow = fits & (new > old)
    pops = torch.where(grow, need - held, 0)
    toks = torch.where(grow, new - old, 0)
    free = s["state"][1]
    cp, ct = pops.cumsum(0), toks.cumsum(0)
    given = grow & (cp <= free) & (ct <= T)
    cut = fits & (new <= old)
    pops, toks = torch.where(given, pops, 0), torch.where(given, toks, 0)
    push = torch.where(cut, held - need, 0)
    ep, et, eu = pops.cumsum(0) - pops, toks.cumsum(0) - toks, push.cumsum(0) - push
    j = torch.arange(per, device=old.device)
    take = given[:, None] & (j >= held[:, None]) & (j < need[:, None])
    frm = (s["state"][0] + ep[:, None] + j - held[:, None]) % cap
    back = cut[:, None] & (j >= need[:, None]) & (j < held[:, None])
    to = (s["state"][0] + free + eu[:, None] + j - need[:, None]) % cap
    table.copy_(torch.where(take, ring[frm], table))
    wide = torch.cat([ring, ring[:1]])
    wide.scatter_(0, torch.where(back, to, cap).reshape(-1), table.reshape(-1))
    ring.copy_(wide[:cap])
    now = torch.where(given | cut, new, old)
    total = toks.sum()
    start = torch.cat([et, total[None]]).to(torch.int32)
    t = torch.arange(T, device=old.device)
    r = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=c["requests"] - 1)
    ok = t < total
    pos = old[r] + t - start[r]
    page = table[r, (pos // P).clamp(0, per - 1)]
    minus = torch.full_like(t, -1)
    pick = lambda v: torch.where(ok, v, minus).to(torch.int32)  # noqa: E731
    refused = (~(given | cut)).sum()
    taken = pops.sum()
    after = torch.stack([(s["state"][0] + taken) % cap, free - taken + push.sum(), total, refused]).to(torch.int32)
    return dict(table=table, ring=ring, len=now.to(torch.int32), start=start, slot=pick(page * P + pos % P), req=pick(r),
                pos=pick(pos), state=after)


def _plain_write(s):
    c, P, D, H = s["c"], s["c"]["page"], s["c"]["head_dim"], s["c"]["kv_heads"]
    slot = s["slots"].long()
    page, off = slot // P, slot % P
    k, v = s["k"].float(), s["v"].float()
    h = torch.arange(H, device=slot.device)
    if c["cache"] == I8:
        k, sk = _q8(k)
        v, sv = _q8(v)
        s["ks"][page[:, None], h, off[:, None]] = sk
        s["vs"][page[:, None], h, off[:, None]] = sv
    s["K"][page[:, None], h, off[:, None], :D] = k.to(s["K"].dtype)
    d = torch.arange(D, device=slot.device)
    s["V"][page[:, None, None], h[:, None], (off // 8)[:, None, None], d, (off % 8)[:, None, None]] = v.to(s["V"].dtype)
    return _written(s)


def _written(s):
    """The updated cache: its own rows, or the values that int8 codes stand for, with the scales."""
    K, V = s["K"], s["V"]
    if s["c"]["cache"] == BF16:
        return dict(K=K, V=V)
    return dict(K=K * s["ks"][..., None], V=V * s["vs"].view(*V.shape[:3], 1, 8), ks=s["ks"], vs=s["vs"])


def _plain_attn(s):
    c = s["c"]
    R, H, D, P, L = c["requests"], c["kv_heads"], c["head_dim"], c["page"], c["max_len"]
    table = s["table"].long()
    k = s["K"][table].float()                                                   # [R][n][H][P][Dp]
    v = s["V"][table].float().transpose(-1, -2).reshape(k.shape)
    if c["cache"] == I8:
        k = k * s["ks"][table][..., None]
        v = v * s["vs"][table][..., None]
    n = k.shape[1] * P
    k = k.transpose(1, 2).reshape(R, H, n, -1)[..., :D]
    v = v.transpose(1, 2).reshape(R, H, n, -1)[..., :D]
    q = s["q"].float().view(R, H, c["heads"] // H, D)
    x = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    t = torch.arange(n, device=x.device)
    lens = s["lens"][:, None]
    keep = t < lens
    if c["window"]:
        keep = keep & (t >= lens - c["window"])
    x = torch.where(keep[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(z > 0, z, 1.0)
    return dict(out=o.reshape(R, c["heads"], D).to(TORCH[c["out"]]), lse=(m + torch.log(z)).reshape(R, c["heads"]))


ALPHA, BETA, EPS = 1.0, 0.22, 1e-5     # residual scale, branch scale, epsilon of both norms


def _plain_norm(s):
    y = s["u"].float()
    if s["post"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * s["post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    r = (ALPHA * s["r"].float() + BETA * y)
    h = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["pre"].float()
    return dict(r=r.to(s["r"].dtype), h=h.to(TORCH[s["c"]["out"]]))


def _plain_w8a8(s):
    y = torch.matmul(s["a"].float(), s["w"].float().t())
    return (y * s["sa"][:, None] * s["sw"]).to(TORCH[s["c"]["y"]])


_PLAIN = dict(plan=_plain_plan, write=_plain_write, attn=_plain_attn, norm=_plain_norm, w8a8=_plain_w8a8)


# ------------------------------------------------- the library's operators
def _dt(bq, name):
    return bq.DT_BF16 if name == BF16 else bq.DT_F32


def _kvdesc(bq, s):
    c = s["c"]
    return bq.kvdesc(c["kv_heads"], c["head_dim"], c["page"], s["K"].shape[0], bq.KV_BF16 if c["cache"] == BF16 else bq.KV_INT8)


def _own_plan(s):
    import bit_plane_gemv_amd as bq
    if "h" not in s:
        c = s["c"]
        d = bq.kv_plan_desc(c["requests"], c["page"], s["table"].shape[1], s["ring"].numel(), c["tokens"])
        buf = torch.empty(bq.kv_plan_size(d), dtype=torch.uint8, device="cuda")
        s["h"] = (d, buf, bq.kv_plan_views(d, buf))
    d, buf, views = s["h"]
    bq.kv_plan(d, s["old"], s["new"], s["ring"], s["state"], s["table"], buf)
    return dict(views, table=s["table"], ring=s["ring"])


def _own_write(s):
    import bit_plane_gemv_amd as bq
    if "h" not in s:
        s["h"] = _kvdesc(bq, s)
    bq.kv_write(s["h"], s["k"], s["v"], _dt(bq, s["c"]["x"]), s["slots"], s["cache"])
    return _written(s)


def _own_attn(s):
    import bit_plane_gemv_amd as bq
    c = s["c"]
    if "h" not in s:
        d = bq.attn_desc(_kvdesc(bq, s), c["heads"], c["requests"], s["table"].shape[1], c["max_len"],
                         window=c["window"], q_dtype=_dt(bq, c["q"]), out_dtype=_dt(bq, c["out"]))
        s["h"] = (d, torch.zeros(bq.paged_attn_workspace(d), dtype=torch.uint8, device="cuda"),
                  torch.empty(s["q"].shape, dtype=TORCH[c["out"]], device="cuda"),
                  torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda"))
    d, ws, out, lse = s["h"]
    bq.paged_attn(d, s["q"], s["cache"], s["table"], s["lens"], out, ws, lse=lse)
    return dict(out=out, lse=lse)


def _own_norm(s):
    import bit_plane_gemv_amd as bq
    c = s["c"]
    if "h" not in s:
        d = bq.norm_desc(c["rows"], c["width"], u_dtype=_dt(bq, c["u"]), r_dtype=_dt(bq, c["r"]),
                         w_dtype=_dt(bq, c["w"]), out_dtype=_dt(bq, c["out"]), res_scale=ALPHA, branch_scale=BETA,
                         eps_post=EPS, eps_pre=EPS, gate_stride=c["width"] if c["gate"] == "token" else 0)
        s["h"] = (d, torch.empty_like(s["r"]), torch.empty(s["r"].shape, dtype=TORCH[c["out"]], device="cuda"))
    d, r, h = s["h"]
    bq.block_norm(d, s["u"], s["r"], s["post"], s["gate"], s["pre"], r, h)
    return dict(r=r, h=h)


def _own_w8a8(s):
    import bit_plane_gemv_amd as bq
    c = s["c"]
    if "h" not in s:
        d = bq.w8a8_desc(c["M"], c["N"], c["K"], y_dtype=_dt(bq, c["y"]))
        s["h"] = (d, torch.empty((c["M"], c["N"]), dtype=TORCH[c["y"]], device="cuda"),
                  torch.zeros(bq.w8a8_workspace(d), dtype=torch.uint8, device="cuda"))
    d, y, ws = s["h"]
    bq.gemm_w8a8(d, s["a"], s["sa"], s["w"], s["sw"], y, ws)
    return y


_OWN = dict(plan=_own_plan, write=_own_write, attn=_own_attn, norm=_own_norm, w8a8=_own_w8a8)


# -------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "plan":
        R, P, T = c["requests"], c["page"], c["tokens"]
        # lengths in and out, starts, three words a token, and the table entries that tokens and pages touch
        return dict(bytes=4 * (4 * R + 3 * T + T // P + R), flops=0)
    if c["op"] == "write":
        n = 2 * c["tokens"] * c["kv_heads"] * c["head_dim"]
        return dict(bytes=n * (2 if c["x"] == BF16 else 4) + n * (2 if c["cache"] == BF16 else 1) +
                    (8 * c["tokens"] * c["kv_heads"] if c["cache"] == I8 else 0) + 4 * c["tokens"], flops=0)
    if c["op"] == "attn":
        share = 1.0 if c["fill"] == "full" else 1 / 3
        L = c["max_len"] * share
        if c["window"]:
            L = min(L, c["window"])
        n = c["requests"] * L * c["kv_heads"]
        row = 2 * c["head_dim"] * (2 if c["cache"] == BF16 else 1) + (8 if c["cache"] == I8 else 0)
        qo = c["requests"] * c["heads"] * (c["head_dim"] * ((2 if c["q"] == BF16 else 4) + (2 if c["out"] == BF16 else 4)) + 4)
        return dict(bytes=n * row + qo, flops=4.0 * c["requests"] * L * c["heads"] * c["head_dim"])
    if c["op"] == "norm":
        size = lambda t: 2 if t == BF16 else 4  # noqa: E731
        n = c["rows"] * c["width"]
        gate = {"none": 0, "channel": c["width"], "token": n}[c["gate"]] * size(c["w"])
        return dict(bytes=n * (size(c["u"]) + 2 * size(c["r"]) + size(c["out"])) + gate +
                    c["width"] * size(c["w"]) * (1 + int(c["post"])), flops=10.0 * n)
    M, N, K = c["M"], c["N"], c["K"]
    return dict(bytes=M * K + N * K + 4 * (M + N) + M * N * (2 if c["y"] == BF16 else 4), flops=2.0 * M * N * K)


# ------------------------------------------------------------------- exact
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "plan":
        return None                                              # whole numbers only
    if c["op"] == "norm":
        u, r = s["u"].double(), s["r"].double()
        if c["post"]:
            u = u / torch.sqrt((u * u).sum(1) / c["width"] + EPS).unsqueeze(1) * s["post"].double()
        if s["gate"] is not None:
            u = u * s["gate"].double()
        r = r * ALPHA + u * BETA
        norm = torch.sqrt((r * r).sum(1) / c["width"] + EPS)
        return dict(r=r, h=r / norm.unsqueeze(1) * s["pre"].double())
    if c["op"] == "w8a8":
        y = torch.empty(c["M"], c["N"], dtype=torch.float64, device="cuda")
        w = s["w"].double() * s["sw"].double().unsqueeze(1)
        for i in range(0, c["M"], 1024):
            b = slice(i, i + 1024)
            y[b] = torch.mm(s["a"][b].double() * s["sa"][b].double().unsqueeze(1), w.t())
        return y
    if c["op"] == "write":
        P, D = c["page"], c["head_dim"]
        slot = s["slots"].long().cpu()
        if c["cache"] == I8:
            res = dict(K=None, V=None, ks=s["ks"].double(), vs=s["vs"].double())
            for name, x in (("ks", s["k"]), ("vs", s["v"])):
                flat = res[name].transpose(1, 2).reshape(-1, c["kv_heads"])
                flat[slot.cuda()] = x.double().abs().max(dim=2).values / 127
                res[name] = flat.view(-1, P, c["kv_heads"]).transpose(1, 2).contiguous()
            return res
        K, V = s["K"].double(), s["V"].double()
        for t in range(c["tokens"]):
            page, off = divmod(int(slot[t]), P)
            K[page, :, off, :D] = s["k"][t].double()
            V[page, :, off // 8, :D, off % 8] = s["v"][t].double()
        return dict(K=K, V=V)
    R, A, H, D, P = c["requests"], c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    out = torch.zeros(R, A, D, dtype=torch.float64, device="cuda")
    lse = torch.full((R, A), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n <= lo:
            continue
        pos = torch.arange(lo, n, device="cuda")
        page = s["table"][i].long()[pos // P]
        for h in range(H):
            k, v = s["K"][page, h, pos % P].double(), s["V"][page, h, pos % P // 8, :, pos % P % 8].double()
            if c["cache"] == I8:
                k, v = k * s["ks"][page, h, pos % P].double()[:, None], v * s["vs"][page, h, pos % P].double()[:, None]
            mine = slice(h * (A // H), (h + 1) * (A // H))
            x = s["q"][i, mine].double() @ k[:, :D].t() / math.sqrt(D)
            lse[i, mine] = torch.logsumexp(x, 1)
            out[i, mine] = torch.softmax(x, 1) @ v[:, :D]
    return dict(out=out, lse=lse)
