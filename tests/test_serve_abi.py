"""Refusals, sizes and layouts of the operators that serve prompts and shared pages (no GPU needed)."""
import ctypes

import pytest

import bit_plane_gemv_amd as bq

P = 1 << 20        # fake, well-aligned addresses: every call here fails before any device call
BIG = 1 << 60


def status(fn, *args):
    return getattr(bq._lib, fn)(*args)


def size(fn, desc):
    n = ctypes.c_size_t(0)
    return status(fn, desc, ctypes.byref(n)), n.value


def kv(**k):
    d = dict(kv_heads=4, head_dim=64, page=16, pages=10, dtype=bq.KV_BF16)
    d.update(k)
    return bq.KvDesc(*d.values())


def prompt(cache=None, **k):
    d = dict(heads=8, requests=3, tokens=40, table_stride=8, max_len=100, window=0, sinks=0, q_dtype=bq.DT_F32,
             out_dtype=bq.DT_BF16, scale=0.1)
    d.update(k)
    return bq.PromptDesc(cache or kv(), *d.values())


def shared(cache=None, groups=2, max_prefix=50, **k):
    d = dict(heads=8, requests=3, table_stride=8, max_len=100, window=0, q_dtype=bq.DT_F32, out_dtype=bq.DT_BF16, scale=0.1)
    d.update(k)
    return bq.SharedDesc(bq.AttnDesc(cache or kv(), *d.values()), groups, max_prefix)


def pages(**k):
    d = dict(requests=4, page=16, table_stride=8, pool=30, moves=30)
    d.update(k)
    return bq.KvPagesDesc(*d.values())


def rope(**k):
    d = dict(tokens=5, q_heads=4, k_heads=2, head_dim=64, rot=64, layout=0, x_dtype=0, out_dtype=1, w_dtype=0, eps=1e-6, mscale=1.0)
    d.update(k)
    return bq.RopeDesc(*d.values())


CACHE = [(dict(dtype=2), bq.E_ARG), (dict(kv_heads=0), bq.E_SHAPE), (dict(head_dim=257), bq.E_SHAPE), (dict(page=12), bq.E_SHAPE),
         (dict(pages=0), bq.E_SHAPE)]
ATTN = [(dict(heads=0), bq.E_SHAPE), (dict(heads=6), bq.E_SHAPE), (dict(heads=16388), bq.E_SHAPE), (dict(requests=0), bq.E_SHAPE),
        (dict(requests=8193), bq.E_SHAPE), (dict(table_stride=0), bq.E_SHAPE), (dict(max_len=0), bq.E_SHAPE), (dict(max_len=129), bq.E_SHAPE),
        (dict(window=-1), bq.E_SHAPE), (dict(q_dtype=2), bq.E_ARG), (dict(out_dtype=16), bq.E_ARG), (dict(scale=float("nan")), bq.E_ARG),
        (dict(scale=float("inf")), bq.E_ARG)]


@pytest.mark.parametrize("bad,want", [(dict(cache=kv(**b)), w) for b, w in CACHE] + ATTN + [
    (dict(tokens=0), bq.E_SHAPE), (dict(tokens=(1 << 20) + 1), bq.E_SHAPE), (dict(tokens=1 << 20, heads=128), bq.E_SHAPE),
    (dict(sinks=-1), bq.E_SHAPE), (dict(sinks=1), bq.E_SHAPE), (dict(sinks=-1, window=4), bq.E_SHAPE)])
def test_prompt_descriptor(bad, want):
    assert size("bitq_prompt_attn_workspace", prompt(**bad))[0] == want
    assert status("bitq_prompt_attn", prompt(**bad), P, 1 << 15, P, BIG, P, P, P, P, None, P, BIG, None) == want


@pytest.mark.parametrize("bad,want", [(dict(cache=kv(**b)), w) for b, w in CACHE] + ATTN + [
    (dict(window=4), bq.E_SHAPE), (dict(groups=0), bq.E_SHAPE), (dict(groups=4), bq.E_SHAPE), (dict(max_prefix=0), bq.E_SHAPE),
    (dict(max_prefix=101), bq.E_SHAPE)])
def test_shared_descriptor(bad, want):
    assert size("bitq_shared_attn_workspace", shared(**bad))[0] == want
    assert status("bitq_shared_attn", shared(**bad), P, 1 << 15, P, BIG, P, P, P, P, P, None, P, BIG, None) == want


def attention_calls():
    d, s = prompt(tokens=4, table_stride=80, max_len=1200), shared()
    c = bq.kv_cache_size(kv())
    yield ("bitq_prompt_attn", d, ["q", "stride", "cache", "bytes", "table", "start", "lens", "out", "lse", "ws", "ws_bytes"], c,
           size("bitq_prompt_attn_workspace", d)[1])
    yield ("bitq_shared_attn", s, ["q", "stride", "cache", "bytes", "table", "lens", "start", "prefix", "out", "lse", "ws", "ws_bytes"], c,
           size("bitq_shared_attn_workspace", s)[1])


@pytest.mark.parametrize("fn,desc,names,cache,ws", attention_calls(), ids=["prompt", "shared"])
def test_attention_arguments(fn, desc, names, cache, ws):
    def call(**k):
        a = {n: P for n in names}
        a.update(stride=512, bytes=cache, lse=None, ws_bytes=ws)
        a.update(k)
        return status(fn, desc, *a.values(), None)
    assert ws > 0
    for n in names:
        if n in ("stride", "bytes", "lse", "ws_bytes"):
            continue
        assert call(**{n: None}) == bq.E_ARG, n
        assert call(**{n: P + (1 if n == "out" else 2 if n not in ("cache", "ws") else 128)}) == bq.E_ALIGN, n
    assert call(lse=P + 2) == bq.E_ALIGN
    assert call(stride=511) == bq.E_SHAPE and call(stride=(1 << 40) + 1) == bq.E_SHAPE
    assert call(bytes=cache - 1) == bq.E_CAPACITY and call(ws_bytes=ws - 1) == bq.E_CAPACITY
    assert status(fn, None, *[P] * len(names), None) == bq.E_ARG


@pytest.mark.parametrize("fn,desc,names,cache,ws", attention_calls(), ids=["prompt", "shared"])
def test_attention_outputs_lie_apart(fn, desc, names, cache, ws):
    sep = {n: P + (i << 32) for i, n in enumerate(names)} | dict(stride=512, bytes=cache, lse=P + (1 << 40), ws_bytes=ws)
    order = [n for n in names if n != "lse"]
    for o in ("out", "lse", "ws"):
        for n in order:
            if n in (o, "stride", "bytes", "ws_bytes"):
                continue
            a = sep | {o: sep[n]}
            assert status(fn, desc, *(a[m] for m in names), None) == bq.E_ARG, (o, n)


def test_prompt_tiles_fit_a_launch():
    d = dict(heads=2048, requests=8192, tokens=1, table_stride=8, max_len=8)
    assert size("bitq_prompt_attn_workspace", prompt(kv(kv_heads=2048, page=8, pages=1), **d))[0] == bq.E_SHAPE
    assert size("bitq_prompt_attn_workspace", prompt(kv(kv_heads=1024, page=8, pages=1), **d))[0] == bq.OK


def test_attention_workspaces_stay_bounded():
    """Partial results take 256 MB at most, whatever the sizes; whole prompts need none."""
    for H, G, D in ((1, 1, 64), (8, 8, 128), (32, 4, 256), (1, 128, 128)):
        for T in (1, 5, 100, 4096, 1 << 19):
            for R in (1, 64, 8192):
                if T * H * G > 1 << 26:
                    continue
                e, n = size("bitq_prompt_attn_workspace", prompt(kv(kv_heads=H, head_dim=D, pages=1 << 20), heads=H * G, requests=R,
                                                                 tokens=T, table_stride=1 << 20, max_len=1 << 20))
                assert e == bq.OK and n <= (256 << 20) + 256
                assert n == 0 or T * G * H <= 1 << 17, (H, G, T)
        for R in (1, 64, 8192):
            e, n = size("bitq_shared_attn_workspace", shared(kv(kv_heads=H, head_dim=D, pages=1 << 20), heads=H * G, requests=R,
                                                             table_stride=1 << 20, max_len=1 << 20, groups=1, max_prefix=1 << 19))
            # (one piece of the prefix and one of each request's own tokens at least)
            assert e == bq.OK and n <= max(256 << 20, 2 * R * H * G * (D + 2) * 4) + 256


@pytest.mark.parametrize("bad", [dict(requests=0), dict(requests=8193), dict(page=0), dict(page=24), dict(page=2048), dict(table_stride=0),
                                 dict(table_stride=1 << 27), dict(pool=0), dict(pool=1 << 27), dict(moves=0), dict(moves=(1 << 28) + 1)])
def test_pages_descriptor(bad):
    for fn in ("bitq_kv_pages_size", "bitq_kv_pages_workspace"):
        assert size(fn, pages(**bad))[0] == bq.E_SHAPE
    assert status("bitq_kv_fork", pages(**bad), P, P, P, P, P, P, P, P, BIG, P, BIG, None) == bq.E_SHAPE
    assert status("bitq_kv_compact", pages(**bad), P, P, P, P, P, BIG, P, BIG, None) == bq.E_SHAPE


def test_pages_layout():
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    d = pages(requests=70, moves=100)
    assert bq.kv_pages_size(d) == 256 + up(280) + 2 * up(400)
    import torch
    v = bq.kv_pages_views(d, torch.zeros(bq.kv_pages_size(d), dtype=torch.uint8))
    assert {k: x.numel() for k, x in v.items()} == dict(state=4, len=70, frm=100, to=100)
    assert v["to"].storage_offset() * 4 == 256 + up(280) + up(400)


@pytest.mark.parametrize("fn", ["bitq_kv_fork", "bitq_kv_compact"])
def test_pages_arguments(fn):
    d = pages()
    names = ["src", "keep", "len", "ring", "state", "table", "out"] if fn == "bitq_kv_fork" else ["len", "table", "out", "ring"]
    res, ws = bq.kv_pages_size(d), bq.kv_pages_workspace(d)
    base = {n: P + (i << 16) for i, n in enumerate(names)} | dict(result=P + (8 << 16), rb=res, ws=P + (9 << 16), wb=ws)

    def call(desc=d, **k):
        return status(fn, desc, *(base | k).values(), None)
    for n in names + ["result", "ws"]:
        assert call(**{n: None}) == bq.E_ARG, n
        assert call(**{n: base[n] + (2 if n in names else 64)}) == bq.E_ALIGN, n
    assert call(rb=res - 1) == bq.E_CAPACITY and call(wb=ws - 1) == bq.E_CAPACITY
    outs = [n for n in ("ring", "out", "result", "ws")]
    for o in outs:                                   # no output over an input or another output
        for n in names + ["result", "ws"]:
            if n != o:
                assert call(**{n: base[o]}) == bq.E_ARG, (o, n)
    assert call(out=base["table"] + 4 * 31) == bq.E_ARG
    assert status(fn, None, *base.values(), None) == bq.E_ARG
    if fn == "bitq_kv_fork":
        assert call(desc=pages(moves=3)) == bq.E_SHAPE


def test_copy_arguments():
    c = bq.kv_cache_size(kv())
    far = P + (1 << 30)

    def call(desc=kv(), frm=far, to=far + 4096, moves=5, cache=P, n=c):
        return status("bitq_kv_copy", desc, frm, to, moves, cache, n, None)
    for bad, want in CACHE:
        assert call(kv(**bad)) == want
    assert call(None) == bq.E_ARG and call(frm=None) == bq.E_ARG and call(to=None) == bq.E_ARG and call(cache=None) == bq.E_ARG
    assert call(frm=far + 2) == bq.E_ALIGN and call(to=far + 1) == bq.E_ALIGN and call(cache=P + 128) == bq.E_ALIGN
    assert call(moves=-1) == bq.E_SHAPE and call(moves=(1 << 28) + 1) == bq.E_SHAPE and call(n=c - 1) == bq.E_CAPACITY
    assert call(frm=P + c - 4) == bq.E_ARG and call(to=P + 256) == bq.E_ARG


@pytest.mark.parametrize("bad,want", [
    (dict(tokens=0), bq.E_SHAPE), (dict(tokens=(1 << 24) + 1), bq.E_SHAPE), (dict(q_heads=-1), bq.E_SHAPE), (dict(k_heads=16385), bq.E_SHAPE),
    (dict(q_heads=0, k_heads=0), bq.E_SHAPE), (dict(tokens=1 << 24, q_heads=16), bq.E_SHAPE), (dict(head_dim=0), bq.E_SHAPE),
    (dict(head_dim=257), bq.E_SHAPE), (dict(rot=-2), bq.E_SHAPE), (dict(rot=3), bq.E_SHAPE), (dict(rot=66), bq.E_SHAPE),
    (dict(layout=2), bq.E_ARG), (dict(x_dtype=2), bq.E_ARG), (dict(out_dtype=16), bq.E_ARG), (dict(w_dtype=3), bq.E_ARG),
    (dict(eps=-1.0), bq.E_ARG), (dict(eps=float("nan")), bq.E_ARG), (dict(mscale=float("inf")), bq.E_ARG)])
def test_rope_descriptor(bad, want):
    assert status("bitq_qk_rope", rope(**bad), P, 1 << 20, P, 1 << 20, P, P, P, P, P, 1 << 20, P, 1 << 20, None) == want


def test_rope_arguments():
    names = ["q", "qs", "k", "ks", "qw", "kw", "table", "pos", "qo", "qos", "ko", "kos"]
    base = {n: P + (i << 20) for i, n in enumerate(names)} | dict(qs=256, ks=128, qos=256, kos=128)

    def call(desc=None, **k):
        return status("bitq_qk_rope", desc or rope(), *(base | k).values(), None)
    for n in ("q", "k", "table", "pos", "qo", "ko"):
        assert call(**{n: None}) == bq.E_ARG, n
    for n, off in (("q", 2), ("k", 1), ("qw", 2), ("kw", 1), ("table", 4), ("pos", 2), ("qo", 1), ("ko", 1)):
        assert call(**{n: base[n] + off}) == bq.E_ALIGN, n
    for n, least in (("qs", 256), ("ks", 128), ("qos", 256), ("kos", 128)):
        assert call(**{n: least - 1}) == bq.E_SHAPE and call(**{n: (1 << 36) + 1}) == bq.E_SHAPE
    # outputs over what is read, or over each other
    assert call(qo=base["q"]) == bq.E_ARG                                    # (another type)
    assert call(qo=base["k"]) == bq.E_ARG and call(ko=base["q"] + 64) == bq.E_ARG and call(ko=base["qo"] + 512) == bq.E_ARG
    for n in ("qw", "kw", "table", "pos"):
        assert call(qo=base[n]) == bq.E_ARG, n
    same = rope(out_dtype=0)
    assert call(same, qo=base["q"], qos=260) == bq.E_ARG                     # in place with another stride
    assert call(same, qo=base["q"] + 1024) == bq.E_ARG                       # a row further on
    assert status("bitq_qk_rope", None, *base.values(), None) == bq.E_ARG


def test_rope_takes_rows_side_by_side():
    """q, k and their outputs may be columns of one buffer; what is left is the device check."""
    row = 8 * 64
    d = rope(out_dtype=0)
    ok = (bq.E_DEVICE, bq.E_UNSUPPORTED)
    a = dict(q=P, qs=row, k=P + 4 * 4 * 64, ks=row, qw=None, kw=None, table=1 << 30, pos=1 << 31, qo=P, qos=row, ko=P + 4 * 4 * 64, kos=row)
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses")
    assert status("bitq_qk_rope", d, *a.values(), None) in ok
    a.update(ko=P + 4 * 6 * 64)                                              # k's output where the values are
    assert status("bitq_qk_rope", d, *a.values(), None) in ok
    a.update(ko=P + 4 * 3 * 64)                                              # over the last head of q
    assert status("bitq_qk_rope", d, *a.values(), None) == bq.E_ARG
    a.update(ko=P + 4 * 7 * 64)                                              # reaches into the next token's row of q
    assert status("bitq_qk_rope", d, *a.values(), None) == bq.E_ARG
