"""Refusals, sizes and layouts of the operators of include/bitq_lm.h (no GPU needed)."""
import ctypes

import pytest

import bit_plane_gemv_amd as bq

P = 1 << 20        # fake, well-aligned addresses: every call here fails before any device call
BIG = 1 << 60


def status(fn, *args):
    return getattr(bq._lib, fn)(*args)


def kv(**k):
    d = dict(kv_heads=4, head_dim=64, page=16, pages=10, dtype=bq.KV_BF16)
    d.update(k)
    return bq.KvDesc(*d.values())


def plan(**k):
    d = dict(requests=4, page=16, table_stride=8, ring=30, tokens=64)
    d.update(k)
    return bq.KvPlanDesc(*d.values())


def attn(cache=None, **k):
    d = dict(heads=8, requests=3, table_stride=8, max_len=100, window=0, q_dtype=bq.DT_F32, out_dtype=bq.DT_BF16, scale=0.1)
    d.update(k)
    return bq.AttnDesc(cache or kv(), *d.values())


def norm(**k):
    d = dict(rows=3, width=64, u_dtype=0, r_dtype=0, w_dtype=0, out_dtype=0, u_stride=64, r_stride=64, ro_stride=64,
             h_stride=64, gate_stride=0, res_scale=1.0, branch_scale=1.0, eps_post=1e-5, eps_pre=1e-5)
    d.update(k)
    return bq.NormDesc(*d.values())


def w8(**k):
    d = dict(M=4, N=32, K=64, y_dtype=bq.DT_F32, lda=64, ldw=64, ldy=32, flags=0)
    d.update(k)
    return bq.W8A8Desc(*d.values())


@pytest.mark.parametrize("bad,want", [
    (dict(dtype=2), bq.E_ARG), (dict(kv_heads=0), bq.E_SHAPE), (dict(kv_heads=1025), bq.E_SHAPE), (dict(head_dim=0), bq.E_SHAPE),
    (dict(head_dim=257), bq.E_SHAPE), (dict(page=12), bq.E_SHAPE), (dict(page=4), bq.E_SHAPE), (dict(page=2048), bq.E_SHAPE),
    (dict(page=-16), bq.E_SHAPE), (dict(pages=0), bq.E_SHAPE), (dict(pages=1 << 27), bq.E_SHAPE),
])
def test_cache_geometry(bad, want):
    n = ctypes.c_size_t(0)
    assert status("bitq_kv_cache_size", kv(**bad), ctypes.byref(n)) == want
    assert status("bitq_kv_write", kv(**bad), P, P, 0, 4096, 4096, P, 1, P, BIG, None) == want
    assert status("bitq_paged_attn_workspace", attn(kv(**bad)), ctypes.byref(n)) == want


def test_cache_size_matches_the_documented_layout():
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    for H, D, page, pages, dt in [(1, 1, 8, 1, 0), (4, 64, 16, 10, 0), (3, 80, 32, 7, 1), (5, 255, 8, 3, 1)]:
        Dp, e = (D + 31) // 32 * 32, 2 if dt == bq.KV_BF16 else 1
        want = 2 * up(pages * H * page * Dp * e) + (2 * up(pages * H * page * 4) if dt == bq.KV_INT8 else 0)
        assert bq.kv_cache_size(bq.kvdesc(H, D, page, pages, dt)) == want
    assert status("bitq_kv_cache_size", None, None) == bq.E_ARG
    d = bq.kv_plan_desc(5, 16, 4, 9, 70)
    assert bq.kv_plan_size(d) == 256 + up(20) + up(24) + 3 * up(280)


@pytest.mark.parametrize("bad", [dict(requests=0), dict(requests=8193), dict(page=0), dict(page=24), dict(table_stride=0),
                                 dict(table_stride=1 << 27), dict(ring=0), dict(ring=1 << 27), dict(tokens=0),
                                 dict(tokens=(1 << 24) + 1)])
def test_plan_descriptor(bad):
    n = ctypes.c_size_t(0)
    assert status("bitq_kv_plan_size", plan(**bad), ctypes.byref(n)) == bq.E_SHAPE
    assert status("bitq_kv_plan", plan(**bad), P, P, P, P, P, P, BIG, None) == bq.E_SHAPE


def test_plan_arguments():
    n = bq.kv_plan_size(plan())
    far = P + (1 << 22)
    ok = [far, far + 4096, far + 8192, far + 12288, far + 16384]
    for i in range(5):
        a = list(ok)
        a[i] = None
        assert status("bitq_kv_plan", plan(), *a, P, n, None) == bq.E_ARG
        a[i] = ok[i] + 2
        assert status("bitq_kv_plan", plan(), *a, P, n, None) == bq.E_ALIGN
    assert status("bitq_kv_plan", plan(), *ok, None, n, None) == bq.E_ARG
    assert status("bitq_kv_plan", plan(), *ok, P + 64, n, None) == bq.E_ALIGN
    assert status("bitq_kv_plan", plan(), *ok, P, n - 1, None) == bq.E_CAPACITY
    assert status("bitq_kv_plan", None, *ok, P, n, None) == bq.E_ARG
    for i in (0, 1, 3):                              # lengths or state inside the plan buffer that is written
        a = list(ok)
        a[i] = P + 256
        assert status("bitq_kv_plan", plan(), *a, P, n, None) == bq.E_ARG


def test_write_arguments():
    c = bq.kv_cache_size(kv())
    good = (P, P, bq.DT_F32, 256, 256, P, 3, P, c, None)

    def call(**k):
        names = ["k", "v", "dt", "ks", "vs", "slots", "tokens", "cache", "bytes", "stream"]
        a = dict(zip(names, good))
        a.update(k)
        return status("bitq_kv_write", kv(), *a.values())
    for name in ("k", "v", "slots", "cache"):
        assert call(**{name: None}) == bq.E_ARG
    assert call(dt=bq.DT_ACT) == bq.E_ARG
    assert call(ks=255) == bq.E_SHAPE and call(vs=255) == bq.E_SHAPE and call(ks=1 << 41) == bq.E_SHAPE
    assert call(tokens=-1) == bq.E_SHAPE and call(tokens=(1 << 24) + 1) == bq.E_SHAPE
    assert call(k=P + 2) == bq.E_ALIGN and call(v=P + 1, dt=bq.DT_BF16) == bq.E_ALIGN and call(slots=P + 2) == bq.E_ALIGN
    assert call(cache=P + 128) == bq.E_ALIGN and call(bytes=c - 1) == bq.E_CAPACITY
    assert status("bitq_kv_write", None, *good) == bq.E_ARG


@pytest.mark.parametrize("bad,want", [
    (dict(heads=0), bq.E_SHAPE), (dict(heads=6), bq.E_SHAPE), (dict(heads=16388), bq.E_SHAPE), (dict(requests=0), bq.E_SHAPE),
    (dict(requests=65536), bq.E_SHAPE), (dict(table_stride=0), bq.E_SHAPE), (dict(max_len=0), bq.E_SHAPE),
    (dict(max_len=129), bq.E_SHAPE), (dict(window=-1), bq.E_SHAPE), (dict(q_dtype=2), bq.E_ARG), (dict(out_dtype=16), bq.E_ARG),
    (dict(scale=float("nan")), bq.E_ARG), (dict(scale=float("inf")), bq.E_ARG), (dict(requests=65535, heads=256), bq.E_SHAPE),
])
def test_attention_descriptor(bad, want):
    n = ctypes.c_size_t(0)
    assert status("bitq_paged_attn_workspace", attn(**bad), ctypes.byref(n)) == want
    assert status("bitq_paged_attn", attn(**bad), P, 1 << 20, P, BIG, P, P, P, None, P, BIG, None) == want


def test_attention_arguments():
    d = attn(table_stride=100, max_len=1500)
    c, w = bq.kv_cache_size(kv()), bq.paged_attn_workspace(d)
    assert w > 0 and bq.paged_attn_workspace(attn(max_len=100)) == 0     # one pass of a workgroup needs no workspace
    good = dict(q=P, qs=512, cache=P, cb=c, table=P, lens=P, out=P, lse=P, ws=P, wb=w, st=None)

    def call(**k):
        a = dict(good)
        a.update(k)
        return status("bitq_paged_attn", d, *a.values())
    for name in ("q", "cache", "table", "lens", "out", "ws"):
        assert call(**{name: None}) == bq.E_ARG
    assert call(qs=511) == bq.E_SHAPE
    for name, by in (("q", 2), ("table", 2), ("lens", 2), ("lse", 2), ("out", 1), ("cache", 128), ("ws", 128)):
        assert call(**{name: P + by}) == bq.E_ALIGN, name
    assert call(cb=c - 1) == bq.E_CAPACITY and call(wb=w - 1) == bq.E_CAPACITY
    assert status("bitq_paged_attn_workspace", d, None) == bq.E_ARG
    assert status("bitq_paged_attn_workspace", None, None) == bq.E_ARG


@pytest.mark.parametrize("bad,want", [
    (dict(rows=0), bq.E_SHAPE), (dict(rows=(1 << 24) + 1), bq.E_SHAPE), (dict(width=0), bq.E_SHAPE), (dict(width=32769), bq.E_SHAPE),
    (dict(u_dtype=16), bq.E_ARG), (dict(r_dtype=2), bq.E_ARG), (dict(w_dtype=3), bq.E_ARG), (dict(out_dtype=2), bq.E_ARG),
    (dict(u_stride=63), bq.E_SHAPE), (dict(r_stride=63), bq.E_SHAPE), (dict(ro_stride=63), bq.E_SHAPE), (dict(h_stride=63), bq.E_SHAPE),
    (dict(gate_stride=63), bq.E_SHAPE), (dict(gate_stride=-64), bq.E_SHAPE), (dict(u_stride=1 << 41), bq.E_SHAPE),
    (dict(res_scale=float("nan")), bq.E_ARG), (dict(branch_scale=float("inf")), bq.E_ARG), (dict(eps_post=-1.0), bq.E_ARG),
    (dict(eps_pre=float("nan")), bq.E_ARG),
])
def test_norm_descriptor(bad, want):
    q = [P + 4096 * i for i in range(8)]
    assert status("bitq_block_norm", norm(**bad), q[0], q[1], q[2], q[3], q[4], q[5], q[6], None, None) == want


def test_norm_arguments():
    names = ["u", "r", "post", "gate", "pre", "ro", "h", "d"]
    good = {n: P + 4096 * i for i, n in enumerate(names)} | dict(d=None)

    def call(desc=None, **k):
        a = dict(good)
        a.update(k)
        return status("bitq_block_norm", desc or norm(), *a.values(), None)
    assert call(u=None) == bq.E_ARG and call(h=None) == bq.E_ARG
    assert call(d=P) == bq.E_ARG and call(norm(out_dtype=bq.DT_ROW8)) == bq.E_ARG      # scales belong to int8 rows
    assert call(h=good["u"]) == bq.E_ARG and call(h=good["r"]) == bq.E_ARG and call(h=good["ro"]) == bq.E_ARG
    assert call(ro=good["u"]) == bq.E_ARG
    assert call(norm(ro_stride=72), ro=good["r"]) == bq.E_SHAPE
    for n in ("u", "r", "post", "gate", "pre", "ro", "h"):
        assert call(**{n: good[n] + 2}) == bq.E_ALIGN, n
    assert call(norm(out_dtype=bq.DT_ROW8), d=P + 2) == bq.E_ALIGN


@pytest.mark.parametrize("bad,want", [
    (dict(M=0), bq.E_SHAPE), (dict(N=0), bq.E_SHAPE), (dict(K=0), bq.E_SHAPE), (dict(K=24), bq.E_SHAPE),
    (dict(K=131072, lda=131072, ldw=131072), bq.E_SHAPE), (dict(lda=48), bq.E_SHAPE), (dict(ldw=72), bq.E_SHAPE),
    (dict(lda=1 << 23), bq.E_SHAPE), (dict(ldy=31), bq.E_SHAPE), (dict(M=1 << 20, N=1 << 20, ldy=1 << 20), bq.E_SHAPE),
    (dict(y_dtype=2), bq.E_ARG), (dict(flags=2), bq.E_ARG), (dict(flags=1, y_dtype=bq.DT_BF16), bq.E_ARG),
])
def test_product_descriptor(bad, want):
    n = ctypes.c_size_t(0)
    assert status("bitq_w8a8_workspace", w8(**bad), ctypes.byref(n)) == want
    assert status("bitq_gemm_w8a8", w8(**bad), P, P, P, P, P, P, BIG, None) == want


def test_product_arguments():
    def call(desc, a=P, sa=P, w=P, sw=P, y=P, ws=P, wb=BIG):
        return status("bitq_gemm_w8a8", desc, a, sa, w, sw, y, ws, wb, None)
    for n in ("a", "w", "y", "sa", "sw"):
        assert call(w8(), **{n: None}) == bq.E_ARG
    assert call(w8(), a=P + 8) == bq.E_ALIGN and call(w8(), w=P + 8) == bq.E_ALIGN
    assert call(w8(), y=P + 2) == bq.E_ALIGN and call(w8(), sa=P + 2) == bq.E_ALIGN and call(w8(), sw=P + 1) == bq.E_ALIGN
    d = w8(M=64, N=512, K=8192 + 6144, lda=14336, ldw=14336, ldy=512)
    e = w8(M=100, N=512, K=14336, lda=14336, ldw=14336, ldy=512)
    need = bq.w8a8_workspace(e)
    assert need > 0 and bq.w8a8_workspace(w8()) == 0 and bq.w8a8_workspace(d) >= 0
    assert call(e, ws=None) == bq.E_ARG and call(e, ws=P + 16) == bq.E_ALIGN and call(e, wb=need - 1) == bq.E_CAPACITY


def test_errors_say_what_is_wrong():
    with pytest.raises(bq.BitqError) as e:
        bq.kv_cache_size(bq.kvdesc(4, 300, 16, 1))
    assert e.value.status == bq.E_SHAPE and "head_dim=300" in bq.last_error()
    with pytest.raises(bq.BitqError):
        bq.w8a8_workspace(bq.w8a8_desc(4, 32, 40))
    assert "multiple of 16" in bq.last_error()
