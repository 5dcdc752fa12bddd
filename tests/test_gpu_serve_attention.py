"""prompt_attn and shared_attn against 64-bit references, at the sizes and masks where they can go wrong."""
import numpy as np
import pytest
import torch

import bit_plane_gemv_amd as bq
import lm_reference as lm
import serve_reference as ref
from gpuhelp import say

pytestmark = pytest.mark.gpu
DT = {"f32": (bq.DT_F32, torch.float32), "bf16": (bq.DT_BF16, torch.bfloat16)}


def upload(sections, kv):
    cache = torch.zeros(bq.kv_cache_size(kv), dtype=torch.uint8, device="cuda")
    v = bq.kv_cache_views(kv, cache)
    for name, x in zip(("K", "V", "ks", "vs"), sections):
        if x is not None:
            v[name].copy_(x)
    return cache


def tables(lens, page, stride, rng, spare=2):
    """Rows of random pages for requests of the given lengths; entries past them name pages that nobody holds."""
    held = [lm.ceil_div(max(n, 0), page) for n in lens]
    order = rng.permutation(sum(held) + spare)
    t = np.full((len(lens), stride), order[-1] if spare else 0, dtype=np.int32)
    at = 0
    for r, n in enumerate(held):
        t[r, :n] = order[at:at + n]
        at += n
    return t, sum(held) + spare


def close(got, want, tol, name):
    got = got.double().cpu().numpy()
    same = (got == want) | (np.abs(got - want) <= tol)
    assert same.all(), f"{name}: {np.argwhere(~same)[:5].tolist()}: {got[~same][:5]} for {want[~same][:5]}, tolerance {tol[~same][:5]}"


def run_prompt(new, lens, H, G, D, page, kind, dt, window=0, sinks=0, extra_rows=0, seed=0, scale=None, odd_stride=False,
               max_len=None, odt=None, table=None, pool=None, poison=None, stream=None):
    rng = np.random.default_rng(seed)
    R, A, T = len(new), H * G, sum(new) + extra_rows
    max_len = max(1, max(lens)) if max_len is None else max_len
    stride = lm.ceil_div(max_len, page) + 1
    if table is None:
        table, pool = tables(lens, page, stride, rng)
    sections = lm.cache_sections(pool, H, page, D, kind == "int8", rng)
    if poison:
        poison(sections, table)
    kv = bq.kvdesc(H, D, page, pool, bq.KV_INT8 if kind == "int8" else bq.KV_BF16)
    cache = upload(sections, kv)
    code, t = DT[dt]
    ocode, ot = DT[odt or dt]
    q = torch.from_numpy(rng.standard_normal((T, A, D)).astype(np.float32)).to(t)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    scale = D ** -0.5 if scale is None else scale
    wide = torch.zeros(T, A * D + (3 if odd_stride else 0), dtype=t, device="cuda")
    wide[:, :A * D] = q.view(T, A * D).cuda()
    d = bq.prompt_desc(kv, A, R, T, stride, max_len, window=window, sinks=sinks, q_dtype=code, out_dtype=ocode, scale=scale)
    ws = torch.full((max(1, bq.prompt_attn_workspace(d)),), 0x7F, dtype=torch.uint8, device="cuda")
    out = torch.full((T, A, D), 7.0, dtype=ot, device="cuda")
    lse = torch.full((T, A), 7.0, device="cuda")
    say("prompt", new, lens, H, G, D, page, kind, dt, odt, window, sinks, "workspace", ws.numel())
    bq.prompt_attn(d, wide, cache, torch.from_numpy(table).cuda(), torch.from_numpy(start).cuda(),
                   torch.tensor(lens, dtype=torch.int32, device="cuda"), out, ws, lse=lse, q_stride=wide.shape[1])
    torch.cuda.synchronize()
    terms = 3 if ot is torch.float32 or t is torch.float32 else 2
    want = ref.prompt(q.double().numpy(), sections, table, start, lens, page, np.float32(scale), window, sinks, max_len, terms)
    return out, lse, want, ot


def check_prompt(*a, **k):
    out, lse, (want, wl, tol, ltol), ot = run_prompt(*a, **k)
    left = np.isnan(wl)
    assert (out.cpu()[torch.from_numpy(left)] == 7).all() and (lse.cpu()[torch.from_numpy(left)] == 7).all(), "rows of no request"
    want, wl = np.where(np.isnan(want), 7, want), np.where(left, 7, wl)
    close(out, want, tol + ref.half_step(ot) * (np.abs(want) + tol), "out")
    close(lse, wl, ltol, "lse")


CACHES = ["bf16", "int8"]


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 8, 31, 64, 80, 96, 128, 144, 192, 200, 256])
def test_prompt_head_dimensions(D, dt, kind):
    check_prompt([70, 1, 37], [70, 130, 95], 2, 2, D, 16, kind, dt, seed=D)


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [32, 80, 128, 160, 224, 256])
def test_prompt_single_tokens(D, dt, kind):
    check_prompt([1] * 5, [1, 33, 200, 64, 515], 2, 4, D, 8, kind, dt, seed=D)


@pytest.mark.parametrize("page", [8, 16, 64, 1024])
@pytest.mark.parametrize("G", [1, 3, 7, 16, 20, 40])
def test_prompt_groups_and_pages(G, page):
    check_prompt([9, 3], [300, 77], 2, G, 64, page, "bf16", "bf16", seed=G)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (64, 4), (100, 33), (33, 64), (400, 3), (7, 1000), (128, 128)])
@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("new,lens", [([150, 20], [350, 341]), ([1, 1, 1], [350, 9, 101])])
def test_prompt_windows(new, lens, kind, window, sinks):
    check_prompt(new, lens, 1, 4, 64, 16, kind, "f32", window=window, sinks=sinks, seed=window)
    check_prompt(new, lens, 1, 4, 64, 16, kind, "bf16", window=window, sinks=sinks, seed=window)


def test_prompt_empty_requests_and_rows_of_none():
    check_prompt([0, 5, 0, 0, 40, 0], [0, 5, 17, 0, 40, 3], 2, 2, 64, 16, "bf16", "bf16", extra_rows=9)
    check_prompt([0, 1, 0, 1], [4, 7, 0, 300], 2, 2, 64, 16, "bf16", "bf16", extra_rows=2)
    check_prompt([3, 0], [3, 0], 1, 1, 64, 8, "int8", "f32", extra_rows=64)


def test_prompt_rows_before_position_zero_see_nothing():
    check_prompt([6, 4, 50], [2, 0, 20], 2, 3, 64, 16, "bf16", "f32")
    check_prompt([6, 4, 50], [2, 0, 20], 2, 3, 64, 16, "int8", "bf16", window=3, sinks=1)


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 9, 3)])
def test_prompt_widest_windows(window, sinks):
    """Also for rows before position 0 in a tile with others: a window as wide as its type sees all that came before."""
    check_prompt([40, 9, 5], [17, 100, 3], 2, 2, 64, 16, "bf16", "f32", window=window, sinks=sinks)


def test_prompt_many_requests():
    rng = np.random.default_rng(5)
    new = rng.integers(0, 3, 150).tolist()
    check_prompt(new, [n + int(rng.integers(0, 40)) for n in new], 1, 2, 32, 8, "bf16", "bf16")


def test_prompt_more_requests_than_a_wave_searches_at_once():
    R = 4500
    new = [1 if r % 300 == 7 or r == R - 1 else 0 for r in range(R)]
    check_prompt(new, [5 if n else 0 for n in new], 1, 1, 32, 8, "bf16", "f32")


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_prompt_split_over_workgroups(dt, kind):
    check_prompt([1], [3000], 1, 8, 128, 32, kind, dt)
    check_prompt([5], [3000], 1, 8, 128, 32, kind, dt)
    check_prompt([60, 2], [1500, 2900], 1, 4, 64, 32, kind, dt, window=1000, sinks=40)


def test_prompt_rows_with_odd_strides_and_a_mix_of_types():
    check_prompt([20, 3], [50, 33], 2, 2, 64, 16, "bf16", "bf16", odd_stride=True)
    check_prompt([20, 3], [50, 33], 2, 2, 64, 16, "bf16", "f32", odd_stride=True)
    check_prompt([20, 3], [50, 33], 2, 2, 64, 16, "int8", "bf16", odt="f32")
    check_prompt([20, 3], [50, 33], 2, 2, 72, 16, "bf16", "f32", odt="bf16")


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0, 1e-30])
def test_prompt_scales(scale):
    check_prompt([20, 1], [50, 90], 2, 2, 64, 16, "bf16", "f32", scale=scale)


def test_prompt_lengths_beyond_the_longest_count_as_it():
    rng = np.random.default_rng(3)
    table = rng.permutation(9)[:8].reshape(2, 4).astype(np.int32)
    check_prompt([4, 2], [1000, -5], 1, 2, 64, 16, "bf16", "f32", max_len=40, table=table, pool=9)


def test_prompt_pages_outside_the_pool_read_page_zero():
    table = np.array([[1, 99, -1, 2]], dtype=np.int32)
    out, lse, _, _ = run_prompt([4], [48], 1, 2, 64, 16, "bf16", "f32", max_len=48, table=table, pool=3)
    same, lse2, (want, wl, tol, ltol), ot = run_prompt([4], [48], 1, 2, 64, 16, "bf16", "f32", max_len=48,
                                                       table=np.array([[1, 0, 0, 2]], dtype=np.int32), pool=3)
    assert torch.equal(out, same) and torch.equal(lse, lse2)
    close(out, want, tol + ref.half_step(ot) * (np.abs(want) + tol), "out")


def poison_outside(lens, page):
    """Infinities and NaN in every slot that no request holds."""
    def f(sections, table):
        K, V, ks, vs = sections
        held = {}
        for r, n in enumerate(lens):
            for t in range(n):
                held.setdefault(int(table[r, t // page]), set()).add(t % page)
        for p in range(K.shape[0]):
            for o in range(page):
                if o in held.get(p, ()):
                    continue
                bad = [float("nan"), float("inf"), -float("inf")][(p + o) % 3]
                if ks is None:
                    K[p, :, o], V[p, :, o // 8, :, o % 8] = bad, bad
                else:
                    K[p, :, o], V[p, :, o // 8, :, o % 8] = 127, 127
                    ks[p, :, o], vs[p, :, o] = bad, bad
    return f


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("new,lens,G", [([37, 3], [61, 9], 2), ([1, 1], [61, 9], 4), ([90], [90], 4)])
def test_prompt_ignores_what_lies_outside(new, lens, G, dt, kind):
    check_prompt(new, lens, 2, G, 64, 16, kind, dt, poison=poison_outside(lens, 16))
    check_prompt(new, lens, 2, G, 64, 16, kind, dt, window=20, sinks=2, poison=poison_outside(lens, 16))


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 8])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_prompt_later_tokens_have_no_effect_whatever_they_hold(bad, G, dt, kind):
    """Token 70 of 90 holds what is not finite: rows before it are as without it, the others NaN where they see it."""
    def poison(sections, table):
        K, V, ks, vs = sections
        p, o = int(table[0, 70 // 16]), 70 % 16
        if ks is None:
            K[p, :, o, 3] = bad
            V[p, :, o // 8, 5, o % 8] = bad
        else:
            ks[p, :, o] = bad
            vs[p, :, o] = bad
    for window, sinks in ((0, 0), (10, 2)):
        a = dict(window=window, sinks=sinks)
        out, lse, _, _ = run_prompt([90], [90], 1, G, 64, 16, kind, dt, poison=poison, **a)
        clean, lclean, _, _ = run_prompt([90], [90], 1, G, 64, 16, kind, dt, **a)
        sees = np.array([70 in ref.visible(x, window, sinks) for x in range(90)])
        assert torch.equal(out[~sees], clean[~sees]) and torch.equal(lse[~sees], lclean[~sees])
        if kind == "int8" or np.isnan(bad):
            assert out[sees].isnan().all()           # (an infinite key may also weigh 0 or take all the weight)
        else:
            assert not out[sees][..., 5].isfinite().any()


def test_prompt_value_that_is_not_finite_reaches_its_element_alone():
    def poison(sections, table):
        sections[1][int(table[0, 70 // 16]), :, 70 % 16 // 8, 5, 70 % 8] = float("nan")
    for new in (90, 1):
        out, _, (want, _, tol, _), ot = run_prompt([new], [90], 1, 4, 64, 16, "bf16", "f32", poison=poison)
        rows = [i for i in range(new) if 90 - new + i >= 70]
        assert out[rows][..., 5].isnan().all()
        rest = [e for e in range(64) if e != 5]
        close(out[..., rest], want[..., rest], tol[..., rest] + 2.0 ** -24 * np.abs(want[..., rest]), "out")


def test_prompt_long_cache_past_32_bits():
    """A pool of over 2^32 bytes: the request's pages lie at its end."""
    H, D, page, G = 8, 128, 64, 4
    pool = (5 << 30) // (2 * H * page * D * 2)
    kv = bq.kvdesc(H, D, page, pool)
    cache = torch.zeros(bq.kv_cache_size(kv), dtype=torch.uint8, device="cuda")
    v = bq.kv_cache_views(kv, cache)
    rng = np.random.default_rng(1)
    sections = lm.cache_sections(4, H, page, D, False, rng)
    ids = torch.tensor([pool - 1, pool - 3, pool // 2, pool - 2])
    for name, x in zip(("K", "V"), sections):
        v[name][ids.cuda()] = x.cuda()
    for new, t in ((30, "bf16"), (1, "f32")):
        q = torch.from_numpy(rng.standard_normal((new, H * G, D)).astype(np.float32)).to(DT[t][1])
        d = bq.prompt_desc(kv, H * G, 1, new, 4, 256, q_dtype=DT[t][0], out_dtype=bq.DT_F32)
        ws = torch.empty(max(1, bq.prompt_attn_workspace(d)), dtype=torch.uint8, device="cuda")
        out = torch.empty(new, H * G, D, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        bq.prompt_attn(d, q.cuda(), cache, i32([ids.tolist()]), i32([0, new]), i32([250]), out, ws)
        want, _, tol, _ = ref.prompt(q.double().numpy(), sections, np.arange(4)[None], [0, new], [250], page,
                                     np.float32(D ** -0.5), 0, 0, 256, 3)
        close(out, want, tol + 2.0 ** -24 * np.abs(want), "out")


# ------------------------------------------------------------------ shared
def run_shared(lens, start, prefix, H, G, D, page, kind, dt, seed=0, common=True, max_prefix=None, max_len=None, odt=None,
               poison=None):
    rng = np.random.default_rng(seed)
    R, A = len(lens), H * G
    max_len = max(1, max(lens)) if max_len is None else max_len
    stride = lm.ceil_div(max(max_len, 1), page) + 1
    table, pool = tables([min(max(n, 0), max_len) for n in lens], page, stride, rng)
    of = ref.groups_of(start, R)
    for r in range(R):                               # whole pages of the prefix are the first request's
        if common and of[r] >= 0:
            whole = min(prefix[of[r]], max(lens[r], 0)) // page
            table[r, :whole] = table[max(0, start[of[r]]), :whole]
    sections = lm.cache_sections(pool, H, page, D, kind == "int8", rng)
    if poison:
        poison(sections, table)
    kv = bq.kvdesc(H, D, page, pool, bq.KV_INT8 if kind == "int8" else bq.KV_BF16)
    cache = upload(sections, kv)
    code, t = DT[dt]
    ocode, ot = DT[odt or dt]
    q = torch.from_numpy(rng.standard_normal((R, A, D)).astype(np.float32)).to(t)
    max_prefix = min(max_len, max(1, max(prefix))) if max_prefix is None else max_prefix
    d = bq.shared_desc(bq.attn_desc(kv, A, R, stride, max_len, q_dtype=code, out_dtype=ocode), len(prefix), max_prefix)
    ws = torch.full((bq.shared_attn_workspace(d),), 0x7F, dtype=torch.uint8, device="cuda")
    out, lse = torch.full((R, A, D), 7.0, dtype=ot, device="cuda"), torch.full((R, A), 7.0, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    say("shared", lens, start, prefix, H, G, D, page, kind, dt, odt, "workspace", ws.numel())
    bq.shared_attn(d, q.cuda(), cache, torch.from_numpy(table).cuda(), i32(lens), i32(start), i32(prefix), out, ws, lse=lse)
    torch.cuda.synchronize()
    terms = 3 if ot is torch.float32 or t is torch.float32 else 2
    return out, lse, ref.shared(q.double().numpy(), sections, table, lens, start, prefix, page, np.float32(D ** -0.5), max_len,
                                max_prefix, terms), ot


def check_shared(*a, **k):
    out, lse, (want, wl, tol, ltol), ot = run_shared(*a, **k)
    close(out, want, tol + ref.half_step(ot) * (np.abs(want) + tol), "out")
    close(lse, wl, ltol, "lse")


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 40, 64, 96, 128, 160, 192, 224, 256])
def test_shared_head_dimensions(D, dt, kind):
    check_shared([130, 101, 160, 101, 90, 300], [0, 4, 6], [100, 77], 2, 3, D, 16, kind, dt, seed=D)


@pytest.mark.parametrize("kind", CACHES)
def test_shared_many_rows_of_a_group(kind):
    check_shared([300 + 3 * r for r in range(40)], [0, 40], [290], 1, 5, 64, 16, kind, "bf16")
    check_shared([70 + r for r in range(9)], [0, 9], [64], 1, 40, 64, 64, kind, "f32")


def test_shared_prefixes_that_are_empty_whole_or_longer_than_a_request():
    check_shared([50, 50, 20, 64, 64], [0, 3, 5], [0, 64], 2, 2, 64, 16, "bf16", "f32")
    check_shared([50, 10, 0, 49, 50], [0, 5], [50], 2, 2, 64, 16, "int8", "bf16")
    check_shared([0, 10, 30], [0, 3], [20], 2, 2, 64, 16, "bf16", "f32")           # its first request holds nothing


def test_shared_requests_in_no_group_and_groups_without_requests():
    check_shared([90, 40, 130, 77, 60, 200], [1, 1, 3, 3, 5], [50, 30, 70, 60], 2, 2, 64, 16, "bf16", "f32")
    check_shared([90, 40], [0, 0, 0], [50, 30], 2, 2, 64, 16, "bf16", "bf16")
    check_shared([90, 40], [2, 2], [50], 2, 2, 64, 16, "bf16", "bf16")


def test_shared_copies_of_a_prefix_are_not_read():
    check_shared([90, 95, 99], [0, 3], [80], 2, 2, 64, 16, "bf16", "f32", common=False)


def test_shared_values_out_of_range_count_as_the_nearer_end():
    check_shared([500, -3, 120], [-4, 9], [1000], 2, 2, 64, 16, "bf16", "f32", max_prefix=60, max_len=150)


@pytest.mark.parametrize("kind", CACHES)
def test_shared_ignores_what_lies_outside(kind):
    lens = [61, 70, 66, 9]
    def poison(sections, table):
        pages = {(int(table[r, t // 16]), t % 16) for r, n in enumerate(lens) for t in range(n)}
        K, V, ks, vs = sections
        for p in range(K.shape[0]):
            for o in range(16):
                if (p, o) in pages:
                    continue
                bad = [float("nan"), float("inf"), -float("inf")][(p + o) % 3]
                if ks is None:
                    K[p, :, o], V[p, :, o // 8, :, o % 8] = bad, bad
                else:
                    ks[p, :, o], vs[p, :, o] = bad, bad
    check_shared(lens, [0, 3, 4], [53, 7], 2, 2, 64, 16, kind, "f32", poison=poison)


@pytest.mark.parametrize("kind", CACHES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_shared_long_prefix_is_split(dt, kind):
    check_shared([4010, 4200, 4100], [0, 3], [4000], 1, 4, 64, 64, kind, dt)


@pytest.mark.parametrize("start", [[0, 4, 4, 0, 2], [4, 2, 4, 1, 4]])
def test_shared_groups_that_do_not_ascend_are_not_looked_up_behind_the_requests(start):
    """What such groups give is undefined, but every row is written, and from the buffers of the call alone."""
    out, lse, _, _ = run_shared([40, 50, 60, 70], start, [16, 8, 24, 12], 2, 2, 64, 8, "bf16", "f32", common=False)
    assert not (out == 7.0).all(-1).any() and not (lse == 7.0).any()
