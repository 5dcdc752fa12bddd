"""GPU tests of the operators of include/bitq_lm.h against plain references in 64 bits."""
import math

import numpy as np
import pytest

import bit_plane_gemv_amd as bq
import lm_reference as ref
from gpuhelp import say

pytestmark = pytest.mark.gpu
BF16_ULP = 2.0 ** -8      # half an ulp of bf16 is at most 2^-8 of the value (2^-9 rounding, doubled)


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def close(got, want, tol, what):
    got = np.asarray(got, dtype=np.float64)
    bad = ~(np.abs(got - want) <= tol)
    bad &= ~((got == want) | (np.isnan(got) & np.isnan(want)))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; first {i}: {got[i]} want {want[i]} tol {np.broadcast_to(tol, got.shape)[i]}")


# ------------------------------------------------------------------- plan
def run_plan(old, new, page, stride, ring, head, count, table, T):
    import torch
    d = bq.kv_plan_desc(len(old), page, stride, len(ring), T)
    dev = lambda a: torch.from_numpy(np.array(a, dtype=np.int32)).cuda()  # noqa: E731
    o, n, rg, st, tb = dev(old), dev(new), dev(ring), dev([head, count]), dev(table)
    buf = torch.full((bq.kv_plan_size(d),), 0x5A, dtype=torch.uint8, device="cuda")
    bq.kv_plan(d, o, n, rg, st, tb, buf)
    torch.cuda.synchronize()
    got = {k: v.cpu().numpy().copy() for k, v in bq.kv_plan_views(d, buf).items()}
    got["table"], got["ring"] = tb.cpu().numpy(), rg.cpu().numpy()
    bq.kv_plan(d, o, n, rg, st, tb, buf)          # the same arguments again: the same result
    torch.cuda.synchronize()
    for k, v in bq.kv_plan_views(d, buf).items():
        assert np.array_equal(v.cpu().numpy(), got[k]), f"second call: {k}"
    assert np.array_equal(tb.cpu().numpy(), got["table"]) and np.array_equal(rg.cpu().numpy(), got["ring"])
    return got


def plan_case(rng, R, page, max_len, T, free, kinds):
    stride = ref.ceil_div(max_len, page)
    old = rng.integers(0, max_len + 1, R)
    kind = rng.choice(kinds, R)
    new = old.copy()
    for r in range(R):
        if kind[r] == "grow":
            new[r] = rng.integers(old[r], max_len + 1)
        elif kind[r] == "one":
            new[r] = min(old[r] + 1, max_len)
        elif kind[r] == "prompt":
            old[r], new[r] = 0, rng.integers(1, max_len + 1)
        elif kind[r] == "done":
            new[r] = 0
        elif kind[r] == "cut":
            new[r] = rng.integers(0, old[r] + 1)
        elif kind[r] == "bad":
            old[r], new[r] = [(-1, 5), (3, -7), (3, max_len + page + 1)][rng.integers(3)]
    held = np.maximum(0, -(-old // page))
    cap = int(held.sum()) + max(free, 0) + int(rng.integers(0, 5)) + 1
    ids = rng.permutation(cap)
    table = np.full((R, stride), -1)
    at = 0
    for r in range(R):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    head = int(rng.integers(cap))
    ring = np.full(cap, -1)
    ring[(head + np.arange(free)) % cap] = ids[at:at + free]
    return old, new, page, stride, ring, head, free, table, T


@pytest.mark.parametrize("R,page,max_len,T,free,kinds", [
    (1, 16, 40, 1, 1, ["one"]),
    (1, 8, 8, 8, 0, ["grow", "one"]),
    (7, 8, 100, 500, 40, ["grow", "one", "idle"]),
    (64, 16, 300, 64, 64, ["one"]),
    (64, 16, 300, 64, 2, ["one"]),                                   # pages run out
    (65, 32, 500, 300, 200, ["grow", "one", "prompt"]),              # tokens run out
    (200, 1024, 5000, 4000, 100, ["one", "prompt", "done", "cut", "idle", "bad"]),
    (300, 64, 700, 20000, 3000, ["one", "prompt", "done", "cut", "idle"]),
    (1500, 16, 200, 30000, 9000, ["one", "prompt", "done", "cut", "idle", "bad"]),
    (8192, 8, 64, 70000, 50000, ["one", "prompt", "done", "cut", "idle"]),
    (50, 16, 100, 100, 10, ["done", "cut", "idle"]),                 # nothing grows
])
def test_plan(R, page, max_len, T, free, kinds):
    rng = np.random.default_rng(R * 7919 + page)
    for trial in range(3):
        say("plan", R, page, max_len, T, free, trial)
        args = plan_case(rng, R, page, max_len, T, free, kinds)
        old, new, _, stride, ring, head, count, table, _ = args
        got = run_plan(*args)
        t2, r2 = table.astype(np.int32).copy(), ring.astype(np.int32).copy()
        want = ref.plan(old, new, page, t2, r2, head, count, T)
        want["table"], want["ring"] = t2, r2
        for k, v in want.items():
            assert np.array_equal(got[k], v), f"{k}: {np.argwhere(got[k] != v)[:3].tolist()}"


def test_plan_state_outside_its_range():
    """A head beyond the ring wraps, a count beyond it is cut; pages that find no room are not put back."""
    say("plan bad state")
    table = np.array([[0, 1], [2, -1]])
    ring = np.array([5, 6, 7, 8])
    got = run_plan([0, 10], [20, 0], 16, 2, ring, -3, 99, table, 30)    # head -3 -> 1, count -> 4
    t2, r2 = table.astype(np.int32), ring.astype(np.int32)
    want = ref.plan([0, 10], [20, 0], 16, t2, r2, 1, 4, 30)
    for k, v in want.items():
        assert np.array_equal(got[k], v), k
    assert np.array_equal(got["table"], t2) and np.array_equal(got["ring"], r2)


def test_plan_steps_in_turn():
    """Several steps with two plan buffers in turn, the state and lengths staying on the GPU."""
    import torch
    say("plan in turn")
    rng = np.random.default_rng(5)
    R, page, stride, cap, T = 20, 8, 16, 150, 400
    d = bq.kv_plan_desc(R, page, stride, cap, T)
    bufs = [torch.zeros(bq.kv_plan_size(d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    views = [bq.kv_plan_views(d, b) for b in bufs]
    table, ring = np.full((R, stride), -1, np.int32), rng.permutation(cap).astype(np.int32)
    tb, rg = torch.from_numpy(table).cuda(), torch.from_numpy(ring).cuda()
    views[1]["state"].copy_(torch.tensor([0, cap, 0, 0]))
    views[1]["len"].zero_()
    length, head, count = np.zeros(R, np.int64), 0, cap
    for step in range(12):
        want_len = np.where(rng.random(R) < 0.2, 0, np.minimum(length + rng.integers(0, 20, R), stride * page))
        new = torch.from_numpy(want_len.astype(np.int32)).cuda()
        cur, last = views[step % 2], views[1 - step % 2]
        bq.kv_plan(d, last["len"], new, rg, last["state"], tb, bufs[step % 2])
        w = ref.plan(length, want_len, page, table, ring, head, count, T)
        torch.cuda.synchronize()
        for k, v in w.items():
            assert np.array_equal(cur[k].cpu().numpy(), v), (step, k)
        length, head, count = w["len"].astype(np.int64), int(w["state"][0]), int(w["state"][1])
        used = np.concatenate([table[r, :ref.ceil_div(int(length[r]), page)] for r in range(R)])
        free = ring[(head + np.arange(count)) % cap]
        assert sorted(np.concatenate([used, free]).tolist()) == list(range(cap)), "a page was lost or given twice"


# ------------------------------------------------------------------ write
@pytest.mark.parametrize("T,H,D,page,int8,f32,mode", [
    (1, 1, 1, 8, False, True, "random"),
    (1, 8, 128, 16, False, True, "random"),
    (7, 3, 33, 8, False, False, "random"),
    (64, 8, 128, 16, False, True, "random"),
    (64, 8, 128, 16, True, False, "random"),
    (100, 2, 80, 32, True, True, "runs"),
    (130, 5, 96, 64, False, False, "runs"),
    (700, 8, 128, 64, False, False, "runs"),
    (700, 8, 64, 8, True, False, "runs"),
    (900, 5, 256, 128, False, True, "runs"),
    (1000, 3, 255, 1024, True, True, "runs"),
    (2500, 2, 72, 16, True, False, "mixed"),
    (5000, 1, 40, 8, False, False, "mixed"),
    (1200, 8, 128, 64, False, False, "runs"),                        # from here on 8 tokens a thread
    (1400, 8, 128, 64, True, False, "runs"),
    (2000, 3, 255, 1024, True, True, "runs"),
    (16000, 2, 72, 16, True, False, "mixed"),
    (16000, 2, 72, 8, False, False, "mixed"),
    (30000, 1, 80, 8, False, True, "mixed"),
])
def test_write(T, H, D, page, int8, f32, mode):
    import torch
    say("write", T, H, D, page, int8, f32, mode)
    rng = np.random.default_rng(T + 13 * D)
    pages = ref.ceil_div(T, page) + 40
    total = pages * page
    if mode == "random":
        slots = rng.permutation(total)[:T]
    else:                                         # runs of consecutive slots beginning anywhere in a page
        slots, order = [], rng.permutation(pages)
        for p in order:
            if len(slots) >= T:
                break
            a, b = sorted(rng.integers(0, page + 1, 2)) if mode == "mixed" or rng.random() < 0.3 else (0, page)
            run = list(range(p * page + a, p * page + b))
            if mode == "mixed" and rng.random() < 0.3:
                rng.shuffle(run)
            slots += run
        T = min(T, len(slots))
        slots = np.array(slots[:T])
    slots = slots.astype(np.int32)
    if T > 5:
        slots[T // 2], slots[T // 3] = -1, total  # skipped
    kv = bq.kvdesc(H, D, page, pages, bq.KV_INT8 if int8 else bq.KV_BF16)
    cache = torch.full((bq.kv_cache_size(kv),), 0x11, dtype=torch.uint8, device="cuda")
    views = bq.kv_cache_views(kv, cache)
    before = {n: t.cpu().clone() for n, t in views.items()}
    x = torch.from_numpy(rng.standard_normal((T, 2, H, D)).astype(np.float32))
    x[0, 0, 0] = 0                                # a row of zeros
    if not f32:
        x = x.to(torch.bfloat16)
    xd = x.cuda()
    bq.kv_write(kv, xd[:, 0], xd[:, 1], bq.DT_F32 if f32 else bq.DT_BF16, torch.from_numpy(slots).cuda(), cache)
    torch.cuda.synchronize()
    K, V, ks, vs = (before.get(n) for n in ("K", "V", "ks", "vs"))
    ref.write(K, V, ks, vs, x[:, 0].float(), x[:, 1].float(), slots, page)
    for n, want in (("K", K), ("V", V), ("ks", ks), ("vs", vs)):
        if want is not None:
            got = views[n].cpu()
            same = got.view(torch.int16 if got.dtype == torch.bfloat16 else torch.uint8 if got.dtype == torch.int8 else torch.int32) == \
                want.view(torch.int16 if got.dtype == torch.bfloat16 else torch.uint8 if got.dtype == torch.int8 else torch.int32)
            assert bool(same.all()), f"{n}: {(~same).sum()} differ, first {(~same).nonzero()[0].tolist()}"


def test_write_unaligned_rows_and_no_tokens():
    """Rows at odd element offsets and odd strides; tokens = 0 writes nothing."""
    import torch
    say("write unaligned")
    H, D, page, T = 2, 64, 16, 37
    kv = bq.kvdesc(H, D, page, 4)
    rng = np.random.default_rng(3)
    base = torch.from_numpy(rng.standard_normal(1 + T * 131 + 7 + T * 129 + H * D).astype(np.float32)).to(torch.bfloat16)
    k = base[1:].as_strided((T, H, D), (131, D, 1))
    v = base[1 + T * 131 + 6:].as_strided((T, H, D), (129, D, 1))
    slots = rng.permutation(64)[:T].astype(np.int32)
    cache = torch.zeros(bq.kv_cache_size(kv), dtype=torch.uint8, device="cuda")
    bd = base.cuda()
    bq.kv_write(kv, bd[1:].as_strided((T, H, D), (131, D, 1)), bd[1 + T * 131 + 6:].as_strided((T, H, D), (129, D, 1)),
                bq.DT_BF16, torch.from_numpy(slots).cuda(), cache)
    torch.cuda.synchronize()
    views = bq.kv_cache_views(kv, cache)
    K, V = torch.zeros_like(views["K"].cpu()), torch.zeros_like(views["V"].cpu())
    ref.write(K, V, None, None, k.float(), v.float(), slots, page)
    assert torch.equal(views["K"].cpu(), K) and torch.equal(views["V"].cpu(), V)
    bq.kv_write(kv, bd, bd, bq.DT_BF16, torch.from_numpy(slots).cuda(), cache, tokens=0, k_stride=128, v_stride=128)
    torch.cuda.synchronize()
    assert torch.equal(views["K"].cpu(), K)


# -------------------------------------------------------------- attention
def run_attention(K, V, ks, vs, q, table, lens, page, scale, window, max_len, qf32, of32, q_pad=0, poison=None):
    import torch
    R, A, D = q.shape
    pages, H = K.shape[:2]
    kv = bq.kvdesc(H, D, page, pages, bq.KV_BF16 if ks is None else bq.KV_INT8)
    cache = torch.zeros(bq.kv_cache_size(kv), dtype=torch.uint8, device="cuda")
    for n, t in bq.kv_cache_views(kv, cache).items():
        t.copy_({"K": K, "V": V, "ks": ks, "vs": vs}[n])
    if poison is not None:
        poison(bq.kv_cache_views(kv, cache))
    d = bq.attn_desc(kv, A, R, table.shape[1], max_len, window=window, q_dtype=bq.DT_F32 if qf32 else bq.DT_BF16,
                     out_dtype=bq.DT_F32 if of32 else bq.DT_BF16, scale=scale)
    qd = torch.zeros(R, A * D + q_pad, dtype=torch.float32 if qf32 else torch.bfloat16, device="cuda")
    qd[:, :A * D] = torch.from_numpy(q).reshape(R, -1).cuda()
    out = torch.full((R, A, D), 7.0, dtype=torch.float32 if of32 else torch.bfloat16, device="cuda")
    lse = torch.full((R, A), 7.0, device="cuda")
    ws = torch.full((max(1, bq.paged_attn_workspace(d)),), 0xFF, dtype=torch.uint8, device="cuda")
    bq.paged_attn(d, qd, cache, torch.from_numpy(table.astype(np.int32)).cuda(),
                  torch.from_numpy(np.array(lens, dtype=np.int32)).cuda(), out, ws, lse=lse)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), lse.cpu().numpy()


def attention_case(rng, R, H, G, D, page, lens, int8, qf32, scale_q=1.0):
    import torch
    per = [max(1, ref.ceil_div(max(int(n), 0), page)) for n in lens]
    pages = sum(per) + 2
    K, V, ks, vs = ref.cache_sections(pages, H, page, D, int8, rng)
    ids = rng.permutation(pages)
    table = np.zeros((R, max(per) + 1), dtype=np.int64)
    at = 0
    for r in range(R):
        table[r, :per[r]] = ids[at:at + per[r]]
        at += per[r]
    q = (rng.standard_normal((R, H * G, D)) * scale_q).astype(np.float32)
    if not qf32:
        q = torch.from_numpy(q).to(torch.bfloat16).float().numpy()
    return K, V, ks, vs, q, table


ATTN = [
    # R, H, G, D, page, lens, int8, q f32, out f32, window
    (1, 1, 1, 64, 16, [1], False, False, False, 0),
    (1, 1, 1, 1, 8, [3], False, True, True, 0),
    (3, 2, 1, 128, 16, [0, 1, 31], False, True, True, 0),
    (4, 2, 4, 128, 16, [32, 33, 127, 128], False, False, False, 0),
    (4, 2, 4, 128, 8, [129, 255, 0, 257], True, False, True, 0),
    (2, 4, 8, 128, 32, [2049, 5], False, True, True, 0),
    (2, 4, 8, 128, 32, [2049, 5], True, True, True, 0),
    (3, 1, 16, 80, 64, [700, 64, 63], False, False, True, 0),
    (3, 1, 20, 80, 64, [700, 64, 63], True, False, False, 0),       # two tiles of query heads
    (2, 3, 33, 96, 128, [300, 1000], False, True, False, 0),        # three tiles
    (5, 2, 7, 72, 16, [600, 0, 17, 333, 128], False, True, True, 100),
    (5, 2, 7, 72, 16, [600, 0, 17, 333, 128], True, False, False, 1),
    (2, 1, 2, 256, 1024, [1500, 40], False, True, True, 0),
    (2, 1, 2, 256, 8, [1500, 40], True, False, True, 513),
    (2, 2, 1, 200, 16, [150, 450], False, False, False, 0),
    (1, 2, 3, 160, 16, [901], True, True, True, 0),
    (1, 2, 3, 224, 16, [901], False, True, True, 0),
    (1, 1, 1, 32, 16, [5000], False, False, True, 0),               # one item over the whole grid
    (70, 8, 2, 64, 16, "ragged", False, False, False, 0),
    (70, 8, 2, 64, 16, "ragged", True, True, True, 77),
    (600, 1, 1, 33, 8, "short", False, False, True, 0),             # requests beyond one scan round
    (64, 2, 4, 128, 16, "ragged", False, False, False, 0),          # lengths in one wave's registers: the most, and one more
    (65, 2, 4, 128, 16, "ragged", False, False, False, 0),
    (64, 1, 4, 88, 16, "ragged", True, True, False, 300),
    (1, 1, 3, 64, 64, [70000], False, True, True, 0),               # hundreds of partial results for each head
    (17, 1, 1, 64, 32, [100000] + [1] * 16, True, True, True, 0),
    (600, 1, 1, 40, 16, [20000, 0, 3] * 2 + [1] * 594, False, False, True, 0),
    (400, 2, 3, 64, 16, [7 * i % 65 for i in range(400)], False, True, True, 0),    # workgroups of one wave
    (260, 2, 17, 128, 16, [11 * i % 50 for i in range(260)], True, False, False, 20),
    (150, 2, 2, 256, 32, [13 * i % 129 for i in range(150)], False, False, True, 0),
    (300, 1, 1, 250, 8, [5 * i % 129 for i in range(300)], True, True, False, 0),
    (5000, 1, 1, 32, 8, [3 * i % 40 for i in range(5000)], False, False, False, 0),
    (4096, 1, 1, 256, 8, [300] + [i % 4 for i in range(4095)], False, True, True, 0),   # the most LDS: sums of 4096 requests
    (4097, 1, 2, 64, 16, [300] + [i % 4 for i in range(4096)], True, False, False, 0),  # too many of them: one workgroup an item
    (4096, 1, 1, 256, 8, [1500] + [i % 4 for i in range(4095)], False, True, True, 0),
    (4097, 1, 2, 64, 16, [1500] + [i % 4 for i in range(4096)], True, False, False, 0),
    (64, 2, 4, 128, 16, "long", False, False, False, 0),            # long enough to be split
    (65, 2, 4, 128, 16, "long", True, True, True, 0),
    (64, 1, 4, 88, 16, "long", True, True, False, 1300),
    (70, 4, 2, 64, 16, "long", False, False, True, 1100),
    (30, 3, 20, 96, 32, "long", False, False, False, 0),
    (140, 1, 3, 160, 64, "long", True, False, True, 0),
]


@pytest.mark.parametrize("R,H,G,D,page,lens,int8,qf32,of32,window", ATTN)
def test_attention(R, H, G, D, page, lens, int8, qf32, of32, window):
    say("attn", R, H, G, D, page, int8, qf32, of32, window)
    rng = np.random.default_rng(R * 100 + D + page)
    if lens == "ragged":
        lens = (rng.random(R) ** 3 * 900).astype(int)
        lens[[3, 4]] = 0, 900
    elif lens == "short":
        lens = rng.integers(0, 140, R)
    elif lens == "long":
        lens = (rng.random(R) ** 3 * 3000).astype(int)
        lens[[3, 4]] = 0, 3000
    K, V, ks, vs, q, table = attention_case(rng, R, H, G, D, page, lens, int8, qf32, 2.0)
    max_len = max(1, max(lens))
    scale = D ** -0.5
    out, lse = run_attention(K, V, ks, vs, q, table, lens, page, scale, window, max_len, qf32, of32, q_pad=8)
    want, wlse, tol, ltol = ref.attention(q.astype(np.float64), K, V, ks, vs, table, lens, page, scale, window, max_len)
    close(out, want, tol + (0 if of32 else BF16_ULP * np.abs(want)), "out")
    close(lse, wlse, ltol, "lse")


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("window", [0, 45])
def test_attention_ignores_what_is_outside(int8, window):
    """Infinities and NaN in every slot (and scale) that no request's window covers."""
    import torch
    say("attn poison", int8, window)
    rng = np.random.default_rng(11)
    R, H, G, D, page, lens = 4, 2, 3, 64, 16, [300, 17, 0, 130]
    K, V, ks, vs, q, table = attention_case(rng, R, H, G, D, page, lens, int8, False)
    live = torch.zeros(K.shape[0], page, dtype=torch.bool)
    for r, n in enumerate(lens):
        for t in range(max(0, n - window) if window else 0, n):
            live[table[r, t // page], t % page] = True

    def poison(views):
        dead = ~live.cuda()
        bad = torch.tensor([math.nan, math.inf, -math.inf], device="cuda")
        if int8:
            for n in ("ks", "vs"):
                views[n].copy_(torch.where(dead[:, None], bad[0], views[n]))
            views["K"].copy_(torch.where(dead[:, None, :, None], torch.tensor(-128, dtype=torch.int8, device="cuda"), views["K"]))
        else:
            fill = bad[torch.arange(views["K"].numel(), device="cuda") % 3].to(torch.bfloat16)
            views["K"].copy_(torch.where(dead[:, None, :, None], fill.view_as(views["K"]), views["K"]))
            d8 = dead.view(-1, 1, page // 8, 1, 8)
            views["V"].copy_(torch.where(d8, fill.view_as(views["V"]), views["V"]))

    clean = run_attention(K, V, ks, vs, q, table, lens, page, 0.125, window, 300, False, True)
    dirty = run_attention(K, V, ks, vs, q, table, lens, page, 0.125, window, 300, False, True, poison=poison)
    assert np.array_equal(clean[0], dirty[0]) and np.array_equal(clean[1], dirty[1])
    assert np.all(clean[0][2] == 0) and np.all(clean[1][2] == -np.inf)


@pytest.mark.parametrize("qf32", [False, True])
def test_attention_takes_any_row_stride_of_q(qf32):
    """Rows of q that 16-byte loads can take, and rows that they cannot: the same result."""
    say("attn q stride", qf32)
    rng = np.random.default_rng(16)
    K, V, ks, vs, q, table = attention_case(rng, 3, 2, 5, 64, 16, [200, 33, 64], False, qf32)
    runs = [run_attention(K, V, ks, vs, q, table, [200, 33, 64], 16, 0.125, 0, 200, qf32, True, q_pad=p) for p in (0, 8, 4, 3, 1)]
    for o, l in runs[1:]:
        assert np.array_equal(o, runs[0][0]) and np.array_equal(l, runs[0][1])


def test_attention_lengths_and_pages_outside_their_range():
    """Lengths below 0 count as 0, above max_len as max_len; a page index outside the pool reads page 0."""
    say("attn ranges")
    rng = np.random.default_rng(12)
    lens = [200, 200]
    K, V, ks, vs, q, table = attention_case(rng, 2, 1, 2, 64, 16, lens, False, True)
    a = run_attention(K, V, ks, vs, q, table, [-5, 999], 16, 0.1, 0, 190, True, True)
    b = run_attention(K, V, ks, vs, q, table, [0, 190], 16, 0.1, 0, 190, True, True)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    odd, zero = table.copy(), table.copy()
    odd[1, 3], zero[1, 3] = 1 << 29, 0
    odd[1, 5], zero[1, 5] = -7, 0
    a = run_attention(K, V, ks, vs, q, odd, lens, 16, 0.1, 0, 200, True, True)
    b = run_attention(K, V, ks, vs, q, zero, lens, 16, 0.1, 0, 200, True, True)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_attention_large_scores_and_one_hot():
    """Scores of +-1e4: the weights are one-hot and the output is that token's value."""
    import torch
    say("attn one-hot")
    rng = np.random.default_rng(13)
    n = 777
    K, V, ks, vs, q, table = attention_case(rng, 1, 1, 1, 64, 32, [n], False, True)
    hot = 431
    K[:] = 0
    K[table[0, hot // 32], 0, hot % 32, 0] = 100.0
    K[table[0, 5 // 32], 0, 5, 0] = -100.0
    q[:] = 0
    q[0, 0, 0] = 100.0
    out, lse = run_attention(K, V, ks, vs, q, table, [n], 32, 1.0, 0, n, True, True)
    v = V[table[0, hot // 32], 0, hot % 32 // 8, :64, hot % 8].float().numpy()
    assert np.array_equal(out[0, 0], v)
    close(lse, np.array([[1e4]]), 1e4 * 2.0 ** -22, "lse")
    assert torch.isfinite(torch.from_numpy(out)).all()


def test_attention_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes: the last pages are read where they are."""
    import torch
    say("attn long pool")
    H, D, page = 4, 128, 64
    pages = 70000                                # 70000 * 4 * 64 * 128 * 2 B = 4.6 GB per section
    kv = bq.kvdesc(H, D, page, pages)
    cache = torch.zeros(bq.kv_cache_size(kv), dtype=torch.uint8, device="cuda")
    views = bq.kv_cache_views(kv, cache)
    assert views["K"].numel() * 2 > 1 << 32
    rng = np.random.default_rng(14)
    n = 300
    slots = torch.from_numpy(((pages - 1 - np.arange(n) // page) * page + np.arange(n) % page).astype(np.int32)).cuda()
    x = torch.from_numpy(rng.standard_normal((n, 2, H, D)).astype(np.float32)).to(torch.bfloat16)
    xd = x.cuda()
    bq.kv_write(kv, xd[:, 0], xd[:, 1], bq.DT_BF16, slots, cache)
    table = torch.arange(pages - 1, pages - 7, -1, dtype=torch.int32, device="cuda").view(1, -1)
    d = bq.attn_desc(kv, H, 1, table.shape[1], n, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
    q = torch.from_numpy(rng.standard_normal((1, H, D)).astype(np.float32))
    out = torch.empty(1, H, D, device="cuda")
    ws = torch.zeros(bq.paged_attn_workspace(d), dtype=torch.uint8, device="cuda")
    bq.paged_attn(d, q.cuda(), cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), out, ws)
    torch.cuda.synchronize()
    k, v = x[:, 0].double(), x[:, 1].double()
    s = torch.einsum("hd,thd->ht", q[0].double(), k) * D ** -0.5
    want = torch.einsum("ht,thd->hd", torch.softmax(s, 1), v)
    assert float((out.cpu().double()[0] - want).abs().max()) < 1e-5


# ------------------------------------------------------------------- norm
def host(t, dt):
    import torch
    return torch.from_numpy(t).to(torch.float32 if dt == bq.DT_F32 else torch.bfloat16)


@pytest.mark.parametrize("M,C", [(1, 1), (1, 4096), (3, 7), (5, 64), (2, 513), (4, 1000), (1, 11008), (3, 28672), (2, 32768),
                                 (2, 32767), (1300, 96), (1100, 2048), (1030, 4104), (70, 8192),
                                 (1100, 1000), (300, 4000), (300, 4001), (300, 8001), (3, 5001), (3, 12345)])
@pytest.mark.parametrize("udt,rdt,wdt,odt,post,gate,resid", [
    ("f", "f", "f", "f", True, "channel", True),
    ("b", "b", "b", "b", True, "token", True),
    ("f", "b", "f", "b", False, "none", True),
    ("b", "f", "b", "f", True, "none", False),
    ("f", "f", "b", "8", True, "token", True),
    ("b", "b", "f", "8", False, "none", False),
])
def test_norm(M, C, udt, rdt, wdt, odt, post, gate, resid):
    import torch
    say("norm", M, C, udt, rdt, wdt, odt, post, gate, resid)
    rng = np.random.default_rng(M * 31 + C)
    code = {"f": bq.DT_F32, "b": bq.DT_BF16, "8": bq.DT_ROW8}
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    u, r = host(3 * f(M, C), code[udt]), host(2 * f(M, C), code[rdt])
    if M > 2:
        u[1], r[1] = 0, 0                        # a row of zeros
    w_post, w_pre = host(1 + f(C), code[wdt]), host(1 + f(C), code[wdt])
    g = {"none": None, "channel": host(f(C), code[wdt]), "token": host(f(M, C), code[wdt])}[gate]
    pad = 3 if C < 2000 else 0                   # odd strides (rows off their alignment)

    def dev(t):
        b = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
        b[:, :t.shape[1]] = t.cuda()
        return b
    ud, rd = dev(u), dev(r)
    gd = None if g is None else g.cuda() if gate == "channel" else dev(g)
    ot = {"f": torch.float32, "b": torch.bfloat16, "8": torch.int8}[odt]
    h = torch.zeros(M, C + pad, dtype=ot, device="cuda")
    ro = torch.zeros(M, C + pad, dtype=r.dtype, device="cuda")
    dsc = torch.zeros(M, device="cuda") if odt == "8" else None
    st = C + pad
    d = bq.norm_desc(M, C, code[udt], code[rdt], code[wdt], code[odt], res_scale=0.75, branch_scale=-1.5, eps_post=1e-3,
                     eps_pre=1e-4, gate_stride=st if gate == "token" else 0, u_stride=st, r_stride=st, ro_stride=st,
                     h_stride=st)
    bq.block_norm(d, ud, rd if resid else None, w_post.cuda() if post else None, gd, w_pre.cuda(), ro, h, dsc)
    torch.cuda.synchronize()
    n64 = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    wro, wh, mro, mh = ref.norm(n64(u), n64(r) if resid else None, n64(w_post) if post else None, n64(g), n64(w_pre), 0.75,
                                -1.5, 1e-3, 1e-4)
    # fp32: each element passes fewer than 16 roundings, the sums' relative error stays below that of C / 512 + 16 more
    eps = 2.0 ** -24 * (32 + C / 256)
    close(ro[:, :C].float().cpu().numpy(), wro, eps * mro + (BF16_ULP * np.abs(wro) if rdt == "b" else 0), "r")
    got = h[:, :C].float().cpu().numpy()
    if odt == "8":
        dd = dsc.cpu().numpy().astype(np.float64)[:, None]
        amax = np.abs(wh).max(1, keepdims=True)
        close(dd, amax / 127, eps * mh.max(1, keepdims=True) / 127 + 2.0 ** -23 * amax / 127, "scale")
        close(got * dd, wh, dd * 0.5 * (1 + 1e-5) + 130 * eps * mh, "values")   # half a step, and the value's own error
        assert np.abs(got).max() <= 127
    else:
        close(got, wh, eps * mh + (BF16_ULP * np.abs(wh) if odt == "b" else 0), "h")
    if pad:
        assert float(h[:, C:].float().abs().max()) == 0 and float(ro[:, C:].float().abs().max()) == 0


def test_norm_in_place_and_optional_outputs():
    """r' written over r; no r'; neither norm (a plain row quantizer: the bits of the activation quantizer)."""
    import torch
    say("norm optional")
    rng = np.random.default_rng(2)
    M, C = 37, 416
    u, r = (torch.from_numpy(rng.standard_normal((M, C)).astype(np.float32)).cuda() for _ in range(2))
    pre = torch.ones(C, device="cuda")
    d = bq.norm_desc(M, C)
    ro, h, h2, h3 = (torch.empty(M, C, device="cuda") for _ in range(4))
    bq.block_norm(d, u, r, None, None, pre, ro, h)
    rr = r.clone()
    bq.block_norm(d, u, rr, None, None, pre, rr, h2)
    bq.block_norm(d, u, r, None, None, pre, None, h3)
    torch.cuda.synchronize()
    assert torch.equal(rr, ro) and torch.equal(h, h2) and torch.equal(h, h3)
    q, sc = torch.empty(M, C, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    bq.block_norm(bq.norm_desc(M, C, out_dtype=bq.DT_ROW8), u, None, None, None, None, None, q, sc)
    act = torch.zeros(bq.act_size(M, C), dtype=torch.uint8, device="cuda")
    bq.quantize_act(u, bq.DT_F32, M, C, act)
    torch.cuda.synchronize()
    L = bq.act_layout(M, C)
    q2 = act[L["off_q"]:L["off_q"] + M * L["Kp"]].view(torch.int8).view(M, L["Kp"])[:, :C]
    assert torch.equal(q, q2) and torch.equal(sc, act[L["off_d"]:L["off_d"] + 4 * M].view(torch.float32))


def test_norm_carries_infinities_and_nan():
    import torch
    say("norm nan")
    u = torch.randn(4, 256, device="cuda")
    u[1, 3], u[2, 200] = math.nan, math.inf
    h = torch.empty_like(u)
    bq.block_norm(bq.norm_desc(4, 256), u, None, None, None, torch.ones(256, device="cuda"), None, h)
    bad = ~torch.isfinite(h)
    assert bad[1].all() and bad[2, 200] and not bad[0].any() and not bad[3].any()


# ------------------------------------------------------------------- w8a8
def int_product(a, w):
    """The exact int32 sums (fp64 products of integers below 2^53)."""
    return (a.double() @ w.double().t()).to(__import__("torch").int64)


W8A8 = [(1, 1, 16), (1, 16, 64), (1, 17, 4096), (2, 100, 80), (16, 33, 144), (17, 64, 1040), (33, 130, 272), (48, 40, 2064),
        (64, 300, 512), (49, 4096, 1024), (65, 129, 128), (100, 257, 400), (128, 128, 128), (129, 300, 1040), (200, 512, 4096),
        (257, 1000, 656), (300, 16, 16), (1000, 777, 2000), (513, 2049, 272), (5, 20, 131056), (130, 140, 131056),
        (9, 3000, 1040), (16, 9001, 272), (20, 7000, 528), (64, 300, 6160), (70, 1500, 7008), (520, 8100, 208), (3000, 9100, 80),
        (2500, 3000, 336), (64, 64, 6400), (7, 4095, 8224), (8, 600, 2064), (11, 4097, 144), (3, 17001, 656), (12, 16400, 272),
        (2, 5000, 8192), (16, 8192, 400), (4, 9000, 6160), (600, 60, 8480), (30, 100, 14352), (64, 200, 12304)]


@pytest.mark.parametrize("M,N,K", W8A8)
def test_w8a8(M, N, K):
    import torch
    say("w8a8", M, N, K)
    g = torch.Generator().manual_seed(M * 1000003 + N * 1009 + K)
    lda, ldw, ldy = K + 32, K + 16, N + 3
    a = torch.randint(-128, 128, (M, lda), generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, ldw), generator=g, dtype=torch.int8)
    sa, sw = torch.rand(M, generator=g) * 0.1, torch.rand(N, generator=g) * 0.01
    ad, wd, sad, swd = a.cuda(), w.cuda(), sa.cuda(), sw.cuda()
    want = int_product(ad[:, :K], wd[:, :K]).cpu()
    d = bq.w8a8_desc(M, N, K, lda=lda, ldw=ldw, ldy=ldy, flags=bq.F_ACC_INT32)
    ws = torch.zeros(max(1, bq.w8a8_workspace(d)), dtype=torch.uint8, device="cuda")
    for rep in range(2):
        y = torch.full((M, ldy), 77, dtype=torch.int32, device="cuda")
        bq.gemm_w8a8(d, ad, None, wd, None, y, ws)
        torch.cuda.synchronize()
        got = y.cpu()
        assert torch.equal(got[:, :N].to(torch.int64), want), f"sums differ, first {(got[:, :N] != want).nonzero()[0].tolist()}"
        assert bool((got[:, N:] == 77).all()), "wrote past a row"
        ws.fill_(0x5A)                            # what an earlier call left does not matter
    exact = want.double() * sa.double()[:, None] * sw.double()
    for dt, t, tol in ((bq.DT_F32, torch.float32, 2.0 ** -22), (bq.DT_BF16, torch.bfloat16, BF16_ULP)):
        y = torch.full((M, ldy), 77, dtype=t, device="cuda")
        bq.gemm_w8a8(bq.w8a8_desc(M, N, K, y_dtype=dt, lda=lda, ldw=ldw, ldy=ldy), ad, sad, wd, swd, y, ws)
        torch.cuda.synchronize()
        got = y.double().cpu()
        close(got[:, :N].numpy(), exact.numpy(), tol * exact.abs().numpy(), f"y {t}")
        assert bool((got[:, N:] == 77).all()), "wrote past a row"


@pytest.mark.parametrize("M", [3, 70])
def test_w8a8_extreme_codes(M):
    """Every code -128 at the longest k: the largest sum that int32 holds."""
    import torch
    say("w8a8 extreme", M)
    K, N = 131056, 18
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    d = bq.w8a8_desc(M, N, K, flags=bq.F_ACC_INT32)
    y = torch.empty(M, N, dtype=torch.int32, device="cuda")
    ws = torch.zeros(max(1, bq.w8a8_workspace(d)), dtype=torch.uint8, device="cuda")
    bq.gemm_w8a8(d, a, None, w, None, y, ws)
    torch.cuda.synchronize()
    want = torch.full((M, N), 128 * 128 * K, dtype=torch.int64)
    want[:, 1] = -128 * 127 * K
    assert torch.equal(y.cpu().to(torch.int64), want)


def test_w8a8_takes_the_activation_buffer():
    """q and d of bitq_quantize_act as the token operand."""
    import torch
    say("w8a8 act")
    M, N, K = 9, 70, 416
    x = torch.randn(M, K, device="cuda")
    act = torch.zeros(bq.act_size(M, K), dtype=torch.uint8, device="cuda")
    bq.quantize_act(x, bq.DT_F32, M, K, act)
    L = bq.act_layout(M, K)
    q = act[L["off_q"]:L["off_q"] + M * L["Kp"]].view(torch.int8).view(M, L["Kp"])
    dsc = act[L["off_d"]:L["off_d"] + 4 * M].view(torch.float32)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    sw = torch.rand(N, device="cuda")
    y = torch.empty(M, N, device="cuda")
    bq.gemm_w8a8(bq.w8a8_desc(M, N, K, lda=L["Kp"]), q, dsc, w, sw, y)
    torch.cuda.synchronize()
    want = int_product(q[:, :K], w).double() * dsc.double()[:, None] * sw.double()
    close(y.cpu().numpy(), want.cpu().numpy(), 2.0 ** -22 * want.abs().cpu().numpy(), "y")


# ------------------------------------------------------- streams and graphs
def test_operators_on_a_side_stream_and_in_a_graph():
    """A decode step's operators captured into a graph on a side stream: every replay equals the eager result."""
    import torch
    say("lm graph")
    torch.manual_seed(0)
    R, H, G, D, page, C = 6, 2, 4, 64, 16, 512
    stride, cap, T = 20, 130, R
    pd = bq.kv_plan_desc(R, page, stride, cap, T)
    kv = bq.kvdesc(H, D, page, cap)
    ad = bq.attn_desc(kv, H * G, R, stride, stride * page, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
    nd = bq.norm_desc(R, C, out_dtype=bq.DT_ROW8)
    gd = bq.w8a8_desc(R, 300, C)
    old = torch.tensor([0, 5, 16, 31, 200, 300], dtype=torch.int32, device="cuda")
    new = old + 1
    table = torch.arange(R * stride, dtype=torch.int32, device="cuda").view(R, stride)
    ring = (torch.arange(cap, dtype=torch.int32, device="cuda") + R * stride) % cap
    state = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    plan = torch.empty(bq.kv_plan_size(pd), dtype=torch.uint8, device="cuda")
    views = bq.kv_plan_views(pd, plan)
    cache = torch.zeros(bq.kv_cache_size(kv), dtype=torch.uint8, device="cuda")
    for t in bq.kv_cache_views(kv, cache).values():
        t.normal_()
    x = torch.randn(R, 2, H, D, device="cuda")
    q = torch.randn(R, H * G, D, device="cuda")
    att = torch.empty(R, H * G, D, device="cuda")
    ws = torch.zeros(bq.paged_attn_workspace(ad), dtype=torch.uint8, device="cuda")
    res, pre = torch.randn(R, C, device="cuda"), torch.rand(C, device="cuda")
    ro, h, hs = torch.empty(R, C, device="cuda"), torch.empty(R, C, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    w, sw = torch.randint(-127, 128, (300, C), dtype=torch.int8, device="cuda"), torch.rand(300, device="cuda")
    y = torch.empty(R, 300, device="cuda")
    gws = torch.zeros(max(1, bq.w8a8_workspace(gd)), dtype=torch.uint8, device="cuda")

    def step():
        bq.kv_plan(pd, old, new, ring, state, table, plan)
        bq.kv_write(kv, x[:, 0], x[:, 1], bq.DT_F32, views["slot"], cache)
        bq.paged_attn(ad, q, cache, table, views["len"], att, ws)
        bq.block_norm(nd, att, res, None, None, pre, ro, h, hs)
        bq.gemm_w8a8(gd, h, hs, w, sw, y, gws)

    step()
    torch.cuda.synchronize()
    outs = [*views.values(), table, ring, cache, att, ro, h, hs, y]
    eager = [o.clone() for o in outs]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for rep in range(4):
        for o in (att, ro, y):
            o.fill_(float("nan"))
        plan.fill_(0x5A)
        torch.randn(1 << 18, device="cuda").sum().item()
        graph.replay()
        torch.cuda.synchronize()
        for i, (o, e) in enumerate(zip(outs, eager)):
            assert torch.equal(o.view(torch.uint8), e.view(torch.uint8)), f"replay {rep}, buffer {i}"


def test_outputs_do_not_change_from_run_to_run():
    import torch
    say("lm determinism")
    rng = np.random.default_rng(8)
    K, V, ks, vs, q, table = attention_case(rng, 3, 2, 4, 128, 16, [900, 33, 2000], False, True)
    runs = [run_attention(K, V, ks, vs, q, table, [900, 33, 2000], 16, 0.1, 0, 2000, True, True) for _ in range(3)]
    for o, s in runs[1:]:
        assert np.array_equal(o, runs[0][0]) and np.array_equal(s, runs[0][1])
