"""kv_fork, kv_compact and kv_copy against loops over the requests (exact)."""
import numpy as np
import pytest
import torch

import bit_plane_gemv_amd as bq
import lm_reference as lm
import serve_reference as ref
from gpuhelp import say

pytestmark = pytest.mark.gpu
i32 = lambda x: torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device="cuda")  # noqa: E731


def ring_of(pool, free, head, cap_fill=-7):
    ring = np.full(pool, cap_fill, dtype=np.int32)
    for i, p in enumerate(free):
        ring[(head + i) % pool] = p
    return ring


def fork(src, keep, lens, table, ring, head, count, page, pool, moves=None, times=1, small=True):
    R, S = table.shape
    d = bq.kv_pages_desc(R, page, S, pool, max(R, moves or 0))
    buf = torch.full((bq.kv_pages_size(d),), 0x5A, dtype=torch.uint8, device="cuda")
    ws = torch.full((bq.kv_pages_workspace(d),), 0x5A, dtype=torch.uint8, device="cuda")
    dev_ring, out = i32(ring), i32(np.full((R, S), -9))
    args = (i32(src), i32(keep), i32(lens), dev_ring, i32([head, count]), i32(table), out, buf, ws)
    say("fork", R, S, page, pool, "held", int(sum(lm.ceil_div(max(0, int(n)), page) for n in lens)))
    for _ in range(times):
        bq.kv_fork(d, *args)
    torch.cuda.synchronize()
    v = {k: x.cpu().numpy() for k, x in bq.kv_pages_views(d, buf).items()}
    want_ring = np.array(ring, dtype=np.int64)
    rows, now, copies, state = ref.fork(src, keep, lens, want_ring, head % pool, min(max(count, 0), pool), np.asarray(table), page, pool)
    got = out.cpu().numpy()
    want = np.array([[-9 if x is None else x for x in row] for row in rows], dtype=np.int64).reshape(R, S)
    assert v["state"].tolist() == state
    assert v["len"].tolist() == now
    n = len(copies)
    assert list(zip(v["frm"][:n].tolist(), v["to"][:n].tolist())) == copies
    assert (v["frm"][n:] == -1).all() and (v["to"][n:] == -1).all()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]
    assert np.array_equal(dev_ring.cpu().numpy(), want_ring.astype(np.int32))
    return got, now, copies, state


def pool_state(lens, page, stride, pool, rng, shared=0):
    """A table of random pages (the first `shared` pages of every request common), the ring of the others."""
    held = [lm.ceil_div(max(int(n), 0), page) for n in lens]
    order = rng.permutation(pool)
    table, at = np.full((len(lens), stride), -3, dtype=np.int32), shared
    for r, n in enumerate(held):
        k = min(shared, n)
        table[r, :k] = order[:k]
        table[r, k:n] = order[at:at + n - k]
        at += n - k
    assert at <= pool
    used = {int(x) for r, n in enumerate(held) for x in table[r, :n]}
    return table, [int(p) for p in order if int(p) not in used]


@pytest.mark.parametrize("pool_extra", [0, 3, 500, 45000])     # 45000: more pages than one workgroup's words
@pytest.mark.parametrize("R,page,most", [(1, 8, 30), (4, 16, 100), (13, 8, 64), (70, 32, 500), (300, 8, 900)])
def test_fork_of_random_requests(R, page, most, pool_extra):
    rng = np.random.default_rng(R + pool_extra)
    for shared in (0, 2):
        lens = rng.integers(0, most + 1, R)
        stride = lm.ceil_div(most, page) + 1
        pool = int(sum(lm.ceil_div(int(n), page) for n in lens)) + pool_extra + shared + 1
        table, free = pool_state(lens, page, stride, pool, rng, shared)
        src = np.where(rng.random(R) < 0.5, rng.integers(0, R, R), np.arange(R))
        keep = np.array([rng.integers(0, lens[s] + 1) if rng.random() < 0.6 else lens[s] for s in src])
        head = int(rng.integers(0, pool))
        fork(src, keep, lens, table, ring_of(pool, free, head), head, len(free), page, pool, times=2)


def test_fork_leaves_cuts_frees_and_forks():
    table = np.array([[5, 6, 7, -1], [1, 2, -1, -1], [9, -1, -1, -1]])
    ring = ring_of(12, [0, 3, 4, 8, 10, 11], 2)
    lens = [40, 20, 16]
    fork([0, 1, 2], lens, lens, table, ring, 2, 6, 16, 12)                    # nothing changes
    fork([0, 1, 2], [17, 16, 0], lens, table, ring, 2, 6, 16, 12)             # cuts, inside a page and at its end; an end
    got, now, copies, _ = fork([0, 0, 0], [40, 40, 33], lens, table, ring, 2, 6, 16, 12)
    assert copies == [(7, 0), (7, 3)] and got[1, :3].tolist() == [5, 6, 0]    # request 0 had the page and keeps it
    got, now, copies, _ = fork([1, 0, 2], [20, 40, 16], lens, table, ring, 2, 6, 16, 12)
    assert copies == [] and got[0, :2].tolist() == [1, 2]                     # two requests change places: no copies
    fork([2, 2, 0], [16, 5, 40], lens, table, ring, 2, 6, 16, 12)             # inside a page that another holds whole
    fork([1, 1, 1], [20, 20, 20], lens, table, ring, 2, 6, 16, 12)


def test_fork_of_requests_that_share_pages_already():
    table = np.array([[5, 6, 7], [5, 6, 8], [5, 6, -1]])
    ring = ring_of(12, [0, 1], 0)
    fork([0, 1, 2], [0, 47, 32], [47, 47, 32], table, ring, 0, 2, 16, 12)     # page 7 alone is given back
    fork([0, 1, 2], [0, 0, 32], [47, 47, 32], table, ring, 0, 2, 16, 12)
    fork([0, 1, 2], [20, 47, 32], [47, 47, 32], table, ring, 0, 2, 16, 12)    # cut inside a page that others hold: a copy
    fork([0, 1, 2], [20, 20, 20], [47, 47, 32], table, ring, 0, 2, 16, 12)    # all cut there: the first keeps it
    fork([0, 1, 2], [0, 0, 0], [47, 47, 32], table, ring, 0, 2, 16, 12)


def test_fork_without_free_pages_ends_at_the_last_whole_page():
    table = np.array([[5, 6, 7], [1, -1, -1], [2, -1, -1]])
    for free in ([], [9]):
        _, now, _, state = fork([0, 0, 0], [40, 40, 40], [40, 10, 3], table, ring_of(10, free, 4), 4, len(free), 16, 10)
        assert now == [40, 40 if free else 32, 32] and state[3] == (1 if free else 2)


def test_fork_refuses_what_is_out_of_range():
    table = np.array([[5, 6], [1, 2]])
    ring = ring_of(8, [0, 3, 4], 6)
    _, now, _, state = fork([2, -1], [3, 3], [20, 30], table, ring, 6, 3, 16, 8)
    assert now == [20, 30] and state[3] == 2
    _, now, _, state = fork([1, 1], [31, -2], [20, 30], table, ring, 6, 3, 16, 8)
    assert now == [20, 30] and state[3] == 2
    _, now, _, _ = fork([0, 1], [32, 0], [999, -4], table, ring, 6, 3, 16, 8)  # lengths count as the nearer end
    assert now == [32, 0]


def test_fork_takes_any_head_and_count():
    table = np.array([[5, 6], [1, 2]])
    for head, count in ((-3, 3), (19, 3), (6, 99), (6, -1)):
        fork([0, 0], [20, 20], [20, 30], table, ring_of(8, [0, 3, 4], head % 8), head, count, 16, 8)


@pytest.mark.parametrize("extra", [0, 50000])
def test_fork_hands_on_pages_outside_the_pool(extra):
    pool = 8 + extra
    table = np.array([[50000000, 6], [1, -2]])
    got, _, copies, _ = fork([0, 0], [17, 5], [20, 30], table, ring_of(pool, [0, 3], 0), 0, 2, 16, pool)
    assert copies == [] and got[1, 0] == 50000000


def compact(lens, table, page, pool, places=None):
    R, S = table.shape
    places = pool if places is None else places
    d = bq.kv_pages_desc(R, page, S, pool, places)
    buf = torch.full((bq.kv_pages_size(d),), 0x5A, dtype=torch.uint8, device="cuda")
    ws = torch.full((bq.kv_pages_workspace(d),), 0x5A, dtype=torch.uint8, device="cuda")
    ring, out = i32(np.full(pool, -7)), i32(np.full((R, S), -9))
    say("compact", R, S, page, pool, places)
    for _ in range(2):
        bq.kv_compact(d, i32(lens), i32(table), out, ring, buf, ws)
    torch.cuda.synchronize()
    v = {k: x.cpu().numpy() for k, x in bq.kv_pages_views(d, buf).items()}
    rows, moves, free, state = ref.compact(lens, np.asarray(table), page, pool, places)
    n = len(moves)
    assert v["state"].tolist() == state
    assert v["len"].tolist() == [min(max(int(x), 0), S * page) for x in lens]
    assert list(zip(v["frm"][:n].tolist(), v["to"][:n].tolist())) == moves
    assert (v["frm"][n:] == -1).all() and (v["to"][n:] == -1).all()
    want = np.array([[-9 if x is None else x for x in row] for row in rows], dtype=np.int64).reshape(R, S)
    assert np.array_equal(out.cpu().numpy(), want)
    assert ring.cpu().numpy().tolist() == free + [-7] * (pool - len(free))


@pytest.mark.parametrize("places", [None, 1, 5])
@pytest.mark.parametrize("pool_extra", [0, 1, 40, 2000, 48000])
@pytest.mark.parametrize("R,page,most", [(1, 8, 30), (5, 16, 100), (40, 8, 300), (200, 8, 900)])
def test_compact(R, page, most, pool_extra, places):
    rng = np.random.default_rng(R + pool_extra)
    for shared in (0, 2):
        lens = rng.integers(0, most + 1, R)
        stride = lm.ceil_div(most, page)
        pool = int(sum(lm.ceil_div(int(n), page) for n in lens)) + pool_extra + shared + 1
        table, _ = pool_state(lens, page, stride, pool, rng, shared)
        compact(lens, table, page, pool, places)


def test_compact_of_an_empty_and_of_a_full_pool():
    compact([0, 0], np.array([[3, 4], [1, 2]]), 16, 6)
    compact([32, 32], np.array([[3, 0], [1, 2]]), 16, 4)
    compact([32, 99], np.array([[3, 70], [-1, 2]]), 16, 5)     # pages outside the pool stay as they are
    compact([16], np.array([[0]]), 16, 1)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("H,D,page", [(1, 1, 8), (2, 64, 16), (5, 80, 32), (8, 128, 64), (3, 256, 128), (1, 32, 1024)])
def test_copy(H, D, page, kind):
    pool = 9
    kv = bq.kvdesc(H, D, page, pool, bq.KV_INT8 if kind == "int8" else bq.KV_BF16)
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = torch.randint(0, 256, (bq.kv_cache_size(kv),), generator=g, dtype=torch.uint8, device="cuda")
    want = cache.clone()
    frm, to = [3, 8, -1, 2, 9, 5, 6, 0], [4, 0, 1, -1, 5, 9, 6, 2 ** 31 - 1]
    for a, b in zip(frm, to):
        if 0 <= a < pool and 0 <= b < pool:
            for name, x in bq.kv_cache_views(kv, want).items():
                x.view(torch.uint8)[b] = bq.kv_cache_views(kv, cache)[name].view(torch.uint8)[a]
    bq.kv_copy(kv, i32(frm), i32(to), cache)
    assert torch.equal(cache, want)
    bq.kv_copy(kv, i32(frm), i32(to), cache, moves=0)
    assert torch.equal(cache, want)


def test_copy_past_32_bits():
    kv = bq.kvdesc(8, 128, 64, (5 << 30) // (2 * 8 * 64 * 128 * 2))
    cache = torch.zeros(bq.kv_cache_size(kv), dtype=torch.uint8, device="cuda")
    v = bq.kv_cache_views(kv, cache)
    v["K"][1], v["V"][1] = 2.0, 3.0
    n = kv.pages
    bq.kv_copy(kv, i32([1, n - 1]), i32([n - 2, 0]), cache)
    assert (v["K"][n - 2] == 2).all() and (v["V"][n - 2] == 3).all()
    assert not v["K"][[0, 2, n - 3, n - 1]].any() and not v["V"][[0, 2, n - 3, n - 1]].any()
