"""Forks and compactions of many requests with short rows of the table: what they give, and that they take about as long as with
longer rows."""
import numpy as np
import pytest
import torch

import bit_plane_gemv_amd as bq
import serve_reference as ref
from gpuhelp import say

pytestmark = pytest.mark.gpu
PAGE = 16
i32 = lambda x: torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")  # noqa: E731


class Pool:
    def __init__(self, R, S, seed):
        rng = np.random.default_rng(seed)
        self.R, self.S = R, S
        self.lens = rng.integers(0, S * PAGE + 1, R)
        held = -(-self.lens // PAGE)
        self.pool = int(held.sum()) + R // 4 + 2
        order = rng.permutation(self.pool)
        self.table = np.zeros((R, S), dtype=np.int32)
        at = 0
        for r, n in enumerate(held):
            self.table[r, :n] = order[at:at + n]
            at += n
        self.ring, self.state = np.roll(order, -at).astype(np.int32), [0, self.pool - at]
        self.src = np.where(rng.random(R) < 0.3, rng.integers(0, R, R), np.arange(R))
        self.keep = (self.lens[self.src] * np.where(rng.random(R) < 0.5, 1, rng.random(R))).astype(np.int64)

    def call(self, fork):
        d = bq.kv_pages_desc(self.R, PAGE, self.S, self.pool, self.R if fork else self.pool)
        result, ws = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (bq.kv_pages_size(d), bq.kv_pages_workspace(d)))
        src, keep, lens, ring, table, state = (i32(x) for x in (self.src, self.keep, self.lens, self.ring, self.table, self.state))
        out = torch.full_like(table, -7)
        run = (lambda: bq.kv_fork(d, src, keep, lens, ring, state, table, out, result, ws)) if fork else (
            lambda: bq.kv_compact(d, lens, table, out, ring, result, ws))
        run()
        return d, result, ring, out, run


SIZES = [(97, 1), (96, 64), (97, 64), (48, 65), (49, 65), (2048, 4), (6000, 1)]


@pytest.mark.parametrize("R,S", SIZES)
def test_fork(R, S):
    p = Pool(R, S, R + S)
    say("fork short rows", R, S, p.pool)
    d, result, ring, out, _ = p.call(True)
    v = bq.kv_pages_views(d, result)
    want_ring = p.ring.copy()
    tables, lens, copies, state = ref.fork(p.src, p.keep, p.lens, want_ring, *p.state, p.table, PAGE, p.pool)
    assert v["state"].tolist() == state and v["len"].tolist() == lens and ring.tolist() == want_ring.tolist()
    assert list(zip(v["frm"].tolist(), v["to"].tolist())) == copies + [(-1, -1)] * (R - len(copies))
    assert out.tolist() == [[-7 if x is None else x for x in row] for row in tables]


@pytest.mark.parametrize("R,S", SIZES)
def test_compact(R, S):
    p = Pool(R, S, R + S)
    say("compact short rows", R, S, p.pool)
    d, result, ring, out, _ = p.call(False)
    v = bq.kv_pages_views(d, result)
    tables, moves, free, state = ref.compact(p.lens, p.table, PAGE, p.pool, p.pool)
    assert v["state"].tolist() == state and v["len"].tolist() == p.lens.tolist() and ring.tolist()[:len(free)] == free
    assert list(zip(v["frm"].tolist(), v["to"].tolist())) == moves + [(-1, -1)] * (p.pool - len(moves))
    assert out.tolist() == [[-7 if x is None else x for x in row] for row in tables]


@pytest.mark.parametrize("fork", [True, False])
def test_time_of_short_rows(fork):
    """2048 rows of 4 entries and of 40: the shorter ones may not take three times as long."""
    took = []
    for S in (4, 40):
        run = Pool(2048, S, 1).call(fork)[-1]
        times = []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(20):
                run()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        took.append(min(times))
    assert took[0] < 3 * took[1], took
