"""The operators that serve prompts and shared pages, run as they are used: prompts rotated, written and attended, requests
forked and their pages copied, decode steps on the common prefix, the pool compacted.  On a side stream, in a graph, twice."""
import numpy as np
import pytest
import torch

import bit_plane_gemv_amd as bq
import lm_reference as lm
import serve_reference as ref
from gpuhelp import say
from test_gpu_serve_attention import close

pytestmark = pytest.mark.gpu
i32 = lambda x: torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device="cuda")  # noqa: E731


class Served:
    """R slots on one layer's cache."""

    def __init__(self, R, H, G, D, page, stride, pool, kind, tokens, seed=0):
        self.R, self.H, self.G, self.D, self.page, self.stride, self.pool = R, H, G, D, page, stride, pool
        self.A, self.max_len = H * G, stride * page
        self.kv = bq.kvdesc(H, D, page, pool, bq.KV_INT8 if kind == "int8" else bq.KV_BF16)
        self.cache = torch.zeros(bq.kv_cache_size(self.kv), dtype=torch.uint8, device="cuda")
        self.tables = [torch.full((R, stride), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
        self.ring, self.state, self.lens = torch.arange(pool, dtype=torch.int32, device="cuda"), i32([0, pool]), i32([0] * R)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.freq = torch.from_numpy(bq.rope_table(D, base=10000.0)).cuda()
        self.w = [1 + 0.1 * torch.randn(D, generator=self.g, device="cuda") for _ in range(2)]
        self.table = self.tables[0]

    def grow(self, new, tokens):
        """Requests to the given lengths: plan, projection, rotation, cache write.  Returns the plan's views and the queries."""
        pd = bq.kv_plan_desc(self.R, self.page, self.stride, self.pool, tokens)
        plan = torch.empty(bq.kv_plan_size(pd), dtype=torch.uint8, device="cuda")
        bq.kv_plan(pd, self.lens, new, self.ring, self.state, self.table, plan)
        p = bq.kv_plan_views(pd, plan)
        qkv = torch.randn(tokens, self.A + 2 * self.H, self.D, generator=self.g, device="cuda")
        q, k, v = qkv[:, :self.A], qkv[:, self.A:self.A + self.H], qkv[:, self.A + self.H:]
        d = bq.rope_desc(tokens, self.A, self.H, self.D, x_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
        bq.qk_rope(d, q, k, *self.w, self.freq, p["pos"], q, k)              # in place, in the projection's rows
        bq.kv_write(self.kv, k, v, bq.DT_F32, p["slot"], self.cache)
        self.lens, self.state = p["len"], p["state"]
        return p, q

    def sections(self):
        v = bq.kv_cache_views(self.kv, self.cache)
        return tuple(v[n].cpu() if n in v else None for n in ("K", "V", "ks", "vs"))

    def fork(self, src, keep):
        d = bq.kv_pages_desc(self.R, self.page, self.stride, self.pool, self.R)
        buf, ws = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (bq.kv_pages_size(d), bq.kv_pages_workspace(d)))
        other = self.tables[1] if self.table is self.tables[0] else self.tables[0]
        bq.kv_fork(d, src, keep, self.lens, self.ring, self.state, self.table, other, buf, ws)
        v = bq.kv_pages_views(d, buf)
        bq.kv_copy(self.kv, v["frm"], v["to"], self.cache)
        self.table, self.lens, self.state = other, v["len"], v["state"]
        return v

    def compact(self):
        d = bq.kv_pages_desc(self.R, self.page, self.stride, self.pool, self.pool)
        buf, ws = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (bq.kv_pages_size(d), bq.kv_pages_workspace(d)))
        other = self.tables[1] if self.table is self.tables[0] else self.tables[0]
        bq.kv_compact(d, self.lens, self.table, other, self.ring, buf, ws)
        v = bq.kv_pages_views(d, buf)
        bq.kv_copy(self.kv, v["frm"], v["to"], self.cache)
        self.table, self.state = other, v["state"]
        return v

    def paged(self, q):
        d = bq.attn_desc(self.kv, self.A, self.R, self.stride, self.max_len, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
        ws = torch.empty(max(1, bq.paged_attn_workspace(d)), dtype=torch.uint8, device="cuda")
        out = torch.empty(self.R, self.A, self.D, device="cuda")
        bq.paged_attn(d, q, self.cache, self.table, self.lens, out, ws)
        return out

    def shared(self, q, start, prefix, max_prefix):
        d = bq.shared_desc(bq.attn_desc(self.kv, self.A, self.R, self.stride, self.max_len, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32),
                           len(start) - 1, max_prefix)
        ws = torch.empty(bq.shared_attn_workspace(d), dtype=torch.uint8, device="cuda")
        out = torch.empty(self.R, self.A, self.D, device="cuda")
        bq.shared_attn(d, q, self.cache, self.table, self.lens, start, prefix, out, ws)
        return out


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_prompts_beams_and_compaction(kind):
    """Two prompts, each continued by 3 beams for some steps, with a beam reordered and one ended."""
    say("together", kind)
    R, page = 6, 16
    s = Served(R, H=2, G=4, D=64, page=page, stride=12, pool=60, kind=kind, tokens=200)
    lens = [100, 0, 0, 37, 0, 0]
    p, q = s.grow(i32(lens), 140)
    assert p["state"].tolist()[2:] == [137, 0]
    d = bq.prompt_desc(s.kv, s.A, R, 140, s.stride, s.max_len, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
    ws = torch.empty(max(1, bq.prompt_attn_workspace(d)), dtype=torch.uint8, device="cuda")
    out = torch.full((140, s.A, s.D), 7.0, device="cuda")
    bq.prompt_attn(d, q, s.cache, s.table, p["start"], p["len"], out, ws)
    scale = np.float32(s.D ** -0.5)
    want, _, tol, _ = ref.prompt(q.double().cpu().numpy(), s.sections(), s.table.cpu().numpy(), p["start"].tolist(), lens, page, scale,
                                 0, 0, s.max_len, 3)
    assert (out[137:] == 7).all()
    close(out[:137], want[:137], tol[:137] + 2.0 ** -24 * np.abs(want[:137]), "prompt")
    # the last row of a prompt is what one token's attention gives
    last = torch.zeros(R, s.A, s.D, device="cuda")
    last[0], last[3] = q[99], q[136]
    one = s.paged(last)
    for r, i in ((0, 99), (3, 136)):
        close(one[r], want[i], 2 * tol[i] + 2.0 ** -23 * np.abs(want[i]), "one token")
    # 3 beams of each
    f = s.fork(i32([0, 0, 0, 3, 3, 3]), i32([100, 100, 100, 37, 37, 37]))
    assert f["len"].tolist() == [100] * 3 + [37] * 3 and f["state"].tolist()[2:] == [4, 0]
    start, prefix = i32([0, 3, 6]), i32([100, 37])
    for step in range(20):
        active = np.array([1, 1, 1, 1, 1, step < 9])
        _, q = s.grow(s.lens + i32(active), R)
        rows = torch.zeros(R, s.A, s.D, device="cuda")
        rows[torch.from_numpy(np.flatnonzero(active)).cuda()] = q[:int(active.sum())]
        got = s.shared(rows, start, prefix, 100)
        now = s.lens.tolist()
        want, _, tol, _ = lm.attention(rows.double().cpu().numpy(), *s.sections(), s.table.cpu().numpy(), now, page, scale, 0, s.max_len)
        close(got, want, tol + 2.0 ** -24 * np.abs(want), f"step {step}")
        if step == 5:                                # beam 2 of the first prompt goes on in all of its slots
            s.fork(i32([2, 2, 2, 3, 4, 5]), i32([now[2]] * 3 + now[3:]))
        if step == 9:                                # the last one ends
            assert s.fork(i32(range(R)), i32(now[:5] + [0]))["len"].tolist()[5] == 0
    before = s.paged(rows)
    held = {int(x) for r, n in enumerate(s.lens.tolist()) for x in s.table[r, :lm.ceil_div(n, page)].tolist()}
    free = s.state.tolist()[1]
    assert free + len(held) == s.pool                # no page lost or held twice over all of this
    v = s.compact()
    assert v["state"].tolist()[1] == s.pool - len(held) and v["state"].tolist()[3] == len(held)
    assert torch.equal(s.paged(rows), before)        # the same rows in other places
    assert torch.equal(s.shared(rows, start, prefix, 100), got)
    p, _ = s.grow(s.lens + 1, R)                     # and on
    assert p["state"].tolist()[3] == 0


def test_windows_over_the_same_cache():
    """A window with first tokens, in one call for prompts and single tokens; without sinks it is paged_attn's window."""
    s = Served(4, H=2, G=2, D=96, page=8, stride=40, pool=170, kind="bf16", tokens=300)
    s.grow(i32([300, 120, 1, 64]), 485)
    p, q = s.grow(s.lens + 1, 4)
    outs = {}
    for sinks in (0, 4):
        d = bq.prompt_desc(s.kv, s.A, 4, 4, s.stride, s.max_len, window=50, sinks=sinks, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
        ws = torch.empty(max(1, bq.prompt_attn_workspace(d)), dtype=torch.uint8, device="cuda")
        outs[sinks] = torch.empty(4, s.A, s.D, device="cuda")
        bq.prompt_attn(d, q, s.cache, s.table, p["start"], p["len"], outs[sinks], ws)
        want, _, tol, _ = ref.prompt(q.double().cpu().numpy(), s.sections(), s.table.cpu().numpy(), p["start"].tolist(), p["len"].tolist(),
                                     8, np.float32(s.D ** -0.5), 50, sinks, s.max_len, 3)
        close(outs[sinks], want, tol + 2.0 ** -24 * np.abs(want), f"sinks {sinks}")
    a = bq.attn_desc(s.kv, s.A, 4, s.stride, s.max_len, window=50, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
    ws = torch.empty(max(1, bq.paged_attn_workspace(a)), dtype=torch.uint8, device="cuda")
    one = torch.empty(4, s.A, s.D, device="cuda")
    bq.paged_attn(a, q, s.cache, s.table, s.lens, one, ws)
    want, _, tol, _ = lm.attention(q.double().cpu().numpy(), *s.sections(), s.table.cpu().numpy(), s.lens.tolist(), 8,
                                   np.float32(s.D ** -0.5), 50, s.max_len)
    assert torch.allclose(one, outs[0], rtol=0, atol=float(2 * tol.max()))


def test_on_a_side_stream_and_in_graphs_that_share_a_workspace():
    """Captured on a side stream, replayed with other work between: every replay equals the eager result."""
    say("serve graph")
    s = Served(5, H=2, G=4, D=64, page=16, stride=130, pool=700, kind="bf16", tokens=10)
    s.grow(i32([2000, 30, 700, 700, 16]), 3500)
    R, A, D = s.R, s.A, s.D
    T = 12
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(T, A + s.H, D, generator=g, device="cuda")
    qo, ko = torch.empty(T, A, D, device="cuda"), torch.empty(T, s.H, D, device="cuda")
    pos, start, lens = i32(range(T)), i32([0, 4, 4, 9, 10, 12]), s.lens.clone()
    rd = bq.rope_desc(T, A, s.H, D, x_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
    pd = bq.prompt_desc(s.kv, A, R, T, s.stride, s.max_len, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
    sd = bq.shared_desc(bq.attn_desc(s.kv, A, R, s.stride, s.max_len, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32), 2, 600)
    assert bq.prompt_attn_workspace(pd) > 0
    ws = torch.empty(max(bq.prompt_attn_workspace(pd), bq.shared_attn_workspace(sd)), dtype=torch.uint8, device="cuda")
    o1, l1 = torch.empty(T, A, D, device="cuda"), torch.empty(T, A, device="cuda")
    o2, l2 = torch.empty(R, A, D, device="cuda"), torch.empty(R, A, device="cuda")
    kd = bq.kv_pages_desc(R, 16, s.stride, 700, 700)
    bufs = [torch.empty(bq.kv_pages_size(kd), dtype=torch.uint8, device="cuda") for _ in range(2)]
    pws = torch.empty(bq.kv_pages_workspace(kd), dtype=torch.uint8, device="cuda")
    t2, t3, ring2 = (torch.full_like(y, -1) for y in (s.table, s.table, s.ring))
    src, keep = i32([2, 1, 2, 3, 0]), i32([500, 30, 700, 650, 1999])
    copy = s.cache.clone()

    def attention():
        bq.qk_rope(rd, x[:, :A], x[:, A:], *s.w, s.freq, pos, qo, ko)
        bq.prompt_attn(pd, qo, s.cache, s.table, start, lens, o1, ws, lse=l1)
        bq.shared_attn(sd, qo[:R], s.cache, s.table, lens, i32_start, i32_prefix, o2, ws, lse=l2)

    def paging():
        bq.kv_fork(kd, src, keep, lens, s.ring, s.state, s.table, t2, bufs[0], pws)
        v = bq.kv_pages_views(kd, bufs[0])
        bq.kv_copy(s.kv, v["frm"], v["to"], copy)
        bq.kv_compact(kd, v["len"], t2, t3, ring2, bufs[1], pws)

    i32_start, i32_prefix = i32([1, 4, 5]), i32([25, 16])
    outs = [qo, ko, o1, l1, o2, l2, t2, t3, s.ring, ring2, *bufs, copy]
    for f in (attention, paging):
        f()
    torch.cuda.synchronize()
    eager = [o.clone() for o in outs]
    graphs = []
    for f in (attention, paging):
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                f()
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(graph)
    for rep in range(4):
        for o in (qo, o1, l1, o2, l2):
            o.fill_(float("nan"))
        for o in (t2, t3, ring2):
            o.fill_(-1)
        ws.fill_(0x5A)
        pws.fill_(0x5A)
        torch.randn(1 << 18, device="cuda").sum().item()
        for graph in graphs if rep % 2 else graphs[::-1]:
            graph.replay()
        torch.cuda.synchronize()
        for i, (o, e) in enumerate(zip(outs, eager)):
            assert torch.equal(o.view(torch.uint8), e.view(torch.uint8)), f"replay {rep}, buffer {i}"


def test_two_streams_at_once():
    """Calls on two streams with workspaces of their own do not disturb each other, and repeat bit for bit."""
    s = Served(6, H=2, G=4, D=128, page=32, stride=64, pool=300, kind="int8", tokens=10)
    s.grow(i32([1500, 1500, 1800, 10, 700, 1]), 6000)
    q = torch.randn(6, s.A, s.D, generator=s.g, device="cuda")
    start, prefix = i32([0, 3, 6]), i32([1400, 0])
    want = s.shared(q, start, prefix, 1400)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(10):
        for st in streams:
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(s.shared(q, start, prefix, 1400))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
