"""README.md: its prompts and shared pages, run as they stand."""
import os
import re

import numpy as np
import pytest

import bit_plane_gemv_amd as bq
import serve_reference as ref
from gpuhelp import say

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_prompts_of_the_readme():
    """Three prompts; then the second request becomes a fork of the first and the third one ends."""
    import torch
    say("readme prompts")
    with open(README) as f:
        code = next(b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "rope_table(" in b)
    g = torch.Generator(device="cuda").manual_seed(5)
    lens = [20, 5, 33]
    R, H, heads, head_dim, page, table_stride, pool, max_len = 3, 2, 4, 64, 16, 4, 12, 64
    T = sum(lens)
    dev = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    u8 = lambda n: torch.zeros(max(1, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    kv = bq.kvdesc(H, head_dim, page, pool)
    ring, table = torch.arange(pool, dtype=torch.int32, device="cuda"), torch.zeros(R, table_stride, dtype=torch.int32, device="cuda")
    pd = bq.kv_plan_desc(R, page, table_stride, pool, T)
    plan = u8(bq.kv_plan_size(pd))
    bq.kv_plan(pd, dev(0, 0, 0), dev(*lens), ring, dev(0, pool), table, plan)
    q, k, v = (torch.randn(T, n, head_dim, generator=g, device="cuda") for n in (heads, H, H))    # one projection's, in fp32
    q_w, k_w = (torch.rand(head_dim, generator=g, device="cuda") + 0.5 for _ in range(2))
    q_out, k_out = (torch.empty(T, n, head_dim, dtype=torch.bfloat16, device="cuda") for n in (heads, H))
    out, cache = torch.empty_like(q_out), u8(bq.kv_cache_size(kv))
    ws = u8(bq.prompt_attn_workspace(bq.prompt_desc(kv, heads, R, T, table_stride, max_len)))
    fd = bq.kv_pages_desc(R, page, table_stride, pool, R)
    names = dict(torch=torch, bq=bq, R=R, T=T, heads=heads, head_dim=head_dim, kv=kv, q=q, k=k, v=v, q_w=q_w, k_w=k_w, q_out=q_out,
                 k_out=k_out, p=bq.kv_plan_views(pd, plan), cache=cache, table=table, table_stride=table_stride, max_len=max_len,
                 out=out, ws=ws, src=dev(0, 0, 2), keep=dev(20, 20, 0), ring=ring, table_out=torch.zeros_like(table),
                 result=u8(bq.kv_pages_size(fd)), fork_ws=u8(bq.kv_pages_workspace(fd)))
    exec(code, names)
    torch.cuda.synchronize()
    views = {n: x.cpu() for n, x in bq.kv_cache_views(kv, cache).items() if x is not None}
    at = 0
    for r, n in enumerate(lens):                     # the keys as they were turned, and the projection's values
        for t in range(n):
            page_of = int(table[r, t // page])
            assert torch.equal(views["K"][page_of, :, t % page, :head_dim], k_out[at].cpu())
            assert torch.equal(views["V"][page_of, :, t % page // 8, :head_dim, t % 8], v[at].bfloat16().cpu())
            at += 1
    want, _, tol, _ = ref.prompt(q_out.double().cpu().numpy(), (views["K"], views["V"], None, None), table.cpu().numpy(),
                                 np.cumsum([0] + lens), lens, page, np.float32(head_dim ** -0.5), 0, 0, max_len, 3)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol))
    f = names["f"]
    assert f["len"].tolist() == [20, 20, 0] and f["state"].tolist()[2:] == [1, 0]
    a, b = names["table_out"][:2, :2].tolist()
    assert a == table[0, :2].tolist() and b[0] == a[0] and b[1] != a[1]      # the whole page is shared, the other one copied
    assert torch.equal(views["K"][a[1]], views["K"][b[1]]) and torch.equal(views["V"][a[1]], views["V"][b[1]])
