"""README.md: its decode step, run as it stands."""
import os
import re

import pytest

import bit_plane_gemv_amd as bq
from gpuhelp import say

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_decode_step_of_the_readme():
    """With an idle and a refused request among the others, every request's keys, values and output are its own."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    say("readme decode step")
    with open(README) as f:
        code = next(b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "kv_plan(" in b)
    g = torch.Generator(device="cuda").manual_seed(3)
    R, H, heads, D, page, table_stride, ring_len, max_len = 5, 8, 16, 128, 16, 4, 30, 64
    dev = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    old_lens, new_lens = dev(0, 0, 0, 64, 0), dev(1, 0, 1, 65, 1)        # request 1 is idle, request 3 longer than its table
    ring, state = torch.arange(ring_len, dtype=torch.int32, device="cuda"), dev(0, 20)
    table = torch.arange(20, 20 + R * table_stride, dtype=torch.int32, device="cuda").view(R, table_stride)
    k, v = (torch.randn(R, H, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(R, heads, D, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    plan = torch.empty(bq.kv_plan_size(bq.kv_plan_desc(R, page, table_stride, ring_len, R)), dtype=torch.uint8, device="cuda")
    kv = bq.kvdesc(H, D, page, 4096)
    ws = torch.empty(max(1, bq.paged_attn_workspace(bq.attn_desc(kv, heads, R, table_stride, max_len))), dtype=torch.uint8, device="cuda")
    names = dict(torch=torch, bq=bq, R=R, table_stride=table_stride, ring_len=ring_len, old_lens=old_lens, new_lens=new_lens,
                 ring=ring, state=state, table=table, plan=plan, k=k, v=v, heads=heads, max_len=max_len, q=q, out=out, ws=ws)
    exec(code, names)
    torch.cuda.synchronize()
    assert names["p"]["state"].tolist()[2:] == [3, 1]
    for r in (0, 2, 4):                              # one token each: its value is the output, whatever the score
        assert torch.equal(out[r].view(H, -1, D), v[r][:, None].expand(H, heads // H, D)), r
    assert bool((out[1] == 0).all())
