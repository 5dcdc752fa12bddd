"""examples/decode_serving.py: the attention outputs that the server itself used, in every layer, and requests that have to
wait for pages."""
import importlib.util
import os

import pytest

from gpuhelp import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def example():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("decode_serving", os.path.join(ROOT, "examples", "decode_serving.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("requests,steps,pages", [(6, 80, 7), (5, 60, 2), (2, 60, None), (9, 70, 10)])
def test_requests_that_wait_lose_no_token(example, requests, steps, pages):
    """Every token that reaches the cache is the request's first or the most likely one after the token before it, whether
    or not the request had to wait for a page in between; only written tokens are counted."""
    say("serving pages", requests, steps, pages)
    m = example
    length, pending = [0] * requests, [None] * requests
    counts = dict(written=0, refused=0, ended=0, waited=0)

    def follow(s, tokens, active, logits, lengths):
        fed, best = tokens.tolist(), logits.argmax(1).tolist()
        for r, (n, act) in enumerate(zip(lengths.tolist(), active.tolist())):
            if not act:
                assert n == 0
                length[r], pending[r] = 0, None
                counts["ended"] += 1
                continue
            if pending[r] is not None:
                assert fed[r] == pending[r], (r, length[r])
            if n == length[r]:
                counts["refused"] += 1
                pending[r] = fed[r]                      # it asks again with the same token
            else:
                assert n == length[r] + 1
                counts["written"] += 1
                counts["waited"] += length[r] > 0 and pending[r] is not None and refused[r]
                pending[r] = best[r]
            refused[r] = n == length[r]
            length[r] = n
        used = [x for r in range(requests) for x in s.table[r, :-(-length[r] // m.PAGE)].tolist()]
        assert len(set(used)) == len(used), "a page belongs to two requests"

    refused = [False] * requests
    served, ended = m.serve(requests, steps, follow=follow, pages=pages)
    assert served == counts["written"] and ended > 0 and ended <= counts["ended"]
    if pages is None:
        assert counts["refused"] == 0 and ended == counts["ended"]
    else:
        assert counts["refused"] > 0 and ended < counts["ended"]      # some gave their pages up
        assert pages == 2 or counts["waited"] > 0                     # and some went on after waiting


@pytest.mark.parametrize("requests,steps,max_len,pages", [(6, 45, None, None), (6, 40, None, 7), (4, 420, 2048, None)])
def test_attention_that_the_server_used(example, monkeypatch, requests, steps, max_len, pages):
    """Every layer's attention output of the server's own calls against a dense computation in 64 bits over the keys and
    values of its own writes; the last case splits the requests' tokens over workgroups."""
    import torch
    say("serving attention", requests, steps, max_len, pages)
    m = example
    if max_len:
        monkeypatch.setattr(m, "MAX_LEN", max_len)
    writes, calls = [], []
    write, attend = m.bq.kv_write, m.bq.paged_attn

    def kv_write(kv, k, v, *a, **kw):
        writes.append((k.to(torch.bfloat16).double(), v.to(torch.bfloat16).double()))
        write(kv, k, v, *a, **kw)

    def paged_attn(d, q, cache, table, lens, out, ws, **kw):
        attend(d, q, cache, table, lens, out, ws, **kw)
        calls.append((q[:, :m.HEADS].double(), out.double()))

    monkeypatch.setattr(m.bq, "kv_write", kv_write)
    monkeypatch.setattr(m.bq, "paged_attn", paged_attn)
    history = [[[] for _ in range(requests)] for _ in range(m.LAYERS)]
    checked = step = longest = 0

    def follow(s, tokens, active, logits, lengths):
        nonlocal checked, step, longest
        assert len(writes) == len(calls) == m.LAYERS
        assert not max_len or m.bq.paged_attn_workspace(s.attn) > 0          # split
        for h, (k, v), (q, out) in zip(history, writes, calls):
            for r, n in enumerate(lengths.tolist()):
                if n == len(h[r]) + 1:
                    h[r].append((k[r], v[r]))
                elif n != len(h[r]):
                    assert n == 0
                    h[r].clear()
                if n == 0 or (max_len and step % 16):
                    continue
                longest = max(longest, n)
                K, V = (torch.stack(x, 1) for x in zip(*h[r]))               # [KV_HEADS][n][DIM]
                p = torch.softmax(torch.matmul(q[r].view(m.KV_HEADS, -1, m.DIM), K.transpose(1, 2).contiguous()) * m.DIM ** -0.5, -1)
                want = torch.matmul(p, V).view(m.HEADS, m.DIM)
                # scores of a few units in fp32 (sums of 64 products), weights and sums to match
                assert float((out[r] - want).abs().max()) < 2.0 ** -24 * 64 * 16 * float(V.abs().max()), (r, n)
                checked += 1
        step += 1
        writes.clear()
        calls.clear()

    m.serve(requests, steps, follow=follow, pages=pages)
    assert checked > 50 and (not max_len or longest > 256)
