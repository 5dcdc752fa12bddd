"""examples/decode_serving.py: every step of the served batch against a dense recomputation of each request."""
import importlib.util
import os

import pytest

from gpuhelp import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("decode_serving", os.path.join(ROOT, "examples", "decode_serving.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("requests,steps", [(2, 12), (6, 45)])
def test_served_attention_and_norms_match_a_dense_history(example, requests, steps):
    """The first layer's keys and values of every request are kept aside, as bf16 rounds them: its attention over the
    pages is recomputed from them densely, and the head's logits from the rows that the last norm quantized."""
    import torch
    say("serving example", requests, steps)
    m = example
    history = {}
    checked = 0
    refused = 0

    def follow(s, tokens, active, logits, lengths):
        nonlocal checked, refused
        layer = s.layers[0]
        lens, act = lengths.tolist(), active.tolist()
        pos = (lengths - 1).clamp(min=0).long()
        r0 = s.emb[tokens.long()] + s.pos_emb[pos]
        h0 = (r0.double() / torch.sqrt(r0.double().square().mean(1, keepdim=True) + m.EPS) * s.first.double()).float()
        qkv = layer["qkv"](h0.contiguous()).clone().view(s.R, -1, m.DIM)
        first = torch.empty(s.R, m.HEADS, m.DIM, device="cuda")     # (s.att holds the last layer's)
        m.bq.paged_attn(s.attn, qkv, s.caches[0], s.table, lengths, first, s.ws)
        for r in range(s.R):
            old = history.get(r, [])
            if not act[r]:
                assert lens[r] == 0
                history[r] = []
                continue
            if lens[r] == len(old):                       # no page was left: nothing was written
                refused += 1
                continue
            assert lens[r] == len(old) + 1
            history[r] = old + [qkv[r, m.HEADS:].to(torch.bfloat16).double().cpu()]
            kv = torch.stack(history[r])                  # [n][2 KV_HEADS][DIM]
            q = qkv[r, :m.HEADS].double().cpu().view(m.KV_HEADS, -1, m.DIM)
            k, v = kv[:, :m.KV_HEADS].transpose(0, 1), kv[:, m.KV_HEADS:].transpose(0, 1)
            p = torch.softmax(torch.matmul(q, k.transpose(1, 2)) * m.DIM ** -0.5, -1)
            want = torch.matmul(p, v).reshape(m.HEADS, m.DIM)
            # h0 is rounded apart from the server's: activation codes may differ by one, so keys and values agree
            # to about 1 %
            got = first[r].double().cpu()
            assert float((got - want).norm() / want.norm()) < 0.03, (r, lens[r])
            checked += 1
        y = s.q8.double() * s.q8_scale.double()[:, None] @ (s.head.double() * s.head_scale.double()[:, None]).t()
        assert torch.allclose(logits.double(), y, rtol=1e-5, atol=1e-6)
        used = [int(x) for r in range(s.R) for x in s.table[r, :-(-lens[r] // m.PAGE)].tolist()]
        assert len(set(used)) == len(used), "a page belongs to two requests"

    served, ended = m.serve(requests, steps, follow=follow)
    assert checked > 0 and checked + refused == served
    if steps > m.MAX_LEN // 2:
        assert ended > 0
