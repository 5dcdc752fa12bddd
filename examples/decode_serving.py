"""A small decoder served with packed layers, a paged cache and an int8 head.

    python examples/decode_serving.py [--requests 6] [--steps 40] [--pages 13]

Random weights of a toy shape.  Each step every active request feeds one token: the plan gives it a slot in the paged
cache, the blocks' linear layers run on 2-bit weights with int8 activations (bitq_gemm_smallM), keys and values go to
the cache, attention reads the pages, the residual stream passes the norms before and after each block, and the head is
an int8 product on the rows that the last norm quantized.  Requests begin and end at different steps; their pages go
back to the ring and are used again.  A request that the plan refuses for want of pages asks again with the same token,
and the last request of the batch gives its pages up and begins anew.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_plane_gemv_amd as bq  # noqa: E402

WIDTH, HEADS, KV_HEADS, DIM, FFN, VOCAB, LAYERS = 512, 8, 2, 64, 1024, 1000, 2
PAGE, MAX_LEN = 16, 64
RES, BRANCH, EPS = 1.0, 0.5, 1e-5


class Packed:
    """y = x W^T with W2A8 weights: fp32 rows in and out, 2 to 64 of them."""

    def __init__(self, rng, N, K, rows):
        self.N, self.K = N, K
        self.desc = bq.wdesc("w2a8", N, K)
        W = (rng.standard_normal((N, K)) * K ** -0.5).astype(np.float32)
        self.w = torch.from_numpy(bq.quantize_weights(self.desc, W)).cuda()
        self.act = torch.empty(bq.act_size(rows, K), dtype=torch.uint8, device="cuda")
        self.y = torch.empty(rows, N, device="cuda")

    def __call__(self, x):
        bq.quantize_act(x, bq.DT_F32, x.shape[0], self.K, self.act)
        bq.gemm_smallM(self.desc, self.w, self.act, x.shape[0], self.y, None)
        return self.y


class Server:
    """`requests` slots (2 to 64), each holding one request at a time; `pages` pages of the cache for all of them (at least
    those of one request)."""

    def __init__(self, requests, seed=0, pages=None):
        rng = np.random.default_rng(seed)
        R = self.R = requests
        f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
        self.emb, self.pos_emb = f(VOCAB, WIDTH), 0.1 * f(MAX_LEN, WIDTH)
        self.layers = [dict(qkv=Packed(rng, (HEADS + 2 * KV_HEADS) * DIM, WIDTH, R), o=Packed(rng, WIDTH, HEADS * DIM, R),
                            up=Packed(rng, FFN, WIDTH, R), down=Packed(rng, WIDTH, FFN, R),
                            post=[1 + 0.1 * f(WIDTH) for _ in range(2)], pre=[1 + 0.1 * f(WIDTH) for _ in range(2)],
                            gate=[f(WIDTH) for _ in range(2)]) for _ in range(LAYERS)]
        self.first = 1 + 0.1 * f(WIDTH)                       # the norm before the first block
        head = (0.02 * f(VOCAB, WIDTH)).contiguous()          # the head in int8, a scale per channel
        self.head, self.head_scale = torch.empty(VOCAB, WIDTH, dtype=torch.int8, device="cuda"), torch.empty(VOCAB, device="cuda")
        bq.block_norm(bq.norm_desc(VOCAB, WIDTH, out_dtype=bq.DT_ROW8), head, None, None, None, None, None, self.head,
                      self.head_scale)
        # the cache: one pool of pages per layer, one table and one ring for all layers
        self.stride = MAX_LEN // PAGE
        # (by default half of what every request at full length would need, which is what serve() asks for at most)
        self.pages = R * self.stride // 2 + 1 if pages is None else pages
        self.kv = bq.kvdesc(KV_HEADS, DIM, PAGE, self.pages)
        self.caches = [torch.empty(bq.kv_cache_size(self.kv), dtype=torch.uint8, device="cuda") for _ in range(LAYERS)]
        self.table = torch.full((R, self.stride), -1, dtype=torch.int32, device="cuda")
        self.ring = torch.arange(self.pages, dtype=torch.int32, device="cuda")
        self.plan = bq.kv_plan_desc(R, PAGE, self.stride, self.pages, R)
        self.bufs = [torch.zeros(bq.kv_plan_size(self.plan), dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.views = [bq.kv_plan_views(self.plan, b) for b in self.bufs]
        self.views[0]["state"].copy_(torch.tensor([0, self.pages, 0, 0]))
        self.turn = 0
        self.attn = bq.attn_desc(self.kv, HEADS, R, self.stride, MAX_LEN, q_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
        self.ws = torch.empty(max(1, bq.paged_attn_workspace(self.attn)), dtype=torch.uint8, device="cuda")
        self.norm = bq.norm_desc(R, WIDTH, res_scale=RES, branch_scale=BRANCH, eps_post=EPS, eps_pre=EPS)
        self.last = bq.norm_desc(R, WIDTH, out_dtype=bq.DT_ROW8, res_scale=RES, branch_scale=BRANCH, eps_post=EPS, eps_pre=EPS)
        self.att, self.h = torch.empty(R, HEADS, DIM, device="cuda"), torch.empty(R, WIDTH, device="cuda")
        self.q8, self.q8_scale = torch.empty(R, WIDTH, dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
        self.logits = torch.empty(R, VOCAB, device="cuda")
        self.product = bq.w8a8_desc(R, VOCAB, WIDTH)

    def step(self, tokens, active):
        """Feed tokens[r] to every slot r with active[r] == 1; active[r] == 0 ends its request.  Both int32 on the GPU.
        Returns logits [R][VOCAB] and the lengths after the step (a request refused for want of pages keeps its own)."""
        old = self.views[self.turn]
        now = self.views[1 - self.turn]
        new = torch.where(active > 0, old["len"] + 1, 0)
        bq.kv_plan(self.plan, old["len"], new, self.ring, old["state"], self.table, self.bufs[1 - self.turn])
        self.turn = 1 - self.turn
        # the plan lists new tokens in request order; here every request has at most one: row r = request r
        start, slot = now["start"], now["slot"]
        slots = torch.where(start[1:] > start[:-1], slot[start[:-1].clamp(max=self.R - 1).long()], -1)
        pos = (now["len"] - 1).clamp(min=0).long()
        r = (self.emb[tokens.long()] + self.pos_emb[pos]).contiguous()
        h = self.h
        bq.block_norm(self.norm, r, None, None, None, self.first, None, h)
        for i, layer in enumerate(self.layers):
            qkv = layer["qkv"](h).view(self.R, HEADS + 2 * KV_HEADS, DIM)
            k, v = qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
            bq.kv_write(self.kv, k, v, bq.DT_F32, slots, self.caches[i])
            bq.paged_attn(self.attn, qkv, self.caches[i], self.table, now["len"], self.att, self.ws)
            u = layer["o"](self.att.view(self.R, HEADS * DIM))
            bq.block_norm(self.norm, u, r, layer["post"][0], layer["gate"][0], layer["pre"][0], r, h)
            u = layer["down"](torch.nn.functional.silu(layer["up"](h)))
            if i + 1 < LAYERS:
                bq.block_norm(self.norm, u, r, layer["post"][1], layer["gate"][1], layer["pre"][1], r, h)
            else:
                bq.block_norm(self.last, u, r, layer["post"][1], layer["gate"][1], layer["pre"][1], r, self.q8, self.q8_scale)
        bq.gemm_w8a8(self.product, self.q8, self.q8_scale, self.head, self.head_scale, self.logits)
        return self.logits, now["len"]


def serve(requests, steps, seed=0, follow=None, pages=None):
    """Requests of random lengths on `requests` slots, each continuing with its own most likely token.  follow(server,
    tokens, active, logits, lengths) is called after each step.  Returns the number of tokens served (written to the cache
    and attended) and of requests ended."""
    server = Server(requests, seed, pages)
    rng = np.random.default_rng(seed + 1)
    total = rng.integers(1, MAX_LEN // 2, requests)           # tokens of each slot's request, its first one,
    first = torch.from_numpy(rng.integers(0, VOCAB, requests).astype(np.int32)).cuda()
    left, tokens = total.copy(), first                        # those to come and the next one
    held, yields = np.zeros(requests, int), np.zeros(requests, bool)
    served = ended = 0
    for _ in range(steps):
        active = (left > 0) & ~yields
        act = torch.from_numpy(active.astype(np.int32)).cuda()
        fresh = torch.from_numpy(rng.integers(0, VOCAB, requests).astype(np.int32)).cuda()
        logits, lengths = server.step(tokens, act)
        if follow:
            follow(server, tokens, act, logits, lengths)
        now = lengths.cpu().numpy()
        written = active & (now > held)                       # the other active ones were refused
        served += int(written.sum())
        done = ~active & ~yields                              # an ended slot takes a new request
        ended += int(done.sum())
        total = np.where(done, rng.integers(1, MAX_LEN // 2, requests), total)
        left = np.where(written, left - 1, np.where(active, left, total))
        dev = lambda m: torch.from_numpy(m).cuda()  # noqa: E731
        first = torch.where(dev(done), fresh, first)
        tokens = torch.where(dev(written), logits.argmax(1).to(torch.int32), torch.where(dev(active), tokens, first))
        # the plan serves requests in order and stops at the first that does not fit: unless a request ends by itself, the
        # last one makes room, so the first one always goes on
        yields = np.zeros(requests, bool)
        going = np.flatnonzero(active & (left > 0))
        if (active & ~written).any() and len(going) == active.sum() > 1:
            yields[going[-1]] = True
        held = now
    return served, ended


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=6)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--pages", type=int, help="pages of each layer's cache")
    a = ap.parse_args()
    served, ended = serve(a.requests, a.steps, pages=a.pages)
    torch.cuda.synchronize()
    pages = Server(a.requests, pages=a.pages).pages
    print(f"{served} tokens served, {ended} requests ended, {a.requests} slots, {pages} pages per layer")
