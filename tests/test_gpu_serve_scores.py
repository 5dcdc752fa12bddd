"""prompt_attn and shared_attn where scores are large: whatever a finite score is, the largest one takes all the weight."""
import numpy as np
import pytest
import torch

import bit_plane_gemv_amd as bq
import lm_reference as lm
import serve_reference as ref
from gpuhelp import say
from test_gpu_serve_attention import DT, close, tables, upload

pytestmark = pytest.mark.gpu
D, PAGE = 64, 16
# scale, and the factor of q.  (Scores reach 90 scale factor log2(e): with the last ones just below the largest float.)
LARGE = [(1e9, 1), (-1e9, 1), (1e10, 1), (-1e30, 1), (2.0e36, 1), (-2.0e36, 1), (0.125, 2.0 ** 40), (0.125, 2.0 ** 110)]


def sections_of(pool, lens, table, H, int8, rng):
    """Random values; of the keys element 0 alone, different integers for tokens that are different modulo 181: the places of a
    random order, so that running maxima grow again and again."""
    K, V, ks, vs = lm.cache_sections(pool, H, PAGE, D, int8, rng)
    K.zero_()
    g = np.stack([rng.permutation(181) - 90 for _ in range(H)])
    for r, n in enumerate(lens):
        for t in range(n):
            K[int(table[r, t // PAGE]), :, t % PAGE, 0] = torch.from_numpy(g[:, t % 181]).to(K.dtype)
    if int8:
        ks.fill_(1.0)
    return (K, V, ks, vs), g


def check(out, lse, q0, top, scale, V, vs, table_of, otype, G):
    """The output is the value of the token that scores highest (others are at least 1e8 below it).  Its weight is the only one:
    p and sum p are the same number, so the output is off by the product's, the reciprocal's and its factor's rounding (4 x
    2^-24) and its own; the log-sum by those of the score: two of its factor, the product, the maximum's, and ln 2 (6 x 2^-24)."""
    rows, A = q0.shape
    want, wl = np.zeros((rows, A, D)), np.zeros((rows, A))
    for i in range(rows):
        for h in range(A):
            t, x = top(i, h)
            p, o = table_of(i, t)
            v = V[p, h // G, o // 8, :D, o % 8].double().numpy()
            want[i, h] = v if vs is None else v * float(vs[p, h // G, o])
            wl[i, h] = float(np.float32(scale)) * x
    tol = 4 * 2.0 ** -24 * np.abs(want)
    close(out, want, tol + ref.half_step(otype) * (np.abs(want) + tol), "out")
    close(lse, wl, 6 * 2.0 ** -24 * np.abs(wl), "lse")


def queries(rows, A, factor, dt, rng):
    q = np.zeros((rows, A, D), dtype=np.float32)
    q[..., 0] = rng.choice([-1.0, 1.0], (rows, A)) * factor
    return torch.from_numpy(q).to(dt).cuda(), q[..., 0].astype(np.float64)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("new,length,G", [(1, 1, 4), (2, 2, 4), (1, 90, 4), (1, 1500, 4), (5, 170, 4), (70, 170, 4)])
@pytest.mark.parametrize("scale,factor", LARGE)
def test_prompt_largest_score_takes_all(scale, factor, new, length, G, dt, kind):
    rng = np.random.default_rng(length)
    H, lens = 2, [length]
    table, pool = tables(lens, PAGE, length // PAGE + 1, rng)
    length_seen = min(length, 181)                   # (the same integers again further on: cut them off, below)
    sections, g = sections_of(pool, lens, table, H, kind == "int8", rng)
    for t in range(181, length):                     # further tokens score 0
        sections[0][int(table[0, t // PAGE]), :, t % PAGE] = 0
    kv = bq.kvdesc(H, D, PAGE, pool, bq.KV_INT8 if kind == "int8" else bq.KV_BF16)
    q, q0 = queries(new, H * G, factor, DT[dt][1], rng)
    d = bq.prompt_desc(kv, H * G, 1, new, table.shape[1], length, q_dtype=DT[dt][0], out_dtype=DT[dt][0], scale=scale)
    ws = torch.empty(max(1, bq.prompt_attn_workspace(d)), dtype=torch.uint8, device="cuda")
    out, lse = torch.full((new, H * G, D), 7.0, dtype=DT[dt][1], device="cuda"), torch.full((new, H * G), 7.0, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    say("prompt large scores", scale, factor, new, length, G, dt, kind, "workspace", ws.numel())
    bq.prompt_attn(d, q, upload(sections, kv), torch.from_numpy(table).cuda(), i32([0, new]), i32(lens), out, ws, lse=lse)

    def top(i, h):
        n = min(length - new + i + 1, length_seen)
        x = q0[i, h] * g[h // G][:n]
        t = int(np.argmax(x * np.sign(scale)))
        return t, x[t]
    check(out, lse, q0, top, scale, sections[1], sections[3], lambda i, t: (int(table[0, t // PAGE]), t % PAGE), DT[dt][1], G)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,G", [(3, 4), (40, 4)])
@pytest.mark.parametrize("scale,factor", LARGE)
def test_shared_largest_score_takes_all(scale, factor, R, G, dt, kind):
    rng = np.random.default_rng(R)
    H, lens = 2, rng.integers(60, 181, R).tolist()
    table, pool = tables(lens, PAGE, 12, rng)
    sections, g = sections_of(pool, lens, table, H, kind == "int8", rng)
    prefix = 50
    for r in range(R):                               # whole pages of the prefix are the first request's
        table[r, :prefix // PAGE] = table[0, :prefix // PAGE]
    for t in range(prefix // PAGE * PAGE, prefix):   # and the rest of it is read there
        for r in range(1, R):
            for x in sections[1::2]:
                if x is not None:
                    a = (slice(None), t % PAGE // 8, slice(None), t % PAGE % 8) if x.dim() == 5 else (slice(None), t % PAGE)
                    x[(int(table[r, t // PAGE]),) + a] = x[(int(table[0, t // PAGE]),) + a]
    kv = bq.kvdesc(H, D, PAGE, pool, bq.KV_INT8 if kind == "int8" else bq.KV_BF16)
    q, q0 = queries(R, H * G, factor, DT[dt][1], rng)
    d = bq.shared_desc(bq.attn_desc(kv, H * G, R, 12, 181, q_dtype=DT[dt][0], out_dtype=DT[dt][0], scale=scale), 1, 64)
    ws = torch.empty(bq.shared_attn_workspace(d), dtype=torch.uint8, device="cuda")
    out, lse = torch.full((R, H * G, D), 7.0, dtype=DT[dt][1], device="cuda"), torch.full((R, H * G), 7.0, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    say("shared large scores", scale, factor, R, G, dt, kind, "workspace", ws.numel())
    bq.shared_attn(d, q, upload(sections, kv), torch.from_numpy(table).cuda(), i32(lens), i32([0, R]), i32([prefix]), out, ws, lse=lse)

    def top(i, h):
        x = q0[i, h] * g[h // G][:lens[i]]
        t = int(np.argmax(x * np.sign(scale)))
        return t, x[t]
    check(out, lse, q0, top, scale, sections[1], sections[3], lambda i, t: (int(table[i, t // PAGE]), t % PAGE), DT[dt][1], G)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("new", [2, 40])
def test_prompt_rows_beside_one_of_large_scores_keep_their_bits(new, dt, kind):
    rng = np.random.default_rng(new)
    H, G, lens = 2, 4, [200]
    table, pool = tables(lens, PAGE, 13, rng)
    sections = lm.cache_sections(pool, H, PAGE, D, kind == "int8", rng)
    kv = bq.kvdesc(H, D, PAGE, pool, bq.KV_INT8 if kind == "int8" else bq.KV_BF16)
    cache = upload(sections, kv)
    q = torch.from_numpy(rng.standard_normal((new, H * G, D)).astype(np.float32)).to(DT[dt][1])
    d = bq.prompt_desc(kv, H * G, 1, new, 13, 200, q_dtype=DT[dt][0], out_dtype=DT[dt][0])
    ws = torch.empty(max(1, bq.prompt_attn_workspace(d)), dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    say("prompt one row of large scores", new, dt, kind)
    got = []
    for factor in (1.0, 1e20):
        x = q.clone()
        x[new // 2, 1] *= factor
        out, lse = torch.full((new, H * G, D), 7.0, dtype=DT[dt][1], device="cuda"), torch.full((new, H * G), 7.0, device="cuda")
        bq.prompt_attn(d, x.cuda(), cache, torch.from_numpy(table).cuda(), i32([0, new]), i32(lens), out, ws, lse=lse)
        out[new // 2, 1], lse[new // 2, 1] = 0, 0
        got.append((out, lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 40])
def test_prompt_largest_values(new, dt):
    """64 tokens and values of 2^113: their product is the 2^119 that sums before the division may take."""
    rng = np.random.default_rng(new)
    H, G, lens = 2, 4, [64]
    table, pool = tables(lens, PAGE, 4, rng)
    K, V, ks, vs = lm.cache_sections(pool, H, PAGE, D, False, rng)
    V = (torch.sign(V.float()) * 2.0 ** 113).bfloat16()
    kv = bq.kvdesc(H, D, PAGE, pool)
    q = torch.from_numpy(rng.standard_normal((new, H * G, D)).astype(np.float32) * 4).to(DT[dt][1])
    d = bq.prompt_desc(kv, H * G, 1, new, 4, 64, q_dtype=DT[dt][0], out_dtype=DT[dt][0])
    ws = torch.empty(max(1, bq.prompt_attn_workspace(d)), dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full((new, H * G, D), 7.0, dtype=DT[dt][1], device="cuda")
    say("prompt largest values", new, dt)
    bq.prompt_attn(d, q.cuda(), upload((K, V, ks, vs), kv), torch.from_numpy(table).cuda(), i32([0, new]), i32(lens), out, ws)
    want, _, tol, _ = ref.prompt(q.double().numpy(), (K, V, ks, vs), table, [0, new], lens, PAGE, np.float32(D ** -0.5), 0, 0, 64, 3)
    close(out, want, tol + ref.half_step(DT[dt][1]) * (np.abs(want) + tol), "out")
