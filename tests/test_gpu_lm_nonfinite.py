"""Infinities, NaN and the smallest numbers through the int8 rows of the cache write and the block norm, and through
attention: what is not finite stays so."""
import math

import numpy as np
import pytest

import bit_plane_gemv_amd as bq
import lm_reference as ref
from gpuhelp import say

pytestmark = pytest.mark.gpu
ODD = [math.nan, math.inf, -math.inf, -math.nan]


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("T,H,D,f32,runs", [
    (5, 2, 64, True, False), (40, 3, 33, False, False),                   # a token a thread
    (1400, 8, 128, False, True), (2600, 4, 96, True, True),               # 8 tokens a thread, whole groups
    (16000, 2, 72, False, False), (3001, 3, 250, True, True),             # and groups that are not whole
])
def test_int8_write_keeps_what_is_not_finite(T, H, D, f32, runs):
    """A row with an infinity or NaN stands for NaN in every element; the other rows, among them rows whose 127/amax
    overflows, are those of the reference."""
    import torch
    say("write nonfinite", T, H, D, f32, runs)
    rng = np.random.default_rng(T + D)
    page = 16
    pages = ref.ceil_div(T, page) + 3
    slots = (np.arange(T) + 5 if runs else rng.permutation(pages * page)[:T]).astype(np.int32)
    x = torch.from_numpy(rng.standard_normal((T, 2, H, D)).astype(np.float32))
    x[0, 0, 0], x[1, 1, 0] = 0, 0
    x[0, 0, 0, :3] = torch.tensor([0.0, 1e-38, -2e-39])
    x[1, 1, 0, -2:] = torch.tensor([-1e-40, 0.0])
    if not f32:
        x = x.to(torch.bfloat16)
    bad = torch.zeros(T, 2, H, dtype=torch.bool)
    for i in range(min(60, T * H)):
        t, n, h = int(rng.integers(2, T)), int(rng.integers(2)), int(rng.integers(H))
        x[t, n, h, int(rng.integers(D))] = ODD[i % 4]
        bad[t, n, h] = True
    kv = bq.kvdesc(H, D, page, pages, bq.KV_INT8)
    cache = torch.zeros(bq.kv_cache_size(kv), dtype=torch.uint8, device="cuda")
    xd = x.cuda()
    bq.kv_write(kv, xd[:, 0], xd[:, 1], bq.DT_F32 if f32 else bq.DT_BF16, torch.from_numpy(slots).cuda(), cache)
    torch.cuda.synchronize()
    got = {n: t.cpu() for n, t in bq.kv_cache_views(kv, cache).items()}
    want = {n: torch.zeros_like(t) for n, t in got.items()}
    small = torch.zeros_like(bad)
    small[0, 0, 0] = small[1, 1, 0] = True           # (set by hand below)
    ref.write(*want.values(), *torch.where((bad | small)[..., None], 0.0, x.float()).unbind(1), slots, page)
    p, off = torch.from_numpy(slots // page).long(), torch.from_numpy(slots % page).long()
    k, v = got["K"][p, :, off], got["V"].transpose(-1, -2).reshape(got["K"].shape)[p, :, off]
    wk, wv = want["K"][p, :, off], want["V"].transpose(-1, -2).reshape(got["K"].shape)[p, :, off]
    for n, (q, wq, s, ws) in enumerate(((k, wk, got["ks"], want["ks"]), (v, wv, got["vs"], want["vs"]))):
        s, ws, odd = s[p, :, off], ws[p, :, off], bad[:, n]
        wq[n, 0, :D] = 127 * torch.sign(x[n, n, 0].float())
        ws[n, 0] = float(np.float32(x[n, n, 0].float().abs().amax().item()) / np.float32(127))
        assert bool(torch.isnan(q.float() * s[..., None])[..., :D][odd].all()), "a row that is not finite lost it"
        assert torch.equal(q[~odd], wq[~odd]) and torch.equal(s[~odd], ws[~odd])


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens", [[40, 33, 700], [40, 2500, 3]])
def test_attention_over_rows_that_are_not_finite(int8, lens):
    """NaN in a request's own keys or values: NaN in what reads it, and nowhere else."""
    import torch
    from test_gpu_lm import attention_case, run_attention
    say("attn nonfinite", int8, lens)
    rng = np.random.default_rng(31)
    H, G, D, page = 2, 3, 64, 16
    K, V, ks, vs, q, table = attention_case(rng, 3, H, G, D, page, lens, int8, False)
    clean, clse = run_attention(K, V, ks, vs, q, table, lens, page, 0.125, 0, max(lens), False, True)
    t0, t1 = lens[0] - 9, lens[1] // 2
    if int8:
        ks[table[0, t0 // page], 1, t0 % page] = math.nan
        vs[table[1, t1 // page], 0, t1 % page] = math.nan
    else:
        K[table[0, t0 // page], 1, t0 % page, 7] = math.nan
        V[table[1, t1 // page], 0, t1 % page // 8, :, t1 % 8] = math.nan
    out, lse = run_attention(K, V, ks, vs, q, table, lens, page, 0.125, 0, max(lens), False, True)
    bad = np.zeros((3, H * G), bool)
    bad[0, G:] = bad[1, :G] = True
    assert np.isnan(out[bad]).all() and np.array_equal(out[~bad], clean[~bad])
    bad[1] = False                                   # (the log-sum reads no values)
    assert np.isnan(lse[bad]).all() and np.array_equal(lse[~bad], clse[~bad])


@pytest.mark.parametrize("M,C,pad", [(9, 64, 0), (9, 61, 3), (40, 1000, 0), (1100, 1000, 0), (20, 4096, 0), (300, 4096, 0),
                                     (300, 4097, 2), (20, 8192, 0), (20, 16384, 0), (9, 28672, 0), (9, 28673, 0)])
@pytest.mark.parametrize("post,pre,resid,f32", [(False, False, False, True), (True, True, True, False), (False, True, True, True)])
def test_int8_norm_keeps_what_is_not_finite(M, C, pad, post, pre, resid, f32):
    """A row of h with an infinity or NaN stands for NaN in every element; the other rows are as they are without it."""
    import torch
    say("norm nonfinite", M, C, pad, post, pre, resid, f32)
    g = torch.Generator().manual_seed(M + C)
    t, code = (torch.float32, bq.DT_F32) if f32 else (torch.bfloat16, bq.DT_BF16)
    f = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    u, r = f(M, C + pad).to(t), f(M, C + pad).to(t)
    w = (1 + 0.1 * f(C)).to(t).cuda()
    bad = torch.zeros(M, dtype=torch.bool)
    odd = u.clone()
    for i in range(min(M - 3, 40)):
        m = 2 + i
        odd[m, int(torch.randint(C, (1,), generator=g))] = ODD[i % 4]
        bad[m] = True
    d = bq.norm_desc(M, C, code, code, code, bq.DT_ROW8, res_scale=0.5, branch_scale=0.7, u_stride=C + pad, r_stride=C + pad,
                     h_stride=C)
    runs = []
    for x in (u, odd):
        q, s = torch.full((M, C), 99, dtype=torch.int8, device="cuda"), torch.full((M,), 7.0, device="cuda")
        bq.block_norm(d, x.cuda(), r.cuda() if resid else None, w if post else None, None, w if pre else None, None, q, s)
        torch.cuda.synchronize()
        runs.append((q.cpu(), s.cpu()))
    (q0, s0), (q, s) = runs
    assert bool(torch.isnan(q.float() * s[:, None])[bad].all()), "a row that is not finite lost it"
    assert torch.equal(q[~bad], q0[~bad]) and torch.equal(s[~bad], s0[~bad])


def test_int8_norm_of_the_smallest_rows():
    """Rows whose 127/amax overflows: zeros stay zeros."""
    import torch
    say("norm smallest")
    u = torch.zeros(3, 64, device="cuda")
    u[0, :3] = torch.tensor([1e-38, -2e-39, 1e-38])
    u[1, 5] = -1e-40
    q, s = torch.full((3, 64), 99, dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    bq.block_norm(bq.norm_desc(3, 64, out_dtype=bq.DT_ROW8, branch_scale=1.0), u, None, None, None, None, None, q, s)
    assert torch.equal(q.cpu(), (127 * torch.sign(u)).to(torch.int8).cpu())
    assert torch.equal(s.cpu(), torch.from_numpy(np.float32([1e-38, np.float32(1e-40), 0]) / np.float32(127)))
