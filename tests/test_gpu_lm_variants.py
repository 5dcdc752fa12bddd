"""Every kernel variant of the int8 product, the block norm and the attention, with contiguous outputs and rows on their
alignment.

Which variant a shape takes is asked of the library's own rule, so the lists cannot drift away from it.
"""
import ctypes
import itertools

import numpy as np
import pytest

import bit_plane_gemv_amd as bq
import lm_reference as ref


class Plan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("splits", ctypes.c_int), ("ws_bytes", ctypes.c_size_t)]


FEW, T64, T64x128, T128, T256 = "few", 5, 6, 7, 8
KERNEL = [  # M, N, K, kernel (few tokens: by 16 tokens), k ranges
    (1, 64, 80, 1, 1), (16, 4096, 144, 1, 1), (8, 5136, 272, 1, 1), (7, 9008, 144, 1, 1), (5, 17008, 80, 1, 1),
    (32, 512, 400, 2, 1), (40, 96, 1040, 3, 1), (64, 1008, 528, 4, 1),
    (70, 320, 208, T64, 1), (128, 64, 16, T64, 1), (64, 128, 8208, T64, 8), (100, 1040, 7008, T64, 6),
    (512, 4096, 64, T64x128, 1), (500, 4080, 144, T64x128, 1), (449, 4094, 80, T64x128, 1),
    (1024, 4096, 80, T128, 1), (1000, 4080, 144, T128, 1), (1023, 4097, 272, T128, 1),
    (4096, 4096, 80, T256, 1), (4000, 4080, 144, T256, 1), (4090, 4095, 208, T256, 1),
]


def plan_of(M, N, K):
    f = bq._lib["_ZN4bitq9w8a8_planERK14bitq_w8a8_desc"]
    f.argtypes, f.restype = [ctypes.POINTER(bq.W8A8Desc)], Plan
    return f(ctypes.byref(bq.w8a8_desc(M, N, K)))


@pytest.mark.parametrize("M,N,K,kernel,splits", KERNEL)
def test_each_product_takes_the_kernel_it_is_listed_for(M, N, K, kernel, splits):
    p = plan_of(M, N, K)
    assert (p.kernel, p.splits) == (kernel, splits)


def test_the_products_cover_every_kernel():
    assert {k for *_, k, _ in KERNEL} == set(range(1, 9))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,kernel,splits", KERNEL)
@pytest.mark.parametrize("pad", [0, 8, 1])
def test_product_of_every_kernel(M, N, K, kernel, splits, pad):
    """Contiguous y (pad 0, N a multiple of 16: whole 16-byte stores), rows still on 16 bytes, rows off them."""
    import torch
    from gpuhelp import say
    from test_gpu_lm import BF16_ULP
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    say("w8a8 variant", M, N, K, kernel, pad)
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    codes = lambda *s: torch.randint(-128, 128, s, generator=g, dtype=torch.int8, device="cuda")  # noqa: E731
    a, w = codes(M, K), codes(N, K)
    sa, sw = torch.rand(M, generator=g, device="cuda") * 0.1, torch.rand(N, generator=g, device="cuda") * 0.01
    want = a.double() @ w.double().t()                       # integers below 2^53: exact
    exact = want * sa.double()[:, None] * sw.double()
    for t, flags, tol in ((torch.int32, bq.F_ACC_INT32, 0), (torch.float32, 0, 2.0 ** -22), (torch.bfloat16, 0, BF16_ULP)):
        d = bq.w8a8_desc(M, N, K, bq.DT_BF16 if t == torch.bfloat16 else bq.DT_F32, ldy=N + pad, flags=flags)
        ws = torch.full((max(1, bq.w8a8_workspace(d)),), 0x5A, dtype=torch.uint8, device="cuda")
        y = torch.full((M * (N + pad) + 64,), 77, dtype=t, device="cuda")
        bq.gemm_w8a8(d, a, sa, w, sw, y, ws)
        torch.cuda.synchronize()
        rows, past = y[:M * (N + pad)].view(M, N + pad), y[M * (N + pad):]
        got, ref64 = rows[:, :N].double(), want if flags else exact
        bad = (got - ref64).abs() > tol * ref64.abs()
        assert not bool(bad.any()), (t, bad.nonzero()[0].tolist())
        assert bool((rows[:, N:] == 77).all()) and bool((past == 77).all()), "wrote past a row"


# Widths that take each variant of the norm: one wave a row with one or two chunks of 8 a lane, then 4 and 16 waves
NORM = [(5, 8), (70, 64), (7, 504), (9, 512), (1030, 512), (1100, 520), (1100, 1000), (1030, 1024), (9, 1024), (300, 2048), (300, 4096),
        (300, 8192), (5, 8192), (5, 16384), (5, 32768)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,C", NORM)
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_norm_of_every_variant(M, C, pad):
    """Rows on their alignment (pad 0 and 8) and off it, in each of the 8 pairs of types of u, r and the weights."""
    import torch
    from gpuhelp import say
    from test_gpu_lm import BF16_ULP, close
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rng = np.random.default_rng(M + C)
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    u0, r0, g0, po0, pr0 = 3 * f(M, C + pad), 2 * f(M, C + pad), f(M, C + pad), 1 + f(C), 1 + f(C)
    T = {bq.DT_F32: torch.float32, bq.DT_BF16: torch.bfloat16, bq.DT_ROW8: torch.int8}
    outs = itertools.cycle([bq.DT_F32, bq.DT_BF16, bq.DT_ROW8])
    eps = 2.0 ** -24 * (32 + C / 256)       # an element's roundings, and the sums' relative error
    for ut, rt, wt in itertools.product((bq.DT_F32, bq.DT_BF16), repeat=3):
        ot = next(outs)
        say("norm variant", M, C, pad, ut, rt, wt, ot)
        u, r, gate, post, pre = u0.to(T[ut]), r0.to(T[rt]), g0.to(T[wt]), po0.to(T[wt]), pr0.to(T[wt])
        st = C + pad
        d = bq.norm_desc(M, C, ut, rt, wt, ot, res_scale=0.75, branch_scale=-1.5, eps_post=1e-3, eps_pre=1e-4, gate_stride=st,
                         u_stride=st, r_stride=st, ro_stride=st, h_stride=st)
        ro, h = torch.full((M, st), 7, dtype=T[rt], device="cuda"), torch.full((M, st), 7, dtype=T[ot], device="cuda")
        sc = torch.zeros(M, device="cuda") if ot == bq.DT_ROW8 else None
        bq.block_norm(d, u.cuda(), r.cuda(), post.cuda(), gate.cuda(), pre.cuda(), ro, h, sc)
        torch.cuda.synchronize()
        wro, wh, mro, mh = ref.norm(*(t[..., :C].double().numpy() for t in (u, r, post, gate, pre)), 0.75, -1.5, 1e-3, 1e-4)
        close(ro[:, :C].float().cpu().numpy(), wro, eps * mro + (BF16_ULP * np.abs(wro) if rt == bq.DT_BF16 else 0), "r")
        got = h[:, :C].float().cpu().numpy().astype(np.float64)
        if sc is not None:
            s = sc.cpu().numpy().astype(np.float64)[:, None]
            amax = np.abs(wh).max(1, keepdims=True)
            close(s, amax / 127, eps * mh.max(1, keepdims=True) / 127 + 2.0 ** -23 * amax / 127, "scale")
            close(got * s, wh, s * 0.5 * (1 + 1e-5) + 130 * eps * mh, "values")
        else:
            close(got, wh, eps * mh + (BF16_ULP * np.abs(wh) if ot == bq.DT_BF16 else 0), "h")
        assert bool((h[:, C:] == 7).all()) and bool((ro[:, C:] == 7).all()), "wrote past a row"


# ------------------------------------------------------------- attention
class AttnPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("Dp", "group", "tiles", "items", "grid", "waves")] + [
        ("split", ctypes.c_bool), ("off_part", ctypes.c_size_t), ("ws_bytes", ctypes.c_size_t)]


def attn_plan_of(D, int8, qf32, R, H, A, max_len):
    f = bq._lib["_ZN4bitq9attn_planERK14bitq_attn_desc"]
    f.argtypes, f.restype = [ctypes.POINTER(bq.AttnDesc)], AttnPlan
    kv = bq.kvdesc(H, D, 16, 4096, bq.KV_INT8 if int8 else bq.KV_BF16)
    return f(ctypes.byref(bq.attn_desc(kv, A, R, (max_len + 15) // 16, max_len, q_dtype=bq.DT_F32 if qf32 else bq.DT_BF16)))


# how the tokens are dealt: requests, key-value heads, query heads of each, lengths; split, waves, waves of the join
DEAL = {
    "an item a workgroup": (3, 2, 3, [33, 0, 200], False, 4, 0),
    "an item a wave": (1100, 1, 1, [i % 20 for i in range(1100)], False, 1, 0),
    "split": (2, 1, 2, [3001, 70], True, 4, 8),
    "split, many heads": (300, 2, 2, [1800] + [i % 9 for i in range(299)], True, 4, 1),
    "split, many ranges": (1, 1, 1, [20000], True, 4, 16),
}


@pytest.mark.parametrize("deal", DEAL)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("qf32", [False, True])
def test_each_attention_takes_the_deal_it_is_listed_for(deal, int8, qf32):
    R, H, G, lens, split, waves, join = DEAL[deal]
    for D in range(20, 257, 32):
        p = attn_plan_of(D, int8, qf32, R, H, H * G, max(lens))
        assert (p.Dp, p.split, p.waves) == ((D + 31) // 32 * 32, split, waves), D
        if split:
            assert join == (1 if R * H * G > 512 else 8 if p.grid // p.items < 64 else 16), D


@pytest.mark.gpu
@pytest.mark.parametrize("D", list(range(20, 257, 32)))
@pytest.mark.parametrize("deal", DEAL)
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("qf32", [False, True])
def test_attention_of_every_variant(D, deal, int8, qf32):
    import torch
    from gpuhelp import say
    from test_gpu_lm import BF16_ULP, attention_case, close, run_attention
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    say("attn variant", D, deal, int8, qf32)
    R, H, G, lens, *_ = DEAL[deal]
    K, V, ks, vs, q, table = attention_case(np.random.default_rng(D + R), R, H, G, D, 16, lens, int8, qf32)
    for of32 in (False, True):
        out, lse = run_attention(K, V, ks, vs, q, table, lens, 16, D ** -0.5, 0, max(lens), qf32, of32)
        want, wlse, tol, ltol = ref.attention(q.astype(np.float64), K, V, ks, vs, table, lens, 16, D ** -0.5, 0, max(lens))
        close(out, want, tol + (0 if of32 else BF16_ULP * np.abs(want)), "out")
        close(lse, wlse, ltol, "lse")
