"""qk_rope against 64-bit results."""
import numpy as np
import pytest
import torch

import bit_plane_gemv_amd as bq
import serve_reference as ref
from gpuhelp import say

pytestmark = pytest.mark.gpu
DT = {"f32": (bq.DT_F32, torch.float32), "bf16": (bq.DT_BF16, torch.bfloat16)}


def check(T, A, H, D, rot, layout, x="f32", o="f32", w="f32", norm=True, pos=None, mscale=1.0, eps=1e-6, stride=0, shift=0,
          table=None, place=False, seed=0):
    rng = np.random.default_rng(seed)
    code, t = DT[x]
    ocode, ot = DT[o]
    data = torch.from_numpy(rng.standard_normal((T, (A + 2 * H) * D + stride + shift)).astype(np.float32)).to(t).cuda()
    qkv = data[:, shift:shift + (A + 2 * H) * D].unflatten(1, (A + 2 * H, D))
    q, k = qkv[:, :A], qkv[:, A:A + H]
    wq, wk = ((torch.from_numpy((1 + 0.3 * rng.standard_normal(D)).astype(np.float32)).to(DT[w][1]).cuda()) if norm else None
              for _ in range(2))
    pos = rng.integers(0, 100000, T) if pos is None else np.asarray(pos)
    table = (bq.rope_table(rot, base=10000.0) if rot else np.zeros(1, np.uint64)) if table is None else table
    d = bq.rope_desc(T, A, H, D, rot=rot, layout=bq.ROPE_PAIRS if layout == "pairs" else bq.ROPE_HALF, x_dtype=code,
                     out_dtype=ocode, w_dtype=DT[w][0], eps=eps, mscale=mscale)
    say("rope", T, A, H, D, rot, layout, x, o, w, norm)
    before = [z.double().cpu().numpy() for z in (q, k)]
    whole = data.clone()
    if place:
        qo, ko = q, k
    else:
        qo, ko = (torch.full((T, n, D), 7.0, dtype=ot, device="cuda") for n in (A, H))
    bq.qk_rope(d, q if A else None, k if H else None, wq, wk, torch.from_numpy(table).cuda(),
               torch.from_numpy(pos.astype(np.int32)).cuda(), qo if A else None, ko if H else None)
    torch.cuda.synchronize()
    for name, xx, ww, got, n in (("q", before[0], wq, qo, A), ("k", before[1], wk, ko, H)):
        want, mag = ref.rope(xx, None if ww is None else ww.double().cpu().numpy(), np.maximum(pos, 0), table, rot,
                             layout == "pairs", np.float32(eps), np.float32(mscale))
        # the norm: D / 2 + 8 roundings of 2^-24; sine, cosine and their products: 2^-24 of the terms each, and 2^-28
        tol = mag * 2.0 ** -24 * (D / 2 + 16) + ref.half_step(ot) * np.abs(want)
        g = got.double().cpu().numpy()
        left = pos < 0
        ok = np.abs(g - want) <= tol
        ok[left] = g[left] == (xx[left] if place else 7)
        assert ok.all(), f"{name}: {np.argwhere(~ok)[:4].tolist()} {g[~ok][:4]} for {want[~ok][:4]}, tolerance {tol[~ok][:4]}"
    if place:                                        # what lies beside q and k stays
        rest = whole.clone()
        rest[:, shift:shift + (A + H) * D] = data[:, shift:shift + (A + H) * D]
        assert torch.equal(rest, data)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("x,o", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("D,rot", [(1, 0), (2, 2), (5, 4), (64, 64), (64, 16), (80, 80), (80, 20), (96, 48), (128, 128), (128, 32),
                                   (128, 0), (200, 56), (255, 254), (256, 256), (256, 2)])
def test_rope_heads(D, rot, x, o, layout):
    check(7, 3, 2, D, rot, layout, x, o, norm=True, seed=D)
    check(7, 3, 2, D, rot, layout, x, o, norm=False, seed=D)


@pytest.mark.parametrize("T", [1, 2, 63, 700, 5000])
@pytest.mark.parametrize("A,H", [(1, 1), (8, 2), (0, 3), (5, 0), (40, 8)])
def test_rope_tokens_and_heads(T, A, H):
    check(T, A, H, 64, 64, "half", "bf16", "bf16", w="bf16")


def test_rope_positions():
    far = [0, 1, 2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30, 10 ** 9, 131071, 99999999, 16777217, 5]
    for layout in ("half", "pairs"):
        check(10, 2, 1, 128, 128, layout, pos=far, norm=False)
    check(10, 2, 1, 64, 64, "half", pos=[-1, 3, -1, -2 ** 31, 0, -5, 8, 9, 10, -1])
    check(4, 2, 1, 64, 64, "half", pos=[-1] * 4)


def test_rope_rows_off_their_alignment():
    for x in ("f32", "bf16"):
        check(9, 3, 2, 64, 64, "half", x, x, stride=1)
        check(9, 3, 2, 64, 32, "pairs", x, "bf16", stride=8, shift=1)


@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_rope_in_place(x):
    for D, rot, layout in ((64, 64, "half"), (96, 48, "pairs"), (33, 32, "half")):
        check(11, 5, 2, D, rot, layout, x, x, place=True)
        check(11, 5, 2, D, rot, layout, x, x, place=True, norm=False, pos=[1, -1] * 5 + [7])


def test_rope_scales_and_rows_of_zeros():
    check(5, 2, 1, 64, 64, "half", mscale=1.3)
    check(5, 2, 1, 64, 64, "half", mscale=-0.5, norm=False)
    T, D = 3, 64
    z = torch.zeros(T, 1, D, device="cuda")
    out = torch.full((T, 1, D), 7.0, device="cuda")
    d = bq.rope_desc(T, 1, 0, D, x_dtype=bq.DT_F32, out_dtype=bq.DT_F32, eps=1e-6)
    w = torch.ones(D, device="cuda")
    bq.qk_rope(d, z, None, w, None, torch.from_numpy(bq.rope_table(D)).cuda(), torch.arange(T, dtype=torch.int32, device="cuda"), out,
               None)
    assert not out.any()


def test_rope_what_is_not_finite_stays_in_its_head():
    T, A, D = 4, 3, 64
    x = torch.randn(T, A, D, device="cuda")
    y = x.clone()
    y[1, 1, 40], y[2, 0, 50] = float("inf"), float("nan")
    d = bq.rope_desc(T, A, 0, D, rot=32, x_dtype=bq.DT_F32, out_dtype=bq.DT_F32)
    t, p = torch.from_numpy(bq.rope_table(32)).cuda(), torch.arange(T, dtype=torch.int32, device="cuda")
    outs = [torch.empty(T, A, D, device="cuda") for _ in range(2)]
    for z, o in zip((x, y), outs):
        bq.qk_rope(d, z, None, None, None, t, p, o, None)
    same = torch.ones(T, A, D, dtype=torch.bool, device="cuda")
    same[1, 1, 40] = same[2, 0, 50] = False          # past the rotated elements, without a norm: themselves alone
    assert torch.equal(outs[0][same], outs[1][same])
    assert outs[1][1, 1, 40] == float("inf") and outs[1][2, 0, 50].isnan()


@pytest.mark.parametrize("kind,arg", [("linear", dict(factor=4.0)),
                                      ("ramp", dict(factor=8.0, trained=8192.0, turns_keep=32.0, turns_scale=1.0)),
                                      ("band", dict(factor=8.0, trained=8192.0, turns_keep=4.0, turns_scale=1.0))])
def test_rope_stretched(kind, arg):
    codes = dict(linear=bq.ROPE_LINEAR, ramp=bq.ROPE_RAMP, band=bq.ROPE_BAND)
    table = bq.rope_table(128, base=500000.0, kind=codes[kind], **arg)
    check(40, 4, 2, 128, 128, "half", table=table, mscale=1.2)
