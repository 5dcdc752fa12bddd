"""The weights of prompt_attn and shared_attn keep 24 bits whatever the types of queries and outputs: outputs that are small
differences of large terms show what a weight loses."""
import numpy as np
import pytest
import torch

import bit_plane_gemv_amd as bq
import serve_reference as ref
from gpuhelp import say
from test_gpu_serve_attention import DT, close, tables, upload

pytestmark = pytest.mark.gpu
PAIRS, D, PAGE = 16, 64, 16
SEEN = 1 + 2 * PAIRS                                 # tokens that count; later ones weigh nothing


def sections_of(pool, lens, table, H, int8, rng):
    """Token 0 scores 0 and has no value.  Tokens 1 + 2 i and 2 + 2 i score q0 a and q0 a + 2^-14 and have the values -v and v
    in element i alone: its output is v (w2 - w1) / sum w.  All else scores -120 and has no value.  With q = (q0, 2^-7, 1, 0, ..)
    in bf16 every score is a sum of few products of few bits: exact in fp32."""
    K = torch.zeros(pool, H, PAGE, D, dtype=torch.int8 if int8 else torch.bfloat16)
    V = torch.zeros(pool, H, PAGE // 8, D, 8, dtype=K.dtype)
    ks, vs = (torch.ones(pool, H, PAGE) for _ in range(2)) if int8 else (None, None)
    a = rng.integers(-127, -31, (H, PAIRS))          # in 128ths
    v = torch.from_numpy(rng.uniform(1, 2, (H, PAIRS)).astype(np.float32))
    if int8:
        v = (v / 100).float()                        # the scale of a code of 100
    else:
        v = v.bfloat16().float()
    for r, n in enumerate(lens):
        for t in range(n):
            p, o = int(table[r, t // PAGE]), t % PAGE
            if t >= SEEN:
                K[p, :, o, 2] = -120
            elif t > 0:
                i, up = (t - 1) // 2, (t - 1) % 2
                code = torch.from_numpy(a[:, i])
                K[p, :, o, 0] = (code if int8 else code / 128).to(K.dtype)
                K[p, :, o, 1] = up * (1 if int8 else 2.0 ** -7)
                V[p, :, o // 8, i, o % 8] = (100 if up else -100) if int8 else ((1 if up else -1) * v[:, i]).to(V.dtype)
                if int8:
                    ks[p, :, o], vs[p, :, o] = 2.0 ** -7, v[:, i]
    value = (v.double() * (100 if int8 else 1)).numpy()
    return (K, V, ks, vs), a / 128.0, value


def check(got, q0, G, a, value, otype):
    """got [rows, H G, D] for q0 [rows, H G].  Relative to its weight, what a pair's output may be off by: the exponent's
    factor (two roundings, at most a unit of the score: 2^-23) and its rounding (below 2: 2^-24), the power (an ulp, 2^-23), the
    scale of an int8 value (2^-24), and sums of a few terms on the matrix cores (4 x 2^-23): 7 x 2^-23 for each of the two
    tokens.  The sum of the weights is off by 2^-18 of itself at most (that of 33 of them, 33 x 2^-24, and their own)."""
    rows, A = q0.shape
    h = np.arange(A) // G
    s = q0[..., None] * a[h]                          # [rows, A, PAIRS]
    w1, w2 = np.exp(s), np.exp(s + 2.0 ** -14)
    z = 1 + (w1 + w2).sum(-1, keepdims=True)
    want, tol = np.zeros((rows, A, D)), np.zeros((rows, A, D))
    want[..., :PAIRS] = value[h] * w1 * np.expm1(2.0 ** -14) / z
    tol[..., :PAIRS] = value[h] * (w1 + w2) / z * 7 * 2.0 ** -23 + 2.0 ** -18 * want[..., :PAIRS]
    close(got, want, tol + ref.half_step(otype) * (want + tol), "out")


def queries(rows, A, dt, rng):
    q = np.zeros((rows, A, D), dtype=np.float32)
    q[..., 0] = torch.from_numpy(rng.uniform(0.25, 1, (rows, A)).astype(np.float32)).bfloat16().float().numpy()
    q[..., 1], q[..., 2] = 2.0 ** -7, 1
    return torch.from_numpy(q).to(dt).cuda(), q[..., 0].astype(np.float64)


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("dt,odt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("new,G", [(1, 4), (3, 8), (40, 8)])
def test_prompt_weights_keep_24_bits(new, G, dt, odt, kind):
    rng = np.random.default_rng(new + G)
    H, lens = 2, [SEEN + new]
    table, pool = tables(lens, PAGE, 8, rng)
    sections, a, value = sections_of(pool, lens, table, H, kind == "int8", rng)
    kv = bq.kvdesc(H, D, PAGE, pool, bq.KV_INT8 if kind == "int8" else bq.KV_BF16)
    q, q0 = queries(new, H * G, DT[dt][1], rng)
    d = bq.prompt_desc(kv, H * G, 1, new, 8, 128, q_dtype=DT[dt][0], out_dtype=DT[odt][0], scale=1.0)
    ws = torch.empty(max(1, bq.prompt_attn_workspace(d)), dtype=torch.uint8, device="cuda")
    out = torch.full((new, H * G, D), 7.0, dtype=DT[odt][1], device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    say("prompt weights", new, G, dt, odt, kind, "workspace", ws.numel())
    bq.prompt_attn(d, q, upload(sections, kv), torch.from_numpy(table).cuda(), i32([0, new]), i32(lens), out, ws)
    check(out, q0, G, a, value, DT[odt][1])


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("dt,odt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("R,G", [(3, 4), (40, 8)])
def test_shared_weights_keep_24_bits(R, G, dt, odt, kind):
    rng = np.random.default_rng(R)
    H, lens = 2, [SEEN] * R
    table, pool = tables(lens, PAGE, 8, rng)
    sections, a, value = sections_of(pool, lens, table, H, kind == "int8", rng)
    kv = bq.kvdesc(H, D, PAGE, pool, bq.KV_INT8 if kind == "int8" else bq.KV_BF16)
    q, q0 = queries(R, H * G, DT[dt][1], rng)
    d = bq.shared_desc(bq.attn_desc(kv, H * G, R, 8, 128, q_dtype=DT[dt][0], out_dtype=DT[odt][0], scale=1.0), 1, 64)
    ws = torch.empty(bq.shared_attn_workspace(d), dtype=torch.uint8, device="cuda")
    out = torch.full((R, H * G, D), 7.0, dtype=DT[odt][1], device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    say("shared weights", R, G, dt, odt, kind, "workspace", ws.numel())
    bq.shared_attn(d, q, upload(sections, kv), torch.from_numpy(table).cuda(), i32(lens), i32([0, R]), i32([20]), out, ws)
    check(out, q0, G, a, value, DT[odt][1])
