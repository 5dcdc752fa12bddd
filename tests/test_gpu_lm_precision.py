"""bitq_paged_attn holds queries and softmax weights in fp32: inputs on which two bf16 terms in place of three show.

Every request has two tokens whose contributions cancel, so that an error of a weight (or of a score) far below the
rounding of the output's type is a large part of the output.
"""
import math

import numpy as np
import pytest

import lm_reference as ref

LN2 = float(np.float32(math.log(2)))       # as the scale: scores are powers of two of q . K
D, PAGE, R = 64, 8, 256


def bf16(x):
    import torch
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16).double().numpy()


def half_ulp_bf16(x):
    """Half the distance of bf16 numbers at x."""
    return np.where(x == 0, 0.0, 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 1e-300))) - 8))


def terms(x, n):
    """x rounded to the sum of n bf16 terms."""
    s = np.zeros_like(x)
    for _ in range(n):
        s = s + bf16(x - s)
    return s


def sections(int8, k0, k1, v0, v1, vs0, vs1, ks):
    """One page per request: tokens 0 and 1.  k0, k1 [R][D], v0, v1 [R][D]: elements or codes."""
    import torch
    t = torch.int8 if int8 else torch.bfloat16
    K, V = torch.zeros(R, 1, PAGE, D, dtype=t), torch.zeros(R, 1, 1, D, 8, dtype=t)
    for i, (k, v) in enumerate(((k0, v0), (k1, v1))):
        K[:, 0, i] = torch.from_numpy(k).to(t)
        V[:, 0, 0, :, i] = torch.from_numpy(v).to(t)
    if not int8:
        return K, V, None, None
    s = torch.ones(2, R, 1, PAGE)
    s[0] *= ks
    s[1, :, 0, 0], s[1, :, 0, 1] = torch.from_numpy(vs0), torch.from_numpy(vs1)
    return K, V, s[0], s[1]


def weights_case(int8):
    """Token 0 has the weight 1, token 1 p = 2^k in (1/2, 1); V0 = -p V1 but for V's own rounding.

    Returns the cache's sections, q and a bound on the fp32 error: k comes out exactly, scale log2(e) with two
    roundings, the score with one, 2^x with one ulp (2^-24 below 1); p V1 (p times V's scale first, for int8) and the
    sum with V0 round at the size of V0.  Together fewer than 12 times 2^-24 of |V1| over 1 + p."""
    rng = np.random.default_rng(21)
    n = rng.integers(1, 128, R)
    q, k0, k1 = np.zeros((R, 1, D), np.float32), np.zeros((R, D)), np.zeros((R, D))
    q[:, 0, 0] = 1
    k1[:, 0] = -n if int8 else -n / 128
    p = np.exp(LN2 * -n / 128)
    sign = rng.choice([-1.0, 1.0], (R, D))
    vs0 = vs1 = None
    if int8:
        v1 = sign * rng.integers(64, 128, (R, D))
        v0 = -v1
        vs1 = rng.uniform(0.5, 1, R).astype(np.float32)
        vs0 = (p * vs1 * (1 + 2.0 ** -11 * rng.uniform(-1, 1, R))).astype(np.float32)
        val0, val1 = v0 * vs0[:, None].astype(np.float64), v1 * vs1[:, None].astype(np.float64)
    else:
        v1 = bf16(sign * rng.uniform(0.5, 1, (R, D)))
        v0 = bf16(-p[:, None] * v1)
        val0, val1 = v0, v1
    bound = 12 * 2.0 ** -24 * np.maximum(np.abs(val0), np.abs(val1)) / (1 + p[:, None])
    return sections(int8, k0, k1, v0, v1, vs0, vs1, 1 / 128), q, bound, (p, val0, val1, vs0, vs1, v0, v1)


def scores_case(int8):
    """Scores q_a and q_b of 128 to 256 that differ by less than 1.

    A score's three terms are exact and their sum, scale log2(e) and the product round five times at 2^-24 of 256 (the
    larger of nearest and truncated sums); two scores: 10 times 2^-16, which moves the weights by ln 2 / 4 of that."""
    rng = np.random.default_rng(22)
    q, k0, k1 = np.zeros((R, 1, D), np.float32), np.zeros((R, D)), np.zeros((R, D))
    q[:, 0, 0] = rng.uniform(129, 256, R)
    q[:, 0, 1] = q[:, 0, 0] - rng.uniform(0, 1, R)
    k0[:, 0] = k1[:, 1] = 1
    v0, v1 = (np.rint(rng.uniform(-127, 127, (R, D))) if int8 else bf16(rng.uniform(-1, 1, (R, D))) for _ in range(2))
    one = np.ones(R, np.float32)
    bound = 10 * 2.0 ** -16 * math.log(2) / 4 * np.abs(v0 - v1) + 2.0 ** -21 * np.maximum(np.abs(v0), np.abs(v1))
    return sections(int8, k0, k1, v0, v1, one, one, 1.0), q, bound, (v0, v1)


def reference(case):
    (K, V, ks, vs), q, bound, _ = case
    out, lse, _, _ = ref.attention(q.astype(np.float64), K, V, ks, vs, np.arange(R)[:, None], [2] * R, PAGE, LN2, 0, 2)
    return out[:, 0], lse, bound


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("bf16_out", [False, True])
def test_two_terms_of_a_weight_would_show(int8, bf16_out):
    case = weights_case(int8)
    want, _, bound = reference(case)
    p, val0, val1, vs0, vs1, c0, c1 = case[3]
    for n, most, least in ((3, 0, 0), (2, 1, 0.05)):
        if int8:
            y = terms(vs0.astype(np.float64), n)[:, None] * c0 + terms((p * vs1).astype(np.float32), n)[:, None] * c1
        else:
            y = val0 + terms(p.astype(np.float32).astype(np.float64), n)[:, None] * val1
        y = y / (1 + p[:, None])
        tol = bound + (half_ulp_bf16(want) if bf16_out else 0)
        out = np.mean(np.abs((bf16(y) if bf16_out else y) - want) > tol)
        assert least <= out <= most, (n, out)


@pytest.mark.parametrize("int8", [False, True])
def test_two_terms_of_a_query_would_show(int8):
    case = scores_case(int8)
    want, _, bound = reference(case)
    v0, v1 = case[3]
    for n, most, least in ((3, 0, 0), (2, 1, 0.2)):
        x = terms(case[1][:, 0, :2].astype(np.float64), n)
        w = 1 / (1 + np.exp(LN2 * (x[:, 1] - x[:, 0])))[:, None]
        out = np.mean(np.abs(w * v0 + (1 - w) * v1 - want) > bound)
        assert least <= out <= most, (n, out)


def on_gpu(case, qf32, of32):
    import torch
    from test_gpu_lm import close, run_attention
    from gpuhelp import say
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    say("attn precision", qf32, of32)
    (K, V, ks, vs), q, _, _ = case
    want, wlse, bound = reference(case)
    out, lse = run_attention(K, V, ks, vs, q, np.arange(R)[:, None], [2] * R, PAGE, LN2, 0, 2, qf32, of32)
    close(out[:, 0], want, bound + (0 if of32 else half_ulp_bf16(np.abs(want) + bound)), "out")
    return lse, wlse


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("qf32,of32", [(False, False), (False, True), (True, False), (True, True)])
def test_weights_are_held_in_fp32(int8, qf32, of32):
    on_gpu(weights_case(int8), qf32, of32)


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
def test_scores_of_fp32_queries_are_held_in_fp32(int8):
    lse, want = on_gpu(scores_case(int8), True, True)
    assert np.abs(lse - want).max() <= 5 * 2.0 ** -16 * math.log(2) + 2.0 ** -22 * 256
