"""The attentions' launches stay below 2^32 threads at the ends of what their descriptors may hold (no GPU needed)."""
import itertools

import pytest

import bit_plane_gemv_amd as bq
from test_serve_abi import kv, prompt, shared, size

LIMIT = 1 << 32


def partials(ws, rows, D):
    """Partial results of a row that a workspace of this size holds: 8 bytes and a row of fp32 each."""
    Dp = (D + 31) // 32 * 32
    need = lambda n: (rows * n * 8 + 255) // 256 * 256 + rows * n * Dp * 4  # noqa: E731
    n = ws // (rows * (8 + 4 * Dp))
    while need(n) > ws:                              # (the first part is rounded up to 256 bytes)
        n -= 1
    assert ws == need(n)
    return n


def ends(H, most):
    return [(G, x) for G in (1, 2, 16, 40, 16384 // H) if G * H <= 16384 for x in most if x > 0]


@pytest.mark.parametrize("H", [1, 2, 8, 16, 32, 128, 1024])
@pytest.mark.parametrize("D", [1, 64, 256])
def test_prompt_launches(H, D):
    seen = 0
    for (G, T), R, dt in itertools.product(ends(H, [1, 2, 5, 100, 8192, 1 << 20, (1 << 26) // H]), [1, 64, 511, 4096, 8192], [0, 1]):
        T = min(T, 1 << 20, (1 << 26) // (G * H))
        for dtype in (bq.KV_BF16, bq.KV_INT8):
            e, ws = size("bitq_prompt_attn_workspace", prompt(kv(kv_heads=H, head_dim=D, pages=1 << 20, dtype=dtype), heads=H * G, requests=R,
                                                              tokens=T, table_stride=1 << 20, max_len=1 << 24, q_dtype=dt))
            assert e == bq.OK
            few = T * G <= 32 * R                    # tiles of 32 rows and 128 threads, else of 128 and 256
            pieces = partials(ws, T * H * G, D) if ws else 1
            tiles = T * G // (32 if few else 128) + R
            assert tiles * pieces * H * (128 if few else 256) < LIMIT
            assert (T * H * G + 3) // 4 * 256 < LIMIT or not ws                 # (the join)
            seen += pieces > 1
    assert seen or H == 1024


@pytest.mark.parametrize("H", [1, 2, 8, 16, 32, 128, 1024])
@pytest.mark.parametrize("D", [1, 64, 256])
def test_shared_launches(H, D):
    for (G, R), groups, dt in itertools.product(ends(H, [1, 2, 64, 511, 4096, 8192]), [1, 64, 8192], [0, 1]):
        R = min(R, (1 << 23) // (G * H))
        groups = min(groups, R)
        for most in (1, 1 << 12, 1 << 24):
            e, ws = size("bitq_shared_attn_workspace", shared(kv(kv_heads=H, head_dim=D, pages=1 << 20), groups=groups, max_prefix=most, heads=H * G,
                                                              requests=R, table_stride=1 << 20, max_len=1 << 24, q_dtype=dt))
            assert e == bq.OK
            pieces = partials(ws, R * H * G, D) - 1  # (of the prefix or of the own tokens, which have the others)
            few = R * G <= 32 * groups
            tiles = R * G // (32 if few else 128) + groups
            own = R * ((G + 31) // 32 if G <= 32 else (G + 127) // 128)
            assert pieces >= 1 and (tiles * (128 if few else 256) + own * (128 if G <= 32 else 256)) * pieces * H < LIMIT
            assert (R * H * G + 3) // 4 * 256 < LIMIT
