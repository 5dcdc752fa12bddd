"""shared_attn with more groups than a wave looks at in one step, and with more query heads per key-value head than a tile of
rows holds, against the 64-bit reference."""
import numpy as np
import pytest

from test_gpu_serve_attention import check_shared

pytestmark = pytest.mark.gpu


def groups(n, rng, most=3):
    """Requests of n groups of 0 .. most requests, with some in no group before and behind them: lengths, starts and prefixes."""
    size = rng.integers(0, most + 1, n)
    start = np.concatenate([[2], 2 + np.cumsum(size)])
    R = int(start[-1]) + 3
    prefix = rng.integers(0, 30, n)
    return rng.integers(0, 45, R).tolist(), start.tolist(), prefix.tolist()


@pytest.mark.parametrize("kind,dt", [("bf16", "f32"), ("int8", "bf16")])
@pytest.mark.parametrize("n", [62, 63, 64, 65, 70, 200])
def test_shared_more_groups_than_lanes(n, kind, dt):
    lens, start, prefix = groups(n, np.random.default_rng(n))
    check_shared(lens, start, prefix, 2, 2, 32, 8, kind, dt, seed=n)


def test_shared_more_groups_than_a_wave_searches_at_once():
    lens, start, prefix = groups(4200, np.random.default_rng(1), most=2)
    check_shared(lens, start, prefix, 1, 1, 32, 8, "bf16", "f32")


def test_shared_many_groups_of_one_request_each():
    lens = np.random.default_rng(2).integers(1, 60, 100).tolist()
    check_shared(lens, list(range(101)), [20] * 100, 1, 4, 64, 16, "bf16", "bf16")


@pytest.mark.parametrize("kind,dt", [("bf16", "bf16"), ("int8", "f32")])
@pytest.mark.parametrize("G", [32, 33, 127, 128, 129, 130, 300])
def test_shared_heads_of_a_key_value_head_over_several_tiles(G, kind, dt):
    check_shared([90, 40, 130, 77], [0, 3], [50], 1, G, 64, 16, kind, dt, seed=G)


@pytest.mark.parametrize("n", [64, 70])
def test_shared_many_groups_of_many_heads(n):
    lens, start, prefix = groups(n, np.random.default_rng(n + 1))
    check_shared(lens, start, prefix, 1, 140, 32, 8, "bf16", "f32", seed=n)
