"""prompt_attn and shared_attn refuse scales whose factor in powers of two is no finite number (no GPU needed)."""
import pytest

import bit_plane_gemv_amd as bq
from test_serve_abi import BIG, P, prompt, shared, size, status

MOST = 2.3e38                                        # (the largest float over log2(e) is 2.358..e38)


@pytest.mark.parametrize("scale", [2.4e38, -2.4e38, 3.4e38, -3.4e38])
def test_scales_beyond_the_largest(scale):
    assert size("bitq_prompt_attn_workspace", prompt(scale=scale))[0] == bq.E_ARG
    assert size("bitq_shared_attn_workspace", shared(scale=scale))[0] == bq.E_ARG
    assert status("bitq_prompt_attn", prompt(scale=scale), P, 1 << 15, P, BIG, P, P, P, P, None, P, BIG, None) == bq.E_ARG
    assert status("bitq_shared_attn", shared(scale=scale), P, 1 << 15, P, BIG, P, P, P, P, P, None, P, BIG, None) == bq.E_ARG


@pytest.mark.parametrize("scale", [0.0, MOST, -MOST, 1e-45])
def test_scales_that_are_taken(scale):
    assert size("bitq_prompt_attn_workspace", prompt(scale=scale))[0] == bq.OK
    assert size("bitq_shared_attn_workspace", shared(scale=scale))[0] == bq.OK
