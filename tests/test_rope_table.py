"""bitq_rope_table: frequencies as 64-bit fractions of a turn, against their definition (no GPU needed)."""
import math

import numpy as np
import pytest

import bit_plane_gemv_amd as bq
import serve_reference as ref

STRETCHED = [("plain", bq.ROPE_PLAIN, {}), ("linear", bq.ROPE_LINEAR, dict(factor=4.0)),
             ("ramp", bq.ROPE_RAMP, dict(factor=8.0, trained=8192.0, turns_keep=32.0, turns_scale=1.0)),
             ("ramp", bq.ROPE_RAMP, dict(factor=40.0, trained=4096.0, turns_keep=64.0, turns_scale=0.5)),
             ("band", bq.ROPE_BAND, dict(factor=8.0, trained=8192.0, turns_keep=4.0, turns_scale=1.0))]


@pytest.mark.parametrize("kind,code,arg", STRETCHED)
@pytest.mark.parametrize("rot", [2, 20, 64, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
def test_table(rot, base, kind, code, arg):
    got = bq.rope_table(rot, base=base, kind=code, **arg)
    f = ref.frequencies(rot, base, kind, arg.get("factor", 1), arg.get("trained", 0), arg.get("turns_keep", 0), arg.get("turns_scale", 0))
    turns = f / (2 * math.pi)
    # 64-bit floats hold the reference to a few parts in 2^53
    assert got.dtype == np.uint64 and got.shape == (rot // 2,)
    assert np.all(np.abs(got.astype(np.float64) / 2.0 ** 64 - turns) <= 1e-14 * turns + 2.0 ** -64)


def test_frequencies_above_a_turn_wrap():
    got = bq.rope_table(2, base=2.0, kind=bq.ROPE_LINEAR, factor=0.01)       # 100 radians: 15.9 turns
    assert abs(int(got[0]) / 2.0 ** 64 - (100 / (2 * math.pi)) % 1) < 1e-14


@pytest.mark.parametrize("bad", [dict(rot=0), dict(rot=3), dict(rot=258), dict(rot=-2), dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
                                 dict(kind=4), dict(kind=-1), dict(kind=1, factor=0.0), dict(kind=1, factor=math.inf),
                                 dict(kind=2, trained=0.0), dict(kind=2, turns_keep=1.0), dict(kind=3, turns_scale=0.0),
                                 dict(kind=3, turns_keep=math.nan), dict(kind=2, trained=math.inf)])
def test_refusals(bad):
    a = dict(rot=64, base=10000.0, kind=0, factor=2.0, trained=4096.0, turns_keep=32.0, turns_scale=1.0)
    a.update(bad)
    with pytest.raises(bq.BitqError) as e:
        bq.rope_table(**a)
    assert e.value.status in (bq.E_ARG, bq.E_SHAPE)
