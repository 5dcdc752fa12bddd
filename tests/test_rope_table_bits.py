"""bitq_rope_table against arithmetic of 60 digits, in units of its entries' last bit (no GPU needed)."""
from decimal import ROUND_CEILING, ROUND_FLOOR, Decimal, getcontext

import pytest

import bit_plane_gemv_amd as bq

getcontext().prec = 60
TAU = Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257242")
KINDS = [("plain", bq.ROPE_PLAIN, {}), ("linear", bq.ROPE_LINEAR, dict(factor=4.0)), ("linear", bq.ROPE_LINEAR, dict(factor=0.01)),
         ("ramp", bq.ROPE_RAMP, dict(factor=8.0, trained=8192.0, turns_keep=32.0, turns_scale=1.0)),
         ("ramp", bq.ROPE_RAMP, dict(factor=40.0, trained=4096.0, turns_keep=64.0, turns_scale=0.5)),
         ("ramp", bq.ROPE_RAMP, dict(factor=2.5, trained=131072.0, turns_keep=8.0, turns_scale=3.0)),
         ("band", bq.ROPE_BAND, dict(factor=8.0, trained=8192.0, turns_keep=4.0, turns_scale=1.0))]


def turns(rot, base, kind, factor=1.0, trained=0.0, turns_keep=0.0, turns_scale=0.0):
    base, factor, trained, keep, scale = (Decimal(x) for x in (base, factor, trained, turns_keep, turns_scale))
    whole = lambda x, how: x.to_integral_value(rounding=how)  # noqa: E731
    clamp = lambda x: min(max(x, Decimal(0)), Decimal(1))  # noqa: E731
    for i in range(rot // 2):
        f = (base.ln() * (-2 * i) / rot).exp()
        if kind == "linear":
            f /= factor
        elif kind == "ramp":
            d = lambda x: rot * (trained / (TAU * x)).ln() / (2 * base.ln())  # noqa: E731
            lo, hi = max(whole(d(keep), ROUND_FLOOR), Decimal(0)), min(whole(d(scale), ROUND_CEILING), Decimal(rot - 1))
            t = clamp((i - lo) / max(hi - lo, Decimal("0.001")))
            f = f * (1 - t) + f / factor * t
        elif kind == "band":
            t = clamp((trained * f / TAU - scale) / (keep - scale))
            f = f * t + f / factor * (1 - t)
        yield f / TAU


@pytest.mark.parametrize("kind,code,arg", KINDS)
@pytest.mark.parametrize("rot", [2, 20, 64, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
def test_entries_are_exact_to_their_last_bit(rot, base, kind, code, arg):
    """Computed with 64 bits, each step rounded by 2^-64 of its result at most: w = base^(-2i/rot) to an ulp (2), how much of
    it stays (a ramp: 2; a band: w, three steps and a difference, 6, with the factor keep / (keep - scale) = 4/3: 8 at most), its
    sum with the stretched rest (1) and the turns (1): 12 |turns| units of 2^-64, and the entry's own 1/2."""
    got = bq.rope_table(rot, base=base, kind=code, **arg)
    for i, (g, t) in enumerate(zip(got.tolist(), turns(rot, base, kind, **arg))):
        off = (Decimal(g) - t * 2 ** 64) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        assert off <= Decimal(1) / 2 + 12 * t, (i, float(off), float(t))
