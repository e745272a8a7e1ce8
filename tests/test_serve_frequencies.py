"""Rotary frequencies scaled by parts, with the ramp between whole pairs: against values written out by hand. No GPU needed."""
import math

import numpy as np
import pytest

from oracle import serve as S
from tests.test_serve_contract import lib  # noqa: F401

# double arithmetic, rounded to fp32 once; a ramp's quotient cancels a few digits
RTOL = 2.0 ** -24 + 1e-11


def _get(*args, **kw):
    from sparse_kv_cache_snapkv_gb300 import rkv
    f, m = rkv.rkv_rope_frequencies(*args, **kw)
    return f.numpy().astype(np.float64), m


def test_ends_are_whole_pairs(lib):  # noqa: F811
    """128 dimensions, base 1e6, context 32768: a pair turns 32 times at number 23.59 and once at 39.65, so the ramp goes
    from pair 23 to pair 40."""
    ends = [64 * math.log(32768 / (2 * math.pi * t)) / math.log(1e6) for t in (32, 1)]
    assert 23.5 < ends[0] < 23.7 and 39.6 < ends[1] < 39.7
    got, m = _get(128, 1e6, "by_whole_parts", factor=4.0, ctx=32768, fast=32.0, slow=1.0)
    want = []
    for i in range(64):
        plain = 1e6 ** (-i / 64)
        part = 0.0 if i <= 23 else 1.0 if i >= 40 else (i - 23) / 17  # of the way to a quarter of it
        want.append(plain * (1 - part) + plain / 4 * part)
    np.testing.assert_allclose(got, want, rtol=RTOL)
    assert abs(m - (0.1 * math.log(4) + 1)) <= 2.0 ** -23 * m
    # the other kind has its ends between pairs: some per cent apart on the ramp, the same on both sides of it
    other, m2 = _get(128, 1e6, "by_parts", factor=4.0, ctx=32768, fast=32.0, slow=1.0)
    assert m2 == m and (other[:24] == got[:24]).all() and (other[40:] == got[40:]).all()
    assert 0.01 < np.abs(other / got - 1)[24:40].max() < 0.1


@pytest.mark.parametrize("rot,base,ctx,fast,slow,first,last", [
    (64, 10000.0, 64, 32.0, 1.0, 0, 9),        # the first end is below pair 0
    (16, 10000.0, 3, 1.0, 0.5, 0, 0.001),      # both are: pair 0 stays, all others are divided
    (16, 1.5, 10 ** 9, 2.0, 1.0, 15, 15.001),  # both are behind the last pair: all stay
    (128, 10000.0, 4096, 32.0, 1.0, 20, 46),
])
def test_ends_stay_within_the_head(lib, rot, base, ctx, fast, slow, first, last):  # noqa: F811
    got, _ = _get(rot, base, "by_whole_parts", factor=8.0, ctx=ctx, fast=fast, slow=slow)
    i = np.arange(rot // 2)
    plain, part = base ** (-2.0 * i / rot), np.clip((i - first) / (last - first), 0, 1)
    np.testing.assert_allclose(got, plain * (1 - part) + plain / 8 * part, rtol=RTOL)


@pytest.mark.parametrize("rot", [16, 64, 96, 128])
@pytest.mark.parametrize("base,ctx,factor", [(10000.0, 4096, 16.0), (500000.0, 8192, 8.0), (1e6, 32768, 4.0), (1e4, 2048, 1.0)])
def test_the_oracle_agrees(lib, rot, base, ctx, factor):  # noqa: F811
    got, m = _get(rot, base, "by_whole_parts", factor=factor, ctx=ctx)
    want, wm = S.frequencies("by_whole_parts", rot, base, factor=factor, ctx=ctx)
    np.testing.assert_allclose(got, want, rtol=RTOL)
    assert abs(m - wm) <= 2.0 ** -23 * wm


def test_refusals(lib):  # noqa: F811
    from sparse_kv_cache_snapkv_gb300 import rkv
    good = dict(rot_dim=64, base=10000.0, kind="by_whole_parts", factor=2.0, ctx=1000, fast=32.0, slow=1.0)
    rkv.rkv_rope_frequencies(**good)
    for change in (dict(rot_dim=7), dict(base=1.0), dict(factor=0.5), dict(ctx=0), dict(slow=0.0), dict(fast=1.0)):
        with pytest.raises(rkv.RkvError):
            rkv.rkv_rope_frequencies(**{**good, **change})
