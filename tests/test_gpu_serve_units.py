"""Attention of packed tokens for counts of units around those of the plan that one warp makes (up to 64 pairs of tiles, of
which a lane holds two): short units, empty ones among them, whole and cut."""
import numpy as np
import pytest

from tests.test_gpu_serve_attention import Case

pytestmark = pytest.mark.gpu

COUNTS = [31, 32, 33, 40, 48, 62, 63, 64, 65, 66]


def _checked(c):
    from sparse_kv_cache_snapkv_gb300 import rkv
    out, ws = c.call()
    rkv.rkv_check_status(ws)
    c.check(out)


def _batch(n, seed, most, long_at=None, rows=20000):
    """Up to `most` new tokens of each of n units, none of every fifth and of the last; one unit over `rows` rows."""
    rng = np.random.default_rng(seed)
    news = [0 if u % 5 == 3 else int(x) for u, x in enumerate(rng.integers(1, most + 1, n))]
    news[-1] = 0
    lens = [t + int(x) for t, x in zip(news, rng.integers(0, 300, n))]
    if long_at is not None:
        news[long_at], lens[long_at] = most, rows
    return news, lens


@pytest.mark.parametrize("words", [0, 1])
@pytest.mark.parametrize("n", COUNTS)
def test_short_units(n, words):
    # (with 2 query heads a KV head a pair of tiles is 128 tokens: so many units and few tokens stay one warp's)
    news, lens = _batch(n, n, 3)
    _checked(Case(100 + n, news, lens, n_kv=1, gqa=2, words=words))


@pytest.mark.parametrize("words", [0, 1])
@pytest.mark.parametrize("n,at", [(33, 0), (33, 31), (40, 35), (63, 61), (64, 62), (64, 32), (66, 40)])
def test_one_long_unit_among_them_is_cut(n, at, words):
    news, lens = _batch(n, n + at, 2, at)
    _checked(Case(200 + n + at, news, lens, n_kv=2, gqa=2, words=words))


@pytest.mark.parametrize("n", [33, 50])
def test_units_of_several_pairs(n):
    """64 query heads a KV head: a pair of tiles is 4 tokens, so pairs and units differ, up to 64 pairs in all."""
    news = [1] * n
    for u in range(0, n, 7):
        news[u] = 9
    room = sum(news) // 4 + n
    while room > 64:
        news[news.index(9) if 9 in news else news.index(1)] = 0
        room = sum(news) // 4 + n
    lens = [t + 20 * u for u, t in enumerate(news)]
    _checked(Case(300 + n, news, lens, n_kv=1, gqa=64))


def test_the_last_units_are_empty():
    news = [2] * 34 + [0] * 30
    _checked(Case(400, news, [t + 50 for t in news], n_kv=1, gqa=2))
