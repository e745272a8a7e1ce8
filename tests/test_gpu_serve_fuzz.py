"""Seeded random configurations of the packed attention and of the places against the oracle."""
import numpy as np
import pytest

from oracle import serve as S
from tests.test_gpu_serve_attention import Case
from tests.test_gpu_serve_places import Pool, _rope, _same

pytestmark = pytest.mark.gpu


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


@pytest.mark.parametrize("seed", range(60))
def test_attention(seed):
    from sparse_kv_cache_snapkv_gb300 import rkv
    rng = np.random.default_rng(1000 + seed)
    n, gqa, tree = _log(rng, 1, 20), int(rng.integers(1, 17)), seed % 2 == 1
    n_kv = int(rng.integers(1, max(2, 17 // gqa)))
    most = _log(rng, 1, 200 if not tree else 70)
    news = [int(rng.integers(0, most + 1)) for _ in range(n)]
    lens = [t + (0 if rng.random() < 0.2 else _log(rng, 1, 4000 if n < 5 else 400) - 1) for t in news]
    lens = [max(x, 1) if rng.random() < 0.9 else x for x in lens]
    if sum(news) == 0:
        news[0], lens[0] = 1, max(lens[0], 1)
    block = int(rng.choice([0, 1, 4, 16, 32, 64, 128, 256]))
    c = Case(seed, news, lens, n_kv=n_kv, gqa=gqa, cap=max(lens) + int(rng.integers(0, 50)), block=block,
             words=-(-most // 32) + int(rng.integers(0, 2)) if tree else 0, front=int(rng.integers(0, 5)),
             behind=int(rng.integers(0, 5)), spread=float(rng.choice([0.3, 1.0, 4.0])))
    out, ws = c.call()
    rkv.rkv_check_status(ws)
    c.check(out)


@pytest.mark.parametrize("seed", range(40))
def test_places(seed):
    rng = np.random.default_rng(2000 + seed)
    n, block, most = _log(rng, 1, 300), int(rng.choice([1, 5, 16, 64, 100])), _log(rng, 1, 60)
    room = most * block
    lens = [int(rng.integers(0, room + 1)) if rng.random() < 0.8 else 0 for _ in range(n)]
    extra = [int(rng.integers(0, most - -(-t // block) + 1)) if rng.random() < 0.2 else 0 for t in lens]
    new = [int(rng.integers(0, room - t + 1)) if rng.random() < 0.7 else 0 for t in lens]
    p = Pool(seed, lens, block, most, int(rng.integers(0, n * most // 2 + 2)), extra)
    total = sum(new) + int(rng.integers(0, 20)) or 1
    if p.num == 0:  # a pool of no blocks is refused
        from sparse_kv_cache_snapkv_gb300 import rkv
        with pytest.raises(rkv.RkvError):
            p.reserve(new, total)
        return
    bits = S.reserve(new, p.len, p.held, p.table, p.free, p.count, p.block, total)[1]
    assert bits in (0, 0x20)
    _same(p, new, total, bits=bits, alias=bool(seed % 2))


@pytest.mark.parametrize("seed", range(20))
def test_rope(seed):
    rng = np.random.default_rng(3000 + seed)
    assert _rope(seed, _log(rng, 1, 3000), int(rng.integers(1, 40)), int(rng.integers(1, 9)),
                 rot=16 * int(rng.integers(1, 9)), interleaved=bool(seed % 2), mscale=float(rng.choice([1.0, 0.5, 1.4])),
                 block=int(rng.choice([1, 7, 16, 64])), fused=bool(rng.integers(0, 2)),
                 base=float(rng.choice([10000.0, 500000.0]))) == 0
