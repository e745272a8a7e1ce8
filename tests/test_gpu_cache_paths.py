"""The cache calls where their work is laid out another way: as many parts as there are CTAs, more units than
a launch's threads count one by one, more items than SMs, and large offsets. Against the float64 oracle;
decodes with a tolerance for each query head."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as C
from tests import cache_parity as P
from tests import cache_parity_heads as H

pytestmark = pytest.mark.gpu

D = 128
SCALE = 1.0 / math.sqrt(D)
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def rkv():
    from sparse_kv_cache_snapkv_gb300 import rkv
    rkv.load()
    return rkv


def _ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _rand(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)


def _f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def _held(cache, u, g, t):
    """The numbers that a 4-bit cache's first t rows stand for."""
    return [C.kv4_values(cache[i][u, g, :t].cpu().numpy(), cache[i + 1][u, g, :t].cpu().numpy()) for i in (0, 2)]


def _decode(rkv, kv4, n, n_kv, gqa, cap, lens, units, seed=1, **kw):
    """One decode with weights; the units named are checked."""
    k, v = _rand(seed, n, n_kv, cap, D), _rand(seed + 1, n, n_kv, cap, D)
    q = _rand(seed + 2, n, n_kv * gqa, D)
    out, w = torch.full_like(q, float("nan")), torch.zeros(n, n_kv, cap, device="cuda")
    ln = _ints(lens)
    if kv4:
        cache = rkv.kv4_cache(n, n_kv, cap)
        rkv.rkv_check_status(rkv.rkv_kv4_append(k, v, *cache, _ints([0] * n), torch.empty_like(ln), new_len=ln))
        rkv.rkv_check_status(rkv.rkv_kv4_decode(q, *cache, ln, SCALE, out, weights=w, **kw))
    else:
        rkv.rkv_check_status(rkv.rkv_dense_decode_weights(q, k, v, ln, SCALE, out, w, **kw))
    for u in units:
        t = lens[u]
        for g in range(n_kv):
            heads = slice(g * gqa, (g + 1) * gqa)
            assert not w[u, g, t:].any()
            if t == 0:
                assert not out[u, heads].any()
                continue
            hk, hv = _held(cache, u, g, t) if kv4 else (_f64(k[u, g, :t]), _f64(v[u, g, :t]))
            H.check_decode(_f64(out[u, heads]), _f64(w[u, g, :t]), _f64(q[u, heads]), hk, hv, SCALE, kv4,
                           64 + t // 64, f"unit {u} head {g}")
    assert torch.isfinite(out).all() and torch.isfinite(w).all()


# ------------------------------------------------------------------------------- decodes
@pytest.mark.parametrize("kv4", [True, False])
@pytest.mark.parametrize("gqa", [1, 8])
def test_decode_in_as_many_parts_as_ctas(rkv, kv4, gqa):
    """One (unit, head) over every CTA of the launch: the joins' table of factors at its fullest."""
    _decode(rkv, kv4, 1, 1, gqa, 131071, [131071], [0])


@pytest.mark.parametrize("kv4", [True, False])
@pytest.mark.parametrize("n,n_kv,gqa,cap", [(33, 3, 2, 300), (257, 1, 4, 200), (1100, 2, 1, 40)])
def test_decode_of_many_units(rkv, kv4, n, n_kv, gqa, cap):
    """More units than a warp, or the threads of a CTA, have one each of; many without tokens."""
    lens = [0 if u % 5 == 3 else (u * 37) % (cap + 1) for u in range(n)]
    lens[0], lens[-1] = 0, cap
    _decode(rkv, kv4, n, n_kv, gqa, cap, lens, sorted({0, 1, 31, 32, n // 2, n - 2, n - 1}))
