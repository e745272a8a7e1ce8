"""The cache decodes against the float64 oracle with a tolerance for each query head
(tests/cache_parity_heads.py)."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as C
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


def _cancelling(p, rng):
    """Values of few bits, for probabilities p [T], whose weighted sum nearly vanishes: each token
    takes the value that brings the sum of those before it closest to zero."""
    grid = np.array([m * s for m in (1.0, 1.5, 2.0, 3.0, 4.0, 6.0) for s in (1, -1)])
    v, at = np.zeros(len(p)), 0.0
    for t in np.argsort(-p):
        near = grid[np.argsort(np.abs(at + p[t] * grid))[: 3 if at == 0 else 1]]
        v[t] = rng.choice(near) if at else rng.choice(grid)
        at += p[t] * v[t]
    return v


@pytest.mark.parametrize("gqa", [1, 4])
@pytest.mark.parametrize("T", [5, 24, 300])
def test_kv4_probabilities_keep_their_bits(rkv, gqa, T):
    """Outputs that cancel: the sum is far below its terms, so that what the probabilities lose on
    their way into the product with V shows beside the rounding of the output. Small logits keep
    the exponentials' own error below that."""
    rng = np.random.default_rng(T)
    n, n_kv = 8, 2
    q = np.zeros((n, n_kv, gqa, D))
    k = np.zeros((n, n_kv, T, D))
    q[..., 0] = rng.uniform(0.5, 1.0, q.shape[:-1])
    k[..., 0] = rng.choice([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], (n, n_kv, T)) * rng.choice([1, -1], (n, n_kv, T))
    k[..., 1] = 6.0  # the block's scale is 1: k and v are held as they are
    q = torch.tensor(q).to(BF)
    v = np.zeros((n, n_kv, T, D))
    for u in range(n):
        for g in range(n_kv):
            p = C.softmax_weights(q[u, g].double().numpy(), k[u, g], SCALE)
            for d in range(D):  # (16 of each block's dimensions for one head after the other)
                v[u, g, :, d] = _cancelling(p[d % gqa], rng) if d % 16 else 6.0  # (scale 1 here too)
    kv, vv = torch.tensor(k).to(BF).cuda(), torch.tensor(v).to(BF).cuda()
    cache, length = rkv.kv4_cache(n, n_kv, T), _ints([0] * n)
    rkv.rkv_check_status(rkv.rkv_kv4_append(kv, vv, *cache, length, length))
    held = [C.kv4_values(cache[i].cpu().numpy(), cache[i + 1].cpu().numpy()) for i in (0, 2)]
    assert np.array_equal(held[0], k) and np.array_equal(held[1], v)
    qd = q.view(n, n_kv * gqa, D).cuda()
    out, w = torch.empty_like(qd), torch.zeros(n, n_kv, T, device="cuda")
    rkv.rkv_check_status(rkv.rkv_kv4_decode(qd, *cache, length, SCALE, out, weights=w))
    got = out.double().cpu().numpy().reshape(n, n_kv, gqa, D)
    for u in range(n):
        for g in range(n_kv):
            H.check_decode(got[u, g], w[u, g].double().cpu().numpy(), q[u, g].double().numpy(), held[0][u, g],
                           held[1][u, g], SCALE, True, 64 + T // 64, f"unit {u} head {g}", most=1e-4)
