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


def _decode_both(rkv, q, k, v, gqa, kv4):
    """q [n, gqa, D], k, v [n, 1, T, D]: outputs and weights, and the numbers that the cache holds."""
    n, _, T, _ = k.shape
    q, k, v = q.to(BF).cuda(), k.to(BF).cuda(), v.to(BF).cuda()
    out, w, length = torch.empty_like(q), torch.zeros(n, 1, T, device="cuda"), _ints([0] * n)
    if kv4:
        cache = rkv.kv4_cache(n, 1, T)
        rkv.rkv_check_status(rkv.rkv_kv4_append(k, v, *cache, length, length))
        rkv.rkv_check_status(rkv.rkv_kv4_decode(q, *cache, length, SCALE, out, weights=w))
        held = [C.kv4_values(cache[i].cpu().numpy(), cache[i + 1].cpu().numpy()) for i in (0, 2)]
    else:
        rkv.rkv_check_status(rkv.rkv_dense_decode_weights(q, k, v, _ints([T] * n), SCALE, out, w))
        held = [x.double().cpu().numpy() for x in (k, v)]
    for u in range(n):
        H.check_decode(out[u].double().cpu().numpy(), w[u, 0].double().cpu().numpy(), q[u].double().cpu().numpy(),
                       held[0][u, 0], held[1][u, 0], SCALE, kv4, 64 + T // 64, f"unit {u}")


@pytest.mark.parametrize("kv4", [True, False])
@pytest.mark.parametrize("gqa", [2, 4, 8])
@pytest.mark.parametrize("T", [33, 1500])
def test_heads_of_very_different_size(rkv, gqa, T, kv4):
    """Keys with scales near the top of the 4-bit format and query heads from 2^-40 to some 100 of logit:
    each head has its own power of two on the way into the product, and its own tolerance here."""
    g = torch.Generator().manual_seed(T + gqa)
    n = 3
    q = torch.randn(n, gqa, D, generator=g)
    k = torch.randn(n, 1, T, D, generator=g) * torch.tensor([3000.0, 3000.0, 2.0 ** -6]).view(n, 1, 1, 1)
    for h in range(gqa):
        q[0, h] *= 2.0 ** (-9 - [0, 3, 31, 12, 1, 5, 20, 8][h])
        q[1, h] *= 2.0 ** (-9 - [12, 0, 8, 2, 40, 1, 3, 2][h])
        q[2, h] *= 2.0 ** (10 - [0, 30, 3, 6, 1, 50, 2, 9][h])
    q[0, 0, ::2] *= 2.0 ** -16   # a head whose values reach over more bits than fp16 has
    q[2, 1, 1::3] = 0.0
    v = torch.randn(n, 1, T, D, generator=g) * torch.tensor([1.0, 5000.0, 2.0 ** -8]).view(n, 1, 1, 1)
    _decode_both(rkv, q, k, v, gqa, kv4)


@pytest.mark.parametrize("kv4", [True, False])
@pytest.mark.parametrize("T", [400, 5000])
def test_maximum_that_moves(rkv, T, kv4):
    """Logits that rise or fall along the sequence, in steps of less and of more than the lag that the running
    maximum is allowed, and one token far above the rest; each for another head."""
    g = torch.Generator().manual_seed(T)
    n, gqa = 4, 4
    q = torch.randn(n, gqa, D, generator=g)
    unit = q / q.norm(dim=-1, keepdim=True)
    ramp = torch.linspace(-1, 1, T).view(T, 1)
    k = torch.randn(n, 1, T, D, generator=g) * 0.1
    k[0, 0] += ramp * unit[0, 0] * 40
    k[1, 0] -= ramp * unit[1, 1] * 120
    k[2, 0, T // 3] += unit[2, 2] * 60
    k[3, 0] += ramp.abs() * unit[3, 3] * 100 - ramp * unit[3, 0] * 9
    v = torch.randn(n, 1, T, D, generator=g)
    _decode_both(rkv, q, k, v, gqa, kv4)
