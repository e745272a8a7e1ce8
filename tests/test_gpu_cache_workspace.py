"""Workspaces of the cache calls: nothing is written behind the size asked for, and one made for the
largest shape serves smaller ones whose own work is split further."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128
SCALE = 1.0 / math.sqrt(D)
GUARD = 1 << 16


@pytest.fixture(scope="module")
def rkv():
    from sparse_kv_cache_snapkv_gb300 import rkv
    rkv.load()
    return rkv


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


class _Guarded:
    """A workspace of `size` bytes with others behind it."""

    def __init__(self, size):
        self.all = torch.full((size + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
        self.all[:256] = 0
        self.ws = self.all[:size]

    def check(self, rkv):
        rkv.rkv_check_status(self.ws)
        assert (self.all[len(self.ws):] == 0x5A).all()


def _decode(rkv, n, n_kv, gqa, cap, ws, kv4):
    q, out = _rand(1, n, n_kv * gqa, D), torch.empty(n, n_kv * gqa, D, dtype=torch.bfloat16, device="cuda")
    w, ln = torch.zeros(n, n_kv, cap, device="cuda"), _ints([cap - u % 3 if cap > 3 else cap for u in range(n)])
    if kv4:
        cache = [(torch.arange(n * n_kv * cap * x, device="cuda") % 113).to(torch.uint8).view(n, n_kv, cap, x)
                 for x in (64, 8, 64, 8)]
        rkv.rkv_kv4_decode(q, *cache, ln, SCALE, out, weights=w, ws=ws)
    else:
        rkv.rkv_dense_decode_weights(q, _rand(2, n, n_kv, cap, D), _rand(3, n, n_kv, cap, D), ln, SCALE, out, w, ws=ws)
    return out, w


@pytest.mark.parametrize("kv4", [True, False])
def test_decode_workspace(rkv, kv4):
    shapes = [(20, 8, 4, 256), (19, 8, 4, 256), (1, 1, 1, 1), (1, 8, 4, 256), (3, 1, 2, 255)]
    largest = _Guarded(rkv.rkv_kv4_decode_workspace_bytes(20, 8, 4, 256, True))
    for s in shapes:
        own = _Guarded(rkv.rkv_kv4_decode_workspace_bytes(*s, True))
        a, b = _decode(rkv, *s, own.ws, kv4), _decode(rkv, *s, largest.ws, kv4)
        own.check(rkv)
        largest.check(rkv)
        assert all(torch.equal(x, y) for x, y in zip(a, b)), s


def test_prompt_workspace(rkv):
    shapes = [(1, 2, 2, 600, 4096), (1, 2, 2, 600, 600), (1, 1, 1, 1, 2000), (2, 2, 2, 40, 600), (1, 2, 2, 256, 4096)]
    largest = _Guarded(rkv.rkv_prompt_weights_workspace_bytes(2, 2, 2, 600, 4096))
    for n, n_kv, gqa, max_q, cap in shapes:
        q, k = _rand(4, n, n_kv * gqa, max_q, D), _rand(5, n, n_kv, cap, D)
        own = _Guarded(rkv.rkv_prompt_weights_workspace_bytes(n, n_kv, gqa, max_q, cap))
        res = []
        for g in (own, largest):
            w = torch.zeros(n, n_kv, cap, device="cuda")
            rkv.rkv_prompt_weights(q, _ints([max_q] * n), k, _ints([cap] * n), SCALE, w, ws=g.ws)
            g.check(rkv)
            res.append(w)
        assert torch.equal(*res)


def test_evict_workspace(rkv):
    largest = _Guarded(rkv.rkv_evict_workspace_bytes(2, 4, 8192, 8000))
    for keep in (8000, 4096, 8191, 1):
        own = _Guarded(rkv.rkv_evict_workspace_bytes(2, 4, 8192, keep))
        res = []
        for g in ((own, largest) if keep <= 8000 else (own,)):
            k, v = _rand(6, 2, 4, 8192, D), _rand(7, 2, 4, 8192, D)
            w = torch.rand(2, 4, 8192, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda")
            pos, ln = torch.full((2, 4, 8192), -1, dtype=torch.int32, device="cuda"), _ints([8192, 8190])
            rkv.rkv_evict(k, v, ln, w, pos, ln.clone(), keep, 1, ln, w, pos, ws=g.ws)
            g.check(rkv)
            res.append((k, v, w, pos, ln))
        assert all(torch.equal(x, y) for r in res[1:] for x, y in zip(res[0], r))
