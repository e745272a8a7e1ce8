"""Arrays that are slices of larger ones: what need not begin on 16 bytes, and the decodes' refusal."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128
SCALE = 1.0 / math.sqrt(D)


@pytest.fixture(scope="module")
def rkv():
    from sparse_kv_cache_snapkv_gb300 import rkv
    rkv.load()
    return rkv


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def test_prompt_and_evict_take_slices_of_units(rkv):
    n, n_kv, gqa, cap, keep = 2, 1, 2, 301, 200
    k, q = _rand(1, n, n_kv, cap, D), _rand(2, n, n_kv * gqa, cap, D)
    ln = _ints([cap, 250])
    res = []
    for sliced in (False, True):
        w = torch.zeros(n + 1, n_kv, cap, device="cuda")[1:] if sliced else torch.zeros(n, n_kv, cap, device="cuda")
        pos = torch.full((n + 1, n_kv, cap), -1, dtype=torch.int32, device="cuda")
        pos = pos[1:] if sliced else pos[:n]
        assert (w.data_ptr() % 16 != 0) == sliced
        rkv.rkv_check_status(rkv.rkv_prompt_weights(q, ln, k, ln, SCALE, w))
        kk, vv, length, src = k.clone(), k.clone(), ln.clone(), torch.zeros(n, n_kv, keep, dtype=torch.int32, device="cuda")
        rkv.rkv_check_status(rkv.rkv_evict(kk, vv, length, w, pos, ln, keep, 8, length, w, pos, src_rows=src))
        res.append((kk, vv, w, pos, length, src))
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_decodes_say_why_they_refuse_a_slice(rkv):
    """(rkv_dense_decode_weights without weights: as any other array that is missing.)"""
    n, n_kv, gqa, cap = 2, 1, 2, 33
    q, out = _rand(3, n, n_kv * gqa, D), torch.zeros(n, n_kv * gqa, D, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(n + 1, n_kv, cap, device="cuda")
    k = _rand(4, n, n_kv, cap, D)
    ln = _ints([cap] * n)
    cache = rkv.kv4_cache(n, n_kv, cap)
    with pytest.raises(ValueError, match="16-byte"):
        rkv.rkv_dense_decode_weights(q, k, k, ln, SCALE, out, w[1:])
    with pytest.raises(ValueError, match="16-byte"):
        rkv.rkv_kv4_decode(q, *cache, ln, SCALE, out, weights=w[1:])
    pools, table = rkv.kv4_cache(4, n_kv, 16), _ints([[0], [1]])
    with pytest.raises(ValueError, match="16-byte"):
        rkv.rkv_kv4_decode_paged(q, *pools, table, _ints([3, 3]), SCALE, out,
                                 weights=torch.zeros(n * n_kv * 16 + 1, device="cuda")[1:].view(n, n_kv, 16))
    with pytest.raises(TypeError, match="weights must be a tensor"):
        rkv.rkv_dense_decode_weights(q, k, k, ln, SCALE, out, None)
    assert not w.any() and not out.any()
    rkv.rkv_check_status(rkv.rkv_dense_decode_weights(q, k, k, ln, SCALE, out, w[:n]))  # the first units do
    assert w[:n].any() and not w[n:].any()
