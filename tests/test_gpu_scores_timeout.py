"""The score passes' bounded waits run out for both of their row layouts (128 and 256 window rows of
a KV group) and for a block that serves one item or many, and the context stays usable."""
import math

import numpy as np
import pytest
import torch

from oracle import rocketkv as O

pytestmark = pytest.mark.gpu

D = 128


@pytest.mark.parametrize("n,n_kv,gqa,window,lens", [
    (2, 2, 4, 32, [2048, 1001]),       # 128 rows
    (2, 2, 8, 32, [2048, 1001]),       # 256 rows
    (200, 1, 4, 16, [400] * 200),      # more items than SMs
    (200, 1, 8, 32, [400] * 200),
])
def test_score_waits_run_out(n, n_kv, gqa, window, lens):
    from sparse_kv_cache_snapkv_gb300 import rkv
    rkv.load()
    g = torch.Generator(device="cuda").manual_seed(7)
    k = torch.randn(n, n_kv, max(lens), D, generator=g, device="cuda").bfloat16()
    q = torch.randn(n, n_kv * gqa, window, D, generator=g, device="cuda").bfloat16()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scale = 1.0 / math.sqrt(D)
    scores = torch.zeros(n, n_kv, max(lens) - window, device="cuda")
    for _ in range(2):
        ws = rkv.rkv_testing_scores_wait_timeout(k, ln, q, scale, scores, wait_limit_ns=2_000_000)
        with pytest.raises(rkv.RkvError) as e:
            rkv.rkv_check_status(ws)
        assert e.value.code == 5 and e.value.bits == 0x4, e.value
    rkv.rkv_check_status(rkv.rkv_snapkv_scores(k, ln, q, scale, scores))
    for u in (0, 1, n - 1):
        for h in range(n_kv):
            ref = O.window_scores(k[u, h, :lens[u]].double().cpu().numpy(),
                                  q[u, h * gqa:(h + 1) * gqa].double().cpu().numpy(), scale)
            got = scores[u, h, :lens[u] - window].double().cpu().numpy()
            assert (np.abs(got - ref) <= 1e-4 * np.abs(ref) + 1e-30).all(), (u, h)


@pytest.mark.parametrize("gqa", [4, 8])
def test_the_shortest_limit(gqa):
    """A microsecond, which no wait for memory meets: every block gives up with copies and products on their
    way, lets those land, and the next call is right."""
    from sparse_kv_cache_snapkv_gb300 import rkv
    rkv.load()
    n, window, L = 200, 32, 1500
    g = torch.Generator(device="cuda").manual_seed(8)
    k = torch.randn(n, 1, L, D, generator=g, device="cuda").bfloat16()
    q = torch.randn(n, gqa, window, D, generator=g, device="cuda").bfloat16()
    ln = torch.full((n,), L, dtype=torch.int32, device="cuda")
    scale = 1.0 / math.sqrt(D)
    scores = torch.zeros(n, 1, L - window, device="cuda")
    ws = rkv.rkv_testing_scores_wait_timeout(k, ln, q, scale, scores, wait_limit_ns=1000)
    with pytest.raises(rkv.RkvError) as e:
        rkv.rkv_check_status(ws)
    assert e.value.bits == 0x4
    rkv.rkv_check_status(rkv.rkv_snapkv_scores(k, ln, q, scale, scores))
    for u in (0, n - 1):
        ref = O.window_scores(k[u, 0].double().cpu().numpy(), q[u].double().cpu().numpy(), scale)
        got = scores[u, 0].double().cpu().numpy()
        assert (np.abs(got - ref) <= 1e-4 * np.abs(ref) + 1e-30).all(), u
