"""The bounded waits of the prompt weights' kernels, made to run out without any GPU fault.

rkv_testing_prompt_wait_timeout (include/rkv_testing.h) never requests one load of block 0, so that
the waits of every role of that block run out: the host reads RKV_DEV_WAIT_TIMEOUT, the other
units' weights are right, and a normal call afterwards (which needs the tensor memory that the block
held) matches the oracle.
"""
import math

import pytest
import torch

from oracle import cache as C
from tests import cache_parity as P

pytestmark = pytest.mark.gpu

D = 128
SCALE = 1.0 / math.sqrt(D)
KEYS, QUERIES, SUMS = 1, 2, 3


def _check(w, q, k, lens, news, gqa, units):
    n_kv = k.shape[1]
    for u in units:
        for g in range(n_kv):
            hk = k[u, g, :lens[u]].double().cpu().numpy()
            hq = q[u, g * gqa:(g + 1) * gqa, :news[u]].double().cpu().numpy()
            P.check_weights(w[u, g, :lens[u]].double().cpu().numpy(), C.prompt_weights(hq, hk, SCALE),
                            0 * hk[:, 0], hq.reshape(-1, D), hk, SCALE, 96 + lens[u] // 16 + gqa * news[u] // 64,
                            f"unit {u} head {g}")


# many more items than SMs with few tiles each (block 0 goes on to others), and fewer with many
@pytest.mark.parametrize("n,n_kv,gqa,max_q,lens,news", [
    (2, 1, 2, 700, [700, 640], [700, 600]),        # a tile holds rows of one head
    (2, 2, 4, 100, [1500, 900], [100, 99]),        # a tile runs on through the heads
    (24, 2, 4, 512, [512] * 24, [512] * 24),
])
@pytest.mark.parametrize("what", [KEYS, QUERIES, SUMS])
def test_prompt_wait_runs_out_and_context_survives(n, n_kv, gqa, max_q, lens, news, what):
    from sparse_kv_cache_snapkv_gb300 import rkv
    rkv.load()
    g = torch.Generator(device="cuda").manual_seed(what)
    k = torch.randn(n, n_kv, max(lens), D, generator=g, device="cuda").bfloat16()
    q = torch.randn(n, n_kv * gqa, max_q, D, generator=g, device="cuda").bfloat16()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ql, ln = ints(news), ints(lens)
    w = torch.zeros(n, n_kv, max(lens), device="cuda")
    for _ in range(2):  # (the second finds what the first left)
        ws = rkv.rkv_testing_prompt_wait_timeout(q, ql, k, ln, SCALE, w, what, 2_000_000)
        with pytest.raises(rkv.RkvError) as e:
            rkv.rkv_check_status(ws)
        assert e.value.code == 5 and e.value.bits == 0x4, e.value
        rkv.rkv_check_status(ws)  # the read cleared the status word
    w.zero_()
    rkv.rkv_check_status(rkv.rkv_prompt_weights(q, ql, k, ln, SCALE, w, ws=ws))
    _check(w, q, k, lens, news, gqa, range(min(n, 3)))


@pytest.mark.parametrize("max_q,cap", [(600, 900), (90, 900)])
def test_the_shortest_limit(max_q, cap):
    """A microsecond, which no wait for memory meets: every block gives up with copies and products on their
    way, lets those land, and the next call is right."""
    from sparse_kv_cache_snapkv_gb300 import rkv
    rkv.load()
    n, n_kv, gqa = 12, 2, 4
    g = torch.Generator(device="cuda").manual_seed(9)
    k = torch.randn(n, n_kv, cap, D, generator=g, device="cuda").bfloat16()
    q = torch.randn(n, n_kv * gqa, max_q, D, generator=g, device="cuda").bfloat16()
    ql, ln = (torch.full((n,), x, dtype=torch.int32, device="cuda") for x in (max_q, cap))
    w = torch.zeros(n, n_kv, cap, device="cuda")
    for what in (KEYS, QUERIES, SUMS):
        ws = rkv.rkv_testing_prompt_wait_timeout(q, ql, k, ln, SCALE, w, what, 1000)
        with pytest.raises(rkv.RkvError) as e:
            rkv.rkv_check_status(ws)
        assert e.value.bits == 0x4
    w.zero_()
    rkv.rkv_check_status(rkv.rkv_prompt_weights(q, ql, k, ln, SCALE, w, ws=ws))
    _check(w, q, k, [cap] * n, [max_q] * n, gqa, (0, n - 1))
