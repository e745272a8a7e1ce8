"""A serving step with fewer free blocks than its requests need: the README's step reports it, the requests that are served
are right, and nothing of the others changes in the cache."""
import math
import os
import re

import numpy as np
import pytest
import torch

from oracle import serve as S
from tests import serve_parity as P

pytestmark = pytest.mark.gpu

D = 128
N_KV, HQ, BLOCK, BLOCKS, MOST = 2, 8, 16, 12, 6
SCALE = 1 / math.sqrt(D)


def _readme():
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), flags=re.S)
    code = [b for b in blocks if "rkv_reserve_slots" in b]
    assert len(code) == 1
    return code[0]


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _state(new, old, held, free, seed):
    """Requests of old[u] cached tokens in held[u] blocks, `free` blocks left, new[u] tokens to come."""
    from sparse_kv_cache_snapkv_gb300 import rkv
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, tokens = len(new), sum(new)
    perm = torch.randperm(BLOCKS, generator=g, device="cuda").int()
    table = torch.full((n, MOST), -1, dtype=torch.int32, device="cuda")
    at = 0
    for u, h in enumerate(held):
        table[u, :h] = perm[at: at + h]
        at += h
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return dict(rkv=rkv, torch=torch, n=n, n_kv=N_KV, hq=HQ, block=BLOCK, scale=SCALE, new_len=_ints(new),
                length=_ints(old), held=_ints(held), table=table, free=perm[at:].clone() if at else perm, count=_ints([free]),
                q_start=_ints([0] * (n + 1)), slots=_ints([0] * tokens), positions=_ints([0] * tokens),
                qkv=normal(tokens, HQ + 2 * N_KV, D), q_turned=torch.zeros(tokens, HQ, D, dtype=torch.bfloat16, device="cuda"),
                out=torch.zeros(tokens, HQ, D, dtype=torch.bfloat16, device="cuda"),
                k_pool=normal(BLOCKS, N_KV, BLOCK, D), v_pool=normal(BLOCKS, N_KV, BLOCK, D))


def _padded(v):
    """The free stack as an array of all blocks, of which the first `count` are on it."""
    free = torch.full((BLOCKS,), -1, dtype=torch.int32, device="cuda")
    free[: len(v["free"])] = v["free"]
    v["free"] = free
    return v


def test_the_readme_step_reports_requests_that_are_not_served():
    from sparse_kv_cache_snapkv_gb300 import rkv
    # request 0 needs two more blocks and one is free; it has more cached rows than new ones, so that the attention by
    # itself finds nothing wrong. Request 1 has room in the block that it holds.
    new, old, held = [30, 3], [40, 10], [3, 1]
    v = _padded(_state(new, old, held, 1, 1))
    pools = [v[p].clone() for p in ("k_pool", "v_pool")]
    with pytest.raises(rkv.RkvError) as e:
        exec(_readme(), v)
    assert e.value.bits == 0x20  # RKV_DEV_NO_BLOCKS
    assert v["length"].tolist() == [40, 13] and v["held"].tolist() == held and v["count"].tolist() == [1]
    assert v["q_start"].tolist() == [0, 30, 33] and (v["slots"][:30] == -1).all()
    assert (v["q_turned"][:30] == 0).all()
    mine = int(v["table"][1, 0])
    for p, was in zip(("k_pool", "v_pool"), pools):
        was[mine, :, 10:13] = v[p][mine, :, 10:13]
        assert torch.equal(v[p], was)
    q, out = (v[x][30:].double().cpu().numpy() for x in ("q_turned", "out"))
    k, w = (v[p][mine, :, :13].double().cpu().numpy() for p in ("k_pool", "v_pool"))
    ref, mag = S.attention(q, k, w, SCALE, S.visible(3, 13))
    P.within(out, ref, P.attention_tolerance(q, k, SCALE, ref, mag), "the request that was served")


def test_the_next_step_serves_it():
    """After blocks came back, the same request with the same tokens."""
    from sparse_kv_cache_snapkv_gb300 import rkv
    v = _padded(_state([30, 3], [40, 10], [3, 1], 1, 2))
    with pytest.raises(rkv.RkvError):
        exec(_readme(), v)
    v["free"][1], v["count"][0] = int((set(range(BLOCKS)) - set(v["table"].flatten().tolist()) -
                                       set(v["free"].tolist()[:1])).pop()), 2
    v["new_len"][1] = 0
    exec(_readme(), v)
    assert v["length"].tolist() == [70, 13] and v["held"].tolist() == [5, 1] and v["count"].tolist() == [0]
    rows = v["table"][0, :5].long()
    k, w = (v[p][rows].transpose(0, 1).flatten(1, 2)[:, :70].double().cpu().numpy() for p in ("k_pool", "v_pool"))
    q, out = (v[x][:30].double().cpu().numpy() for x in ("q_turned", "out"))
    ref, mag = S.attention(q, k, w, SCALE, S.visible(30, 70))
    assert np.isfinite(out).all()
    P.within(out, ref, P.attention_tolerance(q, k, SCALE, ref, mag), "the request, later")
