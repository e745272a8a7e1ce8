"""What the cache calls promise before any launch: hooks' refusals and workspace sizes. No GPU needed."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(1 << 20)   # aligned, non-null, never dereferenced: calls fail validation
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from sparse_kv_cache_snapkv_gb300 import _build, rkv
    _build.build()
    return rkv.load()


def test_prompt_timeout_hook_refusals(lib):
    v = FAKE
    ok = dict(q=v, q_len=v, k=v, len=v, n=1, n_kv=2, gqa=4, head_dim=128, max_q=64, max_len=128, scale=0.1,
              weights=v, what=1, limit=10**6, ws=v, ws_bytes=BIG, stream=None)
    for change, code in ((dict(what=0), 1), (dict(what=4), 1), (dict(limit=999), 1), (dict(limit=10**9 + 1), 1),
                         (dict(head_dim=64), 2), (dict(weights=None), 1), (dict(ws_bytes=300), 3)):
        assert lib.rkv_testing_prompt_wait_timeout(*{**ok, **change}.values()) == code, change
