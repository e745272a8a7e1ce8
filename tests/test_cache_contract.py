"""What the cache calls promise before any launch: hooks' refusals and workspace sizes. No GPU needed."""
import ctypes
import random

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


# the arguments of each *_workspace_bytes: (smallest, largest) or the choices
SIZES = {
    "rkv_kv4_append_workspace_bytes": [(1, 4096)],
    "rkv_kv4_decode_workspace_bytes": [(1, 64), (1, 16), [1, 2, 4, 8], (1, 1 << 20), [0, 1]],
    "rkv_dense_decode_weights_workspace_bytes": [(1, 64), (1, 16), [1, 2, 4, 8], (1, 1 << 20)],
    "rkv_prompt_weights_workspace_bytes": [(1, 64), (1, 16), (1, 64), (1, 1 << 15), (1 << 15, 1 << 18)],
    "rkv_evict_workspace_bytes": [(1, 600), (1, 16), (1, 1 << 20), (1, 1 << 20)],
}


def _pick(rng, span, at_least=None):
    if isinstance(span, list):
        return rng.choice([x for x in span if at_least is None or x >= at_least])
    low = span[0] if at_least is None else at_least
    if rng.random() < 0.3:  # next door
        return min(span[1], low + rng.randint(0, 2))
    return int(round(low * (span[1] / low) ** rng.random()))


@pytest.mark.parametrize("name", sorted(SIZES))
def test_workspaces_do_not_shrink(lib, name):
    rng, size = random.Random(name), getattr(lib, name)
    for _ in range(4000):
        a = [_pick(rng, s) for s in SIZES[name]]
        b = [_pick(rng, s, x) if rng.random() < 0.5 else x for s, x in zip(SIZES[name], a)]
        assert 256 <= size(*a) <= size(*b), (a, b)


@pytest.mark.parametrize("name,small,large", [
    ("rkv_prompt_weights_workspace_bytes", (1, 8, 4, 8192, 8192), (1, 8, 4, 8192, 32768)),
    ("rkv_kv4_decode_workspace_bytes", (19, 8, 4, 256, 0), (20, 8, 4, 256, 0)),
    ("rkv_evict_workspace_bytes", (1, 8, 8192, 4096), (1, 8, 8192, 8000)),
])
def test_workspace_of_the_larger_shape_serves(lib, name, small, large):
    size = getattr(lib, name)
    assert size(*small) <= size(*large)


def test_prompt_workspace_of_what_is_refused_is_none(lib):
    size, top = lib.rkv_prompt_weights_workspace_bytes, 2**31 - 1
    for a in ((1, 1, 1, 1, top), (1, 1, 64, top // 64, top), (2, 1, 1, 1, 2**30), (1, 8, 64, 2**22, 2**22),
              (1, 1, 65, 1, 1), (1, 1, 1, 2, 1), (0, 1, 1, 1, 1)):
        assert size(*a) == 0, a
    # the largest that are taken
    assert 256 < size(1, 1, 1, 1, top - 512) < 2**20  # (one query: a tile's sums, splits of at most the SMs' number)
    assert size(1, 1, 1, top - 512, top - 512) >= 4 * (top - 512)


ODD = ctypes.c_void_p((1 << 20) + 8)


def test_decode_weights_begin_on_16_bytes(lib):
    """As include/rkv.h says of every decode that takes them."""
    v = FAKE
    dense = dict(q=v, k=v, v=v, len=v, n=1, n_kv=2, gqa=4, head_dim=128, max_len=64, scale=0.1, out=v, weights=ODD,
                 ws=v, ws_bytes=BIG, stream=None)
    assert lib.rkv_dense_decode_weights(*dense.values()) == 1
    paged = dict(q=v, new_k=None, new_v=None, kc=v, ks=v, vc=v, vs=v, table=v, len=v, len_out=None, n=1, n_kv=2,
                 gqa=4, head_dim=128, num_blocks=4, block=16, max_blocks=2, scale=0.1, out=v, weights=ODD, ws=v,
                 ws_bytes=BIG, stream=None)
    assert lib.rkv_kv4_decode_paged(*paged.values()) == 1
    import os
    with open(os.path.join(os.path.dirname(__file__), "..", "include", "rkv.h")) as f:
        header = f.read()
    for call in ("weights NULL or [n][n_kv][cap] fp32, 16-byte aligned",
                 "weights [n][n_kv][max_len] fp32, 16-byte aligned"):
        assert call in header
