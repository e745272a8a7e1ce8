"""Outputs, queries and workspaces of the serving step's calls that begin on 16 bytes and not on 32: what the library asks
for is 16. The results are those of arrays on 256 bytes, and nothing around the arrays is written."""
import pytest
import torch

from tests.test_gpu_serve_attention import D, Case

pytestmark = pytest.mark.gpu

SENTINEL = 768.0


def _inside(shape, dtype=torch.bfloat16, value=SENTINEL):
    """A tensor that begins 16 bytes behind a 256-byte boundary, and the array that it lies in."""
    skip = 16 // torch.empty(0, dtype=dtype).element_size()
    size = 1
    for s in shape:
        size *= s
    whole = torch.full((size + 2 * skip,), value, dtype=dtype, device="cuda")
    t = whole[skip: skip + size].view(shape)
    assert whole.data_ptr() % 256 == 0 and t.data_ptr() % 32 == 16
    return t, whole, skip


def _untouched(whole, skip, value=SENTINEL):
    assert (whole[:skip] == value).all() and (whole[-skip:] == value).all()


CASES = {
    "prompt": dict(seed=1, news=[300, 1, 65], lens=[300, 700, 65]),
    "odd group": dict(seed=2, news=[50, 9], lens=[400, 9], gqa=3),
    "paged": dict(seed=3, news=[130, 2], lens=[513, 260], block=16),
    "tree": dict(seed=4, news=[33, 8], lens=[1000, 300], words=2),
    "cut": dict(seed=5, news=[64], lens=[30000]),                # parts lie in the workspace
    "cut, few rows": dict(seed=6, news=[3], lens=[30000], gqa=5),
    "cut tree, paged": dict(seed=7, news=[16, 3], lens=[20000, 900], words=1, block=64),
    "many units": dict(seed=8, news=[2] * 80, lens=[40] * 80, n_kv=1, gqa=2),  # the plan lies there too
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_attention(name):
    from sparse_kv_cache_snapkv_gb300 import rkv
    c = Case(**CASES[name])
    want, ws = c.call()
    rkv.rkv_check_status(ws)
    c.check(want)
    shape, need = want.shape, rkv.rkv_prompt_attention_workspace_bytes(c.n, c.n_kv, c.gqa, c.tokens)
    q, _, _ = _inside(c.q.shape)
    q.copy_(c.q)
    for moved in (("out",), ("ws",), ("out", "ws", "q")):
        out, whole, skip = _inside(shape)
        room, ws_whole, ws_skip = _inside((need,), torch.uint8, 0)
        ws_whole[:ws_skip] = ws_whole[-ws_skip:] = 7
        if "q" in moved:
            c.q = q
        if "out" not in moved:
            out = torch.full_like(want, SENTINEL)
        if "ws" not in moved:
            room = None
        out, ws = c.call(out=out, ws=room)
        rkv.rkv_check_status(ws)
        assert torch.equal(out, want), moved
        _untouched(whole, skip)
        _untouched(ws_whole, ws_skip, 7)


def test_rotary_positions():
    from sparse_kv_cache_snapkv_gb300 import rkv
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(70, 12, D, generator=g, device="cuda").bfloat16()
    pos, slots = torch.arange(70, device="cuda").int(), torch.randperm(80, generator=g, device="cuda")[:70].int()
    freq = rkv.rkv_rope_frequencies()[0].cuda()
    qkv, _, _ = _inside(x.shape)
    qkv.copy_(x)
    results = []
    for source, make in ((x, lambda *s: (torch.full(s, SENTINEL, dtype=torch.bfloat16, device="cuda"), None, 0)),
                         (qkv, lambda *s: _inside(s))):
        out, kc, vc = (make(*s) for s in ((70, 8, D), (5, 2, 16, D), (5, 2, 16, D)))
        ws, _, _ = _inside((rkv.rkv_rope_append_workspace_bytes(),), torch.uint8, 0)
        q, k, v = source.split((8, 2, 2), 1)
        rkv.rkv_check_status(rkv.rkv_rope_append(q, k, v, pos, freq, slots, out[0], kc[0], vc[0], ws=ws))
        results.append((out[0], kc[0], vc[0]))
        for _, whole, skip in (out, kc, vc):
            if whole is not None:
                _untouched(whole, skip)
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("room", [100, 9001])
def test_places(room):
    from sparse_kv_cache_snapkv_gb300 import rkv
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    new, ln, held = ints([room - 40, 0, 30]), ints([3, 0, 16]), ints([1, 0, 1])
    free, count = torch.randperm(1000, device="cuda").int(), ints([900])
    results = []
    for off in (0, 16):
        o = []
        for m in (4, room, room, 3, 3, 1):
            o.append(_inside((m,), torch.int32, -9)[0] if off else torch.full((m,), -9, dtype=torch.int32, device="cuda"))
        table = torch.full((3, 700), 999, dtype=torch.int32, device="cuda")
        ws = _inside((rkv.rkv_reserve_slots_workspace_bytes(3),), torch.uint8, 0)[0] if off else None
        rkv.rkv_check_status(rkv.rkv_reserve_slots(new, ln, held, table, free, count, 16, *o, ws=ws))
        stack, left = free.clone(), o[5].clone()
        ws = _inside((rkv.rkv_release_blocks_workspace_bytes(3),), torch.uint8, 0)[0] if off else None
        rkv.rkv_check_status(rkv.rkv_release_blocks(ints([0, 0, 0]), o[4], table, stack, left, 16, o[4].clone(), left, ws=ws))
        results.append((table, stack, left, *o))
    assert all(torch.equal(a, b) for a, b in zip(*results))
