"""What the serving step's calls promise before any launch: refusals, workspace sizes, frequencies. No GPU needed."""
import ctypes
import random

import numpy as np
import pytest

from oracle import serve as S

FAKE = ctypes.c_void_p(1 << 20)   # aligned, non-null, never dereferenced: calls fail validation
ODD = ctypes.c_void_p((1 << 20) + 8)
OTHER = ctypes.c_void_p(1 << 21)
BIG = 1 << 45
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    from sparse_kv_cache_snapkv_gb300 import _build, rkv
    _build.build()
    return rkv.load()


RESERVE = dict(new_len=FAKE, len=FAKE, held=FAKE, table=FAKE, free=FAKE, count=FAKE, n=4, num_blocks=100, block=16,
               max_blocks=10, max_tokens=64, q_start=FAKE, slots=FAKE, positions=FAKE, len_out=FAKE, held_out=FAKE,
               count_out=FAKE, ws=FAKE, ws_bytes=BIG, stream=None)
RELEASE = dict(len=FAKE, held=FAKE, table=FAKE, free=FAKE, count=FAKE, n=4, num_blocks=100, block=16, max_blocks=10,
               held_out=FAKE, count_out=FAKE, ws=FAKE, ws_bytes=BIG, stream=None)
ROPE = dict(q=FAKE, q_stride=1024, k=FAKE, k_stride=256, v=FAKE, v_stride=256, positions=FAKE, inv_freq=FAKE, slots=FAKE,
            tokens=5, hq=8, n_kv=2, head_dim=128, rot_dim=128, interleaved=0, mscale=1.0, q_out=OTHER, k_pool=FAKE,
            v_pool=FAKE, num_blocks=10, block=16, ws=FAKE, ws_bytes=BIG, stream=None)
PROMPT = dict(q=FAKE, q_stride=1024, q_start=FAKE, k=FAKE, v=FAKE, len=FAKE, n=2, n_kv=2, gqa=4, head_dim=128, tokens=9,
              max_len=64, scale=0.1, out=OTHER, ws=FAKE, ws_bytes=BIG, stream=None)
PAGED = dict(q=FAKE, q_stride=1024, q_start=FAKE, k=FAKE, v=FAKE, table=FAKE, len=FAKE, n=2, n_kv=2, gqa=4, head_dim=128,
             tokens=9, num_blocks=8, block=16, max_blocks=4, scale=0.1, out=OTHER, ws=FAKE, ws_bytes=BIG, stream=None)


def _with_mask(d):
    out = {}
    for k, v in d.items():
        out[k] = v
        if k == "q_start":
            out.update(mask=FAKE, words=2)
    return out


TREE, TREE_PAGED = _with_mask(PROMPT), _with_mask(PAGED)
HOOK = {}
for _k, _v in PROMPT.items():
    HOOK[_k] = _v
    if _k == "out":
        HOOK.update(what=1, limit=10 ** 6)

ATTENTION = [(dict(head_dim=64), 2), (dict(gqa=65), 2), (dict(gqa=0), 1), (dict(n=0), 1), (dict(n_kv=0), 1),
             (dict(tokens=0), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
             (dict(scale=float("inf")), 1), (dict(q=None), 1), (dict(q=ODD), 1), (dict(k=ODD), 1), (dict(v=ODD), 1),
             (dict(out=ODD), 1), (dict(out=FAKE), 1), (dict(q_start=None), 1), (dict(len=None), 1), (dict(v=None), 1),
             (dict(out=None), 1), (dict(q_stride=1020), 1), (dict(q_stride=1016), 1), (dict(q_stride=-1024), 1),
             (dict(ws=None), 3), (dict(ws=ODD), 3), (dict(ws_bytes=1000), 3), (dict(tokens=TOP // 8), 6)]
SIZES = [(dict(n=0), 1), (dict(n=TOP), 1), (dict(num_blocks=0), 1), (dict(block=0), 1), (dict(max_blocks=0), 1),
         (dict(block=-16), 1), (dict(num_blocks=2 ** 27), 1), (dict(max_blocks=2 ** 27), 1), (dict(ws=None), 3),
         (dict(ws_bytes=256), 3)]
CALLS = {
    "rkv_reserve_slots": (RESERVE, SIZES + [({k: None}, 1) for k, v in RESERVE.items() if v is FAKE and k != "ws"] +
                          [(dict(max_tokens=0), 1), (dict(max_tokens=2 ** 30 + 1), 1)]),
    "rkv_release_blocks": (RELEASE, SIZES + [({k: None}, 1) for k, v in RELEASE.items() if v is FAKE and k != "ws"]),
    "rkv_rope_append": (ROPE, [(dict(head_dim=64), 2), (dict(rot_dim=0), 2), (dict(rot_dim=24), 2), (dict(rot_dim=144), 2),
                               (dict(tokens=0), 1), (dict(hq=0), 1), (dict(n_kv=0), 1), (dict(num_blocks=0), 1),
                               (dict(block=0), 1), (dict(q_stride=1016), 1), (dict(k_stride=250), 1), (dict(v_stride=0), 1),
                               (dict(k_stride=128), 1), (dict(interleaved=2), 1), (dict(mscale=float("inf")), 1),
                               (dict(q=ODD), 1), (dict(q_out=ODD), 1), (dict(k_pool=ODD), 1), (dict(slots=None), 1),
                               (dict(q_out=FAKE, q_stride=1280), 1), (dict(inv_freq=None), 1), (dict(positions=None), 1),
                               (dict(ws_bytes=255), 3), (dict(ws=None), 3)]),
    "rkv_prompt_attention": (PROMPT, ATTENTION + [(dict(max_len=0), 1), (dict(max_len=2 ** 30 + 1), 1),
                                                  (dict(max_len=2 ** 30), 6)]),
    "rkv_prompt_attention_paged": (PAGED, ATTENTION + [(dict(block=24), 1), (dict(table=None), 1), (dict(num_blocks=0), 1),
                                                       (dict(num_blocks=2 ** 27), 6), (dict(max_blocks=2 ** 27), 1)]),
    "rkv_tree_attention": (TREE, ATTENTION + [(dict(mask=None), 1), (dict(words=0), 1), (dict(words=33), 1)]),
    "rkv_tree_attention_paged": (TREE_PAGED, ATTENTION + [(dict(mask=None), 1), (dict(words=-1), 1), (dict(table=None), 1)]),
    "rkv_testing_attention_wait_timeout": (HOOK, ATTENTION + [(dict(what=0), 1), (dict(what=4), 1), (dict(limit=999), 1),
                                                              (dict(limit=10 ** 9 + 1), 1)]),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_refusals(lib, name):
    ok, changes = CALLS[name]
    for change, code in changes:
        assert set(change) <= set(ok), change
        assert getattr(lib, name)(*{**ok, **change}.values()) == code, change


WORKSPACES = {
    "rkv_reserve_slots_workspace_bytes": [(1, 100000)],
    "rkv_release_blocks_workspace_bytes": [(1, 100000)],
    "rkv_prompt_attention_workspace_bytes": [(1, 5000), (1, 16), (1, 64), (1, 1 << 20)],
}


@pytest.mark.parametrize("name", sorted(WORKSPACES))
def test_workspaces_do_not_shrink(lib, name):
    rng, size = random.Random(name), getattr(lib, name)
    for _ in range(4000):
        a = [int(round(lo * (hi / lo) ** rng.random())) for lo, hi in WORKSPACES[name]]
        b = [min(hi, x + rng.choice((0, 0, 1, 2, x))) for x, (_, hi) in zip(a, WORKSPACES[name])]
        assert 256 <= size(*a) <= size(*b), (a, b)


def test_workspaces_of_what_is_refused(lib):
    size = lib.rkv_prompt_attention_workspace_bytes
    for a in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 65, 1), (1, 1, 1, 0), (1, 8, 64, 2 ** 22), (TOP, 1, 1, 1)):
        assert size(*a) == 0, a
    assert lib.rkv_reserve_slots_workspace_bytes(0) == lib.rkv_release_blocks_workspace_bytes(-1) == 0


@pytest.mark.parametrize("kind,extra", [("plain", {}), ("linear", dict(factor=8.0)), ("base", dict(factor=4.0)),
                                        ("by_parts", dict(factor=16.0, ctx=4096)),
                                        ("by_parts", dict(factor=4.0, ctx=32768, fast=24.0, slow=2.0)),
                                        ("smooth", dict(factor=8.0, ctx=8192, fast=4.0, slow=1.0)),
                                        ("smooth", dict(factor=1.0, ctx=8192, fast=4.0, slow=1.0))])
@pytest.mark.parametrize("rot", [16, 64, 96, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies(lib, kind, extra, rot, base):
    from sparse_kv_cache_snapkv_gb300 import rkv
    f, m = rkv.rkv_rope_frequencies(rot, base, kind, **extra)
    want, wm = S.frequencies(kind, rot, base, **extra)
    # double arithmetic on both sides, rounded to fp32 once; a ramp's quotient cancels a few digits
    np.testing.assert_allclose(f.numpy().astype(np.float64), want, rtol=2.0 ** -24 + 1e-11)
    assert f.shape == (rot // 2,) and abs(m - wm) <= 2.0 ** -23 * wm


def test_frequency_refusals(lib):
    from sparse_kv_cache_snapkv_gb300 import rkv
    good = dict(rot_dim=64, base=10000.0, kind="by_parts", factor=2.0, ctx=1000, fast=32.0, slow=1.0)
    rkv.rkv_rope_frequencies(**good)
    for change in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=130), dict(base=1.0), dict(base=float("nan")),
                   dict(factor=0.5), dict(factor=float("inf")), dict(ctx=0), dict(slow=0.0), dict(fast=1.0),
                   dict(kind="base", rot_dim=2)):
        with pytest.raises(rkv.RkvError):
            rkv.rkv_rope_frequencies(**{**good, **change})
    with pytest.raises(ValueError):
        rkv.rkv_rope_frequencies(kind="other")


def test_binding_refuses_host_and_odd_tensors(lib):
    import torch
    from sparse_kv_cache_snapkv_gb300 import rkv
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    kv = torch.zeros(1, 2, 16, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    calls = [lambda: rkv.rkv_prompt_attention(q, i[:2], kv, kv, i[:1], 0.1, torch.zeros_like(q)),
             lambda: rkv.rkv_prompt_attention(q.float(), i[:2], kv, kv, i[:1], 0.1, q),
             lambda: rkv.rkv_prompt_attention(q[:, :, :64], i[:2], kv, kv, i[:1], 0.1, q),
             lambda: rkv.rkv_prompt_attention(q[:, ::2], i[:2], kv, kv, i[:1], 0.1, q),
             lambda: rkv.rkv_prompt_attention(q[0], i[:2], kv, kv, i[:1], 0.1, q),
             lambda: rkv.rkv_prompt_attention(None, i[:2], kv, kv, i[:1], 0.1, q),
             lambda: rkv.rkv_prompt_attention_paged(q, i[:2], kv, kv, None, i[:1], 0.1, torch.zeros_like(q)),
             lambda: rkv.rkv_tree_attention(q, i[:2], None, kv, kv, i[:1], 0.1, torch.zeros_like(q)),
             lambda: rkv.rkv_rope_append(q, kv[0], kv[0], i, torch.zeros(64), i, q, kv, kv),
             lambda: rkv.rkv_reserve_slots(i, i, i, i.view(2, 2), i, i[:1], 16, i, i, i, i, i, i[:1])]
    for call in calls:
        with pytest.raises((ValueError, TypeError)):
            call()
