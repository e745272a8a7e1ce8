"""The cache oracle against worked values, and the refusals of the cache calls. No GPU needed."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache as C

FAKE = ctypes.c_void_p(1 << 20)   # aligned, non-null, never dereferenced: calls fail validation
ODD = ctypes.c_void_p((1 << 20) + 8)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from sparse_kv_cache_snapkv_gb300 import _build, rkv
    _build.build()
    return rkv.load()


# ------------------------------------------------------------------------------- the format
def test_scale_numbers_are_fp16_prefixes():
    b = np.arange(C.MAX_SCALE_BYTE + 1)
    half = (b << 7).astype(np.uint16).view(np.float16).astype(np.float64)
    assert np.array_equal(C.scale_number(b), half)
    assert half[-1] == 10240.0 and half[1] == 2.0 ** -17


def test_quantise_worked_block():
    x = np.zeros(128)
    x[:16] = [6, -6, 5, 5.01, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.2501, -0.75, 0, 0.1, -0.1, 4]
    codes, sb = C.kv4_quantise(x)
    assert sb[0] == 15 << 3  # 6 / 6 = 1
    want = [6, -6, 4, 6, 4, 2, 2, 1, 1, 0, 0.5, -1, 0, 0, 0, 4]  # ties to the even code
    assert C.kv4_values(codes, sb)[:16].tolist() == want
    assert codes[7] == 0x68   # low half: dimension 14 = -0.1 -> -0; high half: dimension 15 = 4
    assert not codes[8:].any() and not sb[1:].any()


def test_quantise_edges():
    x = np.zeros((6, 128))
    x[0, :16] = np.nan
    x[0, 0] = 3.0
    x[1, 0], x[1, 1] = np.inf, -np.inf
    x[2, 0] = 6 * 2.0 ** -18       # a tie between scale 0 and the smallest, 2^-17: even, 0
    x[3, 0] = 6 * 2.0 ** -18 * 1.01
    x[4, 0] = 6 * (1 + 1 / 16)     # tie between mantissas 0 and 1: even
    x[5, 0] = 6 * (1 + 3 / 16)     # tie between 1 and 2: even
    codes, sb = C.kv4_quantise(x)
    v = C.kv4_values(codes, sb)
    assert v[0, 0] == 3.0 and not v[0, 1:].any()
    assert v[1, 0] == 61440.0 and v[1, 1] == -61440.0
    assert sb[2, 0] == 0 and not v[2].any()
    assert sb[3, 0] == 1 and v[3, 0] == 3 * 2.0 ** -17  # 3.03 scales
    assert sb[4, 0] == 120 and sb[5, 0] == 122


def test_quantise_is_a_nearest_point():
    """Every value is at most half a step from what it becomes, or clipped at 6 scales."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((200, 128)) * np.exp(3 * rng.standard_normal((200, 1))))
    x = torch.tensor(x).bfloat16().double().numpy()
    codes, sb = C.kv4_quantise(x)
    v = C.kv4_values(codes, sb)
    s = np.repeat(C.scale_number(sb), 16, -1)
    a = np.abs(x)
    step = np.where(a < 2 * s, 0.5, np.where(a < 4 * s, 1.0, 2.0)) * s
    over = np.maximum(a - 6 * s, 0.0)
    assert (np.abs(v - x) <= step / 2 + over).all()
    # exact in bf16 and fp16
    assert np.array_equal(torch.tensor(v).bfloat16().double().numpy(), v)
    assert np.array_equal(torch.tensor(v).half().double().numpy(), v)


def test_weights_sum_to_the_queries():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((4, 9, 128)), rng.standard_normal((30, 128))
    w = C.prompt_weights(q, k, 0.1)
    assert w.shape == (30,) and abs(w.sum() - 36) < 1e-9
    # the last key is seen by one query of each head, the first 21 by all
    one = C.softmax_weights(q[:, -1], k, 0.1)[:, -1].sum()
    assert abs(w[-1] - one) < 1e-12


def test_evict_worked():
    w = np.array([5, 1, 4, 9, 2, 3, 0.5, 0.1])
    pos = np.array([10, 3, 11, 0, -1, -1, -1, -1])
    src, at = C.evict(w, pos, seen=16, keep=5, recent=2)   # rows 6, 7 are the last two
    assert sorted(src.tolist()) == [0, 2, 3, 6, 7]
    assert src.tolist() == [0, 6, 2, 3, 7] and at.tolist() == [10, 14, 11, 0, 15]
    src, at = C.evict(w, pos, seen=16, keep=8, recent=2)
    assert src.tolist() == list(range(8)) and at.tolist() == pos.tolist()
    src, _ = C.evict(np.ones(6), np.full(6, -1), 6, 3, 0)  # ties: lower rows
    assert src.tolist() == [0, 1, 2]


# ------------------------------------------------------------------------------- refusals
def test_append_refusals(lib):
    v = FAKE
    ok = dict(new_k=v, new_v=v, new_len=None, n=1, n_kv=2, head_dim=128, max_new=4, kc=v, ks=v,
              vc=v, vs=v, cap=16, len=v, len_out=v, kval=None, vval=None, ws=v, ws_bytes=BIG,
              stream=None)
    bad = [(dict(head_dim=64), 2), (dict(new_k=None), 1), (dict(new_v=ODD), 1), (dict(kc=None), 1),
           (dict(vs=ODD), 1), (dict(len=None), 1), (dict(len_out=None), 1), (dict(kval=v), 1),
           (dict(kval=v, vval=ODD), 1), (dict(n=0), 1), (dict(n_kv=-1), 1), (dict(max_new=0), 1),
           (dict(cap=0), 1), (dict(cap=(1 << 30) + 1), 1), (dict(n=1 << 20, n_kv=1 << 20), 1),
           (dict(ws=None), 3), (dict(ws=ODD), 3), (dict(ws_bytes=255), 3)]
    for change, code in bad:
        assert lib.rkv_kv4_append(*{**ok, **change}.values()) == code, change


def test_append_paged_refusals(lib):
    v = FAKE
    ok = dict(new_k=v, new_v=v, new_len=None, n=1, n_kv=2, head_dim=128, max_new=4, kc=v, ks=v,
              vc=v, vs=v, num_blocks=4, block=16, table=v, max_blocks=2, len=v, len_out=v,
              kval=None, vval=None, ws=v, ws_bytes=BIG, stream=None)
    for change in (dict(block=8), dict(block=24), dict(table=None), dict(max_blocks=0),
                   dict(num_blocks=0), dict(block=65536, max_blocks=1 << 15)):
        assert lib.rkv_kv4_append_paged(*{**ok, **change}.values()) == 1, change
    assert lib.rkv_kv4_append_paged(*{**ok, "ws_bytes": 8}.values()) == 3


DECODE = dict(q=FAKE, new_k=None, new_v=None, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, len=FAKE,
              len_out=None, n=1, n_kv=2, gqa=4, head_dim=128, cap=64, scale=0.1, out=FAKE,
              weights=None, ws=FAKE, ws_bytes=BIG, stream=None)


def test_decode_refusals(lib):
    v = FAKE
    bad = [(dict(head_dim=256), 2), (dict(gqa=3), 2), (dict(gqa=16), 2), (dict(q=None), 1),
           (dict(q=ODD), 1), (dict(out=ODD), 1), (dict(ks=None), 1), (dict(new_k=v), 1),
           (dict(new_k=v, new_v=v), 1), (dict(len_out=v), 1),
           (dict(new_k=ODD, new_v=v, len_out=v), 1), (dict(weights=ODD), 1), (dict(n=0), 1),
           (dict(cap=0), 1), (dict(cap=(1 << 30) + 1), 1), (dict(scale=0.0), 1),
           (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(scale=-1.0), 1),
           (dict(scale=3e38), 1), (dict(n=1 << 16, n_kv=1 << 14, gqa=8), 1), (dict(ws=None), 3),
           (dict(ws_bytes=256), 3)]
    for change, code in bad:
        assert lib.rkv_kv4_decode(*{**DECODE, **change}.values()) == code, change
    # weights take room for the logits
    need = lib.rkv_kv4_decode_workspace_bytes(1, 2, 4, 64, 0)
    assert lib.rkv_kv4_decode_workspace_bytes(1, 2, 4, 64, 1) >= need + 2 * 4 * 64 * 4
    assert lib.rkv_kv4_decode(*{**DECODE, "weights": v, "ws_bytes": need}.values()) == 3


def test_decode_paged_refusals(lib):
    v = FAKE
    ok = dict(q=v, new_k=None, new_v=None, kc=v, ks=v, vc=v, vs=v, table=v, len=v, len_out=None, n=1,
              n_kv=2, gqa=4, head_dim=128, num_blocks=4, block=16, max_blocks=2, scale=0.1, out=v,
              weights=None, ws=v, ws_bytes=BIG, stream=None)
    for change, code in ((dict(block=4), 1), (dict(table=None), 1), (dict(gqa=5), 2),
                         (dict(ws_bytes=1), 3)):
        assert lib.rkv_kv4_decode_paged(*{**ok, **change}.values()) == code, change


def test_dense_weights_refusals(lib):
    v = FAKE
    ok = dict(q=v, k=v, v=v, len=v, n=1, n_kv=2, gqa=4, head_dim=128, max_len=64, scale=0.1, out=v,
              weights=v, ws=v, ws_bytes=BIG, stream=None)
    for change, code in ((dict(head_dim=64), 2), (dict(gqa=6), 2), (dict(weights=None), 1),
                         (dict(k=ODD), 1), (dict(v=None), 1), (dict(max_len=0), 1),
                         (dict(scale=0.0), 1), (dict(ws_bytes=300), 3)):
        assert lib.rkv_dense_decode_weights(*{**ok, **change}.values()) == code, change


def test_prompt_refusals(lib):
    v = FAKE
    ok = dict(q=v, q_len=v, k=v, len=v, n=1, n_kv=2, gqa=4, head_dim=128, max_q=64, max_len=128,
              scale=0.1, weights=v, ws=v, ws_bytes=BIG, stream=None)
    for change, code in ((dict(head_dim=64), 2), (dict(gqa=65), 2), (dict(gqa=0), 1),
                         (dict(q=ODD), 1), (dict(k=None), 1), (dict(q_len=None), 1),
                         (dict(weights=None), 1), (dict(max_q=0), 1), (dict(max_q=129), 1),
                         (dict(scale=-0.1), 1), (dict(ws_bytes=300), 3),
                         (dict(n=1 << 15, max_len=1 << 20), 6),
                         (dict(n=1 << 12, max_q=1 << 18, max_len=1 << 18), 6)):
        assert lib.rkv_prompt_weights(*{**ok, **change}.values()) == code, change


def test_evict_refusals(lib):
    v = FAKE
    ok = dict(k=v, v=v, len=v, len_out=v, w=v, wo=v, pos=v, pos_out=v, seen=v, n=1, n_kv=2,
              head_dim=128, cap=64, keep=32, recent=4, src=None, ws=v, ws_bytes=BIG, stream=None)
    for change, code in ((dict(head_dim=64), 2), (dict(k=None), 1), (dict(v=ODD), 1),
                         (dict(w=None), 1), (dict(pos_out=None), 1), (dict(seen=None), 1),
                         (dict(keep=0), 1), (dict(recent=33), 1), (dict(recent=-1), 1),
                         (dict(cap=0), 1), (dict(n=0), 1), (dict(ws_bytes=300), 3),
                         (dict(ws=None), 3)):
        assert lib.rkv_evict(*{**ok, **change}.values()) == code, change


def test_binding_refuses_host_tensors_and_wrong_shapes():
    from sparse_kv_cache_snapkv_gb300 import rkv
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    cache = rkv.kv4_cache(2, 2, 32, device="cpu")
    assert [tuple(t.shape) for t in cache] == [(2, 2, 32, 64), (2, 2, 32, 8)] * 2
    with pytest.raises(ValueError):
        rkv.rkv_kv4_decode(bf(2, 8, 128), *cache, i32(2), 0.1, bf(2, 8, 128))
    with pytest.raises(ValueError):  # query heads over KV heads
        rkv.rkv_kv4_decode(bf(2, 7, 128), *cache, i32(2), 0.1, bf(2, 7, 128))
    with pytest.raises(ValueError):  # weights of another capacity
        rkv.rkv_kv4_decode(bf(2, 8, 128), *cache, i32(2), 0.1, bf(2, 8, 128),
                           weights=torch.zeros(2, 2, 33))
    with pytest.raises(TypeError):
        rkv.rkv_kv4_decode(bf(2, 8, 128).half(), *cache, i32(2), 0.1, bf(2, 8, 128))
    with pytest.raises(ValueError):  # another number of KV heads
        rkv.rkv_kv4_append(bf(2, 3, 4, 128), bf(2, 3, 4, 128), *cache, i32(2), i32(2))
    with pytest.raises(ValueError):  # another number of units
        rkv.rkv_kv4_append(bf(1, 2, 4, 128), bf(1, 2, 4, 128), *cache, i32(1), i32(1))
    with pytest.raises(ValueError):  # values of another shape
        rkv.rkv_kv4_append(bf(2, 2, 4, 128), bf(2, 2, 4, 128), *cache, i32(2), i32(2),
                           k_values=bf(2, 2, 5, 128), v_values=bf(2, 2, 5, 128))
    with pytest.raises(ValueError):  # fewer query rows than told
        rkv.rkv_prompt_weights(bf(2, 8, 4, 64), i32(2), bf(2, 2, 16, 128), i32(2), 0.1,
                               torch.zeros(2, 2, 16))
    with pytest.raises(ValueError):
        rkv.rkv_evict(bf(2, 2, 16, 128), bf(2, 2, 16, 128), i32(2), torch.zeros(2, 2, 16),
                      i32(2, 2, 15), i32(2), 8, 2, i32(2), torch.zeros(2, 2, 16), i32(2, 2, 16))
