"""The cache calls where their work is laid out another way: as many parts as there are CTAs, more units than
a launch's threads count one by one, more items than SMs, and large offsets. Against the float64 oracle;
decodes with a tolerance for each query head."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as C
from tests import cache_parity as P
from tests import cache_parity_heads as H

pytestmark = pytest.mark.gpu

D = 128
SCALE = 1.0 / math.sqrt(D)
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def rkv():
    from sparse_kv_cache_snapkv_gb300 import rkv
    rkv.load()
    return rkv


def _ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _rand(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)


def _f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def _held(cache, u, g, t):
    """The numbers that a 4-bit cache's first t rows stand for."""
    return [C.kv4_values(cache[i][u, g, :t].cpu().numpy(), cache[i + 1][u, g, :t].cpu().numpy()) for i in (0, 2)]


def _decode(rkv, kv4, n, n_kv, gqa, cap, lens, units, seed=1, **kw):
    """One decode with weights; the units named are checked."""
    k, v = _rand(seed, n, n_kv, cap, D), _rand(seed + 1, n, n_kv, cap, D)
    q = _rand(seed + 2, n, n_kv * gqa, D)
    out, w = torch.full_like(q, float("nan")), torch.zeros(n, n_kv, cap, device="cuda")
    ln = _ints(lens)
    if kv4:
        cache = rkv.kv4_cache(n, n_kv, cap)
        rkv.rkv_check_status(rkv.rkv_kv4_append(k, v, *cache, _ints([0] * n), torch.empty_like(ln), new_len=ln))
        rkv.rkv_check_status(rkv.rkv_kv4_decode(q, *cache, ln, SCALE, out, weights=w, **kw))
    else:
        rkv.rkv_check_status(rkv.rkv_dense_decode_weights(q, k, v, ln, SCALE, out, w, **kw))
    for u in units:
        t = lens[u]
        for g in range(n_kv):
            heads = slice(g * gqa, (g + 1) * gqa)
            assert not w[u, g, t:].any()
            if t == 0:
                assert not out[u, heads].any()
                continue
            hk, hv = _held(cache, u, g, t) if kv4 else (_f64(k[u, g, :t]), _f64(v[u, g, :t]))
            H.check_decode(_f64(out[u, heads]), _f64(w[u, g, :t]), _f64(q[u, heads]), hk, hv, SCALE, kv4,
                           64 + t // 64, f"unit {u} head {g}")
    assert torch.isfinite(out).all() and torch.isfinite(w).all()


# ------------------------------------------------------------------------------- decodes
@pytest.mark.parametrize("kv4", [True, False])
@pytest.mark.parametrize("gqa", [1, 8])
def test_decode_in_as_many_parts_as_ctas(rkv, kv4, gqa):
    """One (unit, head) over every CTA of the launch: the joins' table of factors at its fullest."""
    _decode(rkv, kv4, 1, 1, gqa, 131071, [131071], [0])


@pytest.mark.parametrize("kv4", [True, False])
@pytest.mark.parametrize("n,n_kv,gqa,cap", [(33, 3, 2, 300), (257, 1, 4, 200), (1100, 2, 1, 40)])
def test_decode_of_many_units(rkv, kv4, n, n_kv, gqa, cap):
    """More units than a warp, or the threads of a CTA, have one each of; many without tokens."""
    lens = [0 if u % 5 == 3 else (u * 37) % (cap + 1) for u in range(n)]
    lens[0], lens[-1] = 0, cap
    _decode(rkv, kv4, n, n_kv, gqa, cap, lens, sorted({0, 1, 31, 32, n // 2, n - 2, n - 1}))


# ------------------------------------------------------------------------------- prompt
@pytest.mark.parametrize("n,n_kv,gqa,max_q,cap", [
    (20, 2, 2, 1024, 1100),   # a tile holds rows of one head: 320 tiles in pass 1, 200 in pass 2
    (180, 2, 1, 300, 520),    # 720 and 1080
    (200, 2, 5, 37, 300),     # a tile runs on through the heads: 400 and 800
])
def test_prompt_of_more_items_than_sms(rkv, n, n_kv, gqa, max_q, cap):
    """CTAs that go on from item to item, in waves from either end, over units without queries, without
    keys, and of any length between."""
    lens = [0 if u % 11 == 5 else cap - (u * 29) % (cap // 2) for u in range(n)]
    news = [0 if u % 7 == 3 else min(lens[u], max_q - (u * 13) % (max_q // 2 + 1)) for u in range(n)]
    lens[0], news[0] = cap, max_q
    k, q = _rand(11, n, n_kv, cap, D), _rand(12, n, n_kv * gqa, max_q, D)
    for u in range(n):
        k[u, :, lens[u]:] = float("nan")
        q[u, :, news[u]:] = float("inf")
    w0 = torch.rand(n, n_kv, cap, device="cuda")
    w1 = w0.clone()
    rkv.rkv_check_status(rkv.rkv_prompt_weights(q, _ints(news), k, _ints(lens), SCALE, w1))
    for u in range(n):
        for g in range(n_kv):
            T, L = news[u], lens[u]
            if T == 0:
                assert torch.equal(w1[u, g], w0[u, g]), u
                continue
            assert torch.equal(w1[u, g, L:], w0[u, g, L:])
            if u % max(1, n // 12) and u != n - 1:
                # every unit's weights add up to its queries: a weight w of a key is within
                # (e_p + terms u) w + 2 u (w + before) of the true one, e_p < 1e-3 for these logits
                added = (w1[u, g, :L].double() - w0[u, g, :L].double()).sum().item()
                assert abs(added - gqa * T) <= 2e-3 * gqa * T + 2.0 ** -22 * L, (u, g)
                continue
            hk, hq = _f64(k[u, g, :L]), _f64(q[u, g * gqa:(g + 1) * gqa, :T])
            P.check_weights(_f64(w1[u, g, :L]), C.prompt_weights(hq, hk, SCALE), _f64(w0[u, g, :L]),
                            hq.reshape(-1, D), hk, SCALE, 96 + L // 16 + gqa * T // 64, f"unit {u} head {g}")


# ------------------------------------------------------------------------------- eviction
def _evict_check(rkv, kv4, n, n_kv, cap, lens, keep, recent, w, pos, alias, units, seed=21):
    """alias: which of (weights, pos, lengths) are written over their inputs."""
    seen = [t + 50 for t in lens]
    if kv4:  # each row its own number, in the scale bytes of K
        rows = [torch.zeros(n, n_kv, cap, x, dtype=torch.uint8, device="cuda") for x in (64, 8, 64, 8)]
        number = torch.arange(n * n_kv * cap, device="cuda").view(n, n_kv, cap, 1)
        for x in rows:
            x.copy_((number >> (8 * (torch.arange(x.shape[-1], device="cuda") % 5))) & 0xff)
    else:
        rows = [torch.randint(0, 1 << 15, (n, n_kv, cap, D), dtype=torch.int16, device="cuda").view(BF) for _ in range(2)]
    was = [x.clone() for x in rows]
    length, win, pin = _ints(lens), w.clone(), pos.clone()
    wo = win if alias[0] else torch.full_like(w, 5.0)
    po = pin if alias[1] else torch.full_like(pos, 9)
    lo = length if alias[2] else torch.zeros_like(length)
    wo0, po0 = wo.clone(), po.clone()
    src = torch.full((n, n_kv, keep), -9, dtype=I32, device="cuda")
    call = rkv.rkv_evict_kv4 if kv4 else rkv.rkv_evict
    rkv.rkv_check_status(call(*rows, length, win, pin, _ints(seen), keep, recent, lo, wo, po, src_rows=src))
    assert lo.tolist() == [min(t, keep) for t in lens]
    for u in units:
        t, m = lens[u], min(lens[u], keep)
        for g in range(n_kv):
            want, at = C.evict(_f64(w[u, g, :t]), pos[u, g, :t].cpu().numpy(), seen[u], keep, recent)
            what = f"unit {u} head {g}"
            assert np.array_equal(src[u, g, :m].cpu().numpy(), want), what
            assert (src[u, g, m:] == -1).all(), what
            ix = torch.tensor(want, device="cuda", dtype=torch.long)
            assert torch.equal(wo[u, g, :m], w[u, g, ix]), what
            assert np.array_equal(po[u, g, :m].cpu().numpy(), at), what
            assert (wo[u, g, m:t] == 0).all() and (po[u, g, m:t] == -1).all(), what
            assert torch.equal(wo[u, g, t:], wo0[u, g, t:]) and torch.equal(po[u, g, t:], po0[u, g, t:]), what
            for now, old in zip(rows, was):
                assert torch.equal(now[u, g, :m].view(torch.uint8), old[u, g, ix].view(torch.uint8)), what
                assert torch.equal(now[u, g, m:].view(torch.uint8), old[u, g, m:].view(torch.uint8)), what


@pytest.mark.parametrize("kv4", [True, False])
@pytest.mark.parametrize("cap,keep,weights", [
    (8193, 4096, "past"), (8193, 8192, "normal"), (20000, 10000, "past"), (20000, 4096, "ties"),
    (40960, 20480, "past"), (40960, 4096, "normal"), (40960, 33, "ties"),
])
def test_evict_a_unit_for_every_sm_at_prompt_length(rkv, cap, keep, weights, kv4):
    """One CTA for each (unit, head), its keys in shared memory and its weights not. `past`: every kept row
    lies past keep, so as many rows move as there can be."""
    n, n_kv = 80, 2
    g = torch.Generator(device="cuda").manual_seed(cap + keep)
    w = torch.exp(2 * torch.randn(n, n_kv, cap, generator=g, device="cuda"))
    lens = [cap if u % 3 == 0 else cap - 1 - (u * 97) % (cap // 3) for u in range(n)]
    lens[7], lens[8], lens[9] = 0, keep, min(cap, keep + 1)
    if weights == "past":
        w[..., keep:] += w.max() + 1
    if weights == "ties":
        w = torch.randint(0, 3, w.shape, generator=g, device="cuda").float()
    pos = torch.full((n, n_kv, cap), -1, dtype=I32, device="cuda")
    known = torch.rand(n, n_kv, keep + 50, generator=g, device="cuda").argsort(-1)[..., :keep]
    pos[::2, :, :keep] = known[::2].int()
    units = [0, 1, 7, 8, 9, n // 2, n - 1]
    for alias in ((True, True, True), (False, False, False), (True, False, False), (False, True, True)):
        _evict_check(rkv, kv4, n, n_kv, cap, lens, keep, min(keep, 16), w, pos, alias, units if all(alias) else units[:4])


@pytest.mark.parametrize("n,cap,keep", [(3, 9000, 5000), (160, 4000, 2500), (1, 270000, 1000)])
@pytest.mark.parametrize("alias", [(True, False, False), (False, True, True)])
def test_evict_over_some_of_its_inputs(rkv, n, cap, keep, alias):
    """Weights written over their input and positions not, and the other way: clusters, one CTA for each with all
    in shared memory, and more rows than a cluster holds."""
    g = torch.Generator(device="cuda").manual_seed(n)
    w = torch.rand(n, 1, cap, generator=g, device="cuda")
    pos = torch.full((n, 1, cap), -1, dtype=I32, device="cuda")
    pos[..., :keep] = torch.rand(n, 1, keep + 50, generator=g, device="cuda").argsort(-1)[..., :keep].int()
    lens = [max(0, cap - 31 * u) for u in range(n)]
    _evict_check(rkv, True, n, 1, cap, lens, keep, 9, w, pos, alias, sorted({0, n // 2, n - 1}))


# ------------------------------------------------------------------------------- offsets past 32 bits
def test_offsets_past_32_bits(rkv):
    """A bf16 cache of 4.8 GB each for K and V, whose last heads lie past 2^32 bytes; rows that no unit has are
    never written, so the arrays need no filling."""
    n, n_kv, gqa, cap = 2, 8, 2, (9 << 17) + 37
    lens = [5, 3000]
    k, v = (torch.empty(n, n_kv, cap, D, dtype=BF, device="cuda") for _ in range(2))
    for u, t in enumerate(lens):
        k[u, :, :t], v[u, :, :t] = _rand(31 + u, n_kv, t, D), _rand(33 + u, n_kv, t, D)
    assert (n * n_kv - 1) * cap * D * 2 > 2**32
    q, ln = _rand(35, n, n_kv * gqa, D), _ints(lens)
    out, w = torch.empty_like(q), torch.zeros(n, n_kv, cap, device="cuda")
    rkv.rkv_check_status(rkv.rkv_dense_decode_weights(q, k, v, ln, SCALE, out, w))
    for u, g in ((0, 0), (1, 7)):
        heads, t = slice(g * gqa, (g + 1) * gqa), lens[u]
        H.check_decode(_f64(out[u, heads]), _f64(w[u, g, :t]), _f64(q[u, heads]), _f64(k[u, g, :t]), _f64(v[u, g, :t]),
                       SCALE, False, 64 + t // 64, f"unit {u}")
    before = w.clone()
    qp = _rand(36, n, n_kv * gqa, 300, D)
    rkv.rkv_check_status(rkv.rkv_prompt_weights(qp, _ints([5, 300]), k, ln, SCALE, w))
    hk, hq = _f64(k[1, 7, :3000]), _f64(qp[1, 14:16])
    P.check_weights(_f64(w[1, 7, :3000]), C.prompt_weights(hq, hk, SCALE), _f64(before[1, 7, :3000]), hq.reshape(-1, D),
                    hk, SCALE, 96 + 3000 // 16 + 10)
    kk, vv, w_was = k[1, 7, :3000].clone(), v[1, 7, :3000].clone(), w.clone()
    pos = torch.full((n, n_kv, cap), -1, dtype=I32, device="cuda")
    rkv.rkv_check_status(rkv.rkv_evict(k, v, ln, w, pos, ln.clone(), 1000, 64, ln, w, pos))
    assert ln.tolist() == [5, 1000]
    src, at = C.evict(_f64(w_was[1, 7, :3000]), np.full(3000, -1), 3000, 1000, 64)
    ix = torch.tensor(src, device="cuda")
    assert torch.equal(k[1, 7, :1000], kk[ix]) and torch.equal(v[1, 7, :1000], vv[ix])
    assert np.array_equal(pos[1, 7, :1000].cpu().numpy(), at)
