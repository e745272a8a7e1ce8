"""The 4-bit cache, the weight-accumulating decodes and prompt, and the eviction, against the
float64 oracle (tolerances: tests/cache_parity.py). Codes, scales, rows and positions are exact."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as C
from tests import cache_parity as P

pytestmark = pytest.mark.gpu

D = 128
SCALE = 1.0 / math.sqrt(D)
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def rkv():
    from sparse_kv_cache_snapkv_gb300 import rkv
    rkv.load()
    return rkv


def _f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def _np(t):
    return t.detach().cpu().numpy()


def _ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def _normal(seed, *shape, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    return (x * torch.exp(spread * torch.randn(*shape[:-2], 1, D, generator=g, device="cuda"))).to(BF)


def _filled_cache(rkv, n, n_kv, cap, seed):
    """Every byte set (as by earlier sequences): rows past a length must not matter."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randint(0, 256, t.shape, generator=g, device="cuda").to(torch.uint8)
            for t in rkv.kv4_cache(n, n_kv, cap)]


def _to_pool(t, table, block):
    """[n][n_kv][cap][w] -> pool with the blocks placed by the table (cap = max_blocks * block)."""
    n, n_kv, cap, w = t.shape
    pool = torch.full((int(table.max()) + 3, n_kv, block, w), 0xEE, dtype=t.dtype, device="cuda")
    pool[table.flatten().long()] = t.view(n, n_kv, cap // block, block, w).transpose(1, 2).flatten(0, 1)
    return pool


def _from_pool(pool, table):
    return pool[table.long()].transpose(1, 2).flatten(2, 3)


# ------------------------------------------------------------------------------- append
@pytest.mark.parametrize("n,n_kv,cap,max_new,lens,news", [
    (1, 1, 1, 1, [0], None),
    (3, 2, 40, 7, [0, 33, 5], [7, 7, 0]),
    (2, 3, 300, 129, [100, 171], [129, 3]),
    (5, 8, 64, 1, [0, 1, 31, 62, 63], None),
])
def test_append(rkv, n, n_kv, cap, max_new, lens, news):
    new_k, new_v = _normal(1, n, n_kv, max_new, D, spread=3.0), _normal(2, n, n_kv, max_new, D)
    cache = _filled_cache(rkv, n, n_kv, cap, 3)
    before = [t.clone() for t in cache]
    length, out = _ints(lens), torch.full((n,), -7, dtype=I32, device="cuda")
    kv, vv = torch.full_like(new_k, 77.0), torch.full_like(new_v, 77.0)
    ws = rkv.rkv_kv4_append(new_k, new_v, *cache, length, out,
                            new_len=None if news is None else _ints(news), k_values=kv, v_values=vv)
    rkv.rkv_check_status(ws)
    news = news or [max_new] * n
    assert out.tolist() == [a + b for a, b in zip(lens, news)] and length.tolist() == lens
    for x, vals, codes, scales, b0, b1 in ((new_k, kv, cache[0], cache[1], before[0], before[1]),
                                           (new_v, vv, cache[2], cache[3], before[2], before[3])):
        wc, wsb = C.kv4_quantise(_f64(x))
        for u in range(n):
            a, t = lens[u], news[u]
            assert np.array_equal(_np(codes[u, :, a:a + t]), wc[u, :, :t])
            assert np.array_equal(_np(scales[u, :, a:a + t]), wsb[u, :, :t])
            assert np.array_equal(_f64(vals[u, :, :t]), C.kv4_values(wc[u, :, :t], wsb[u, :, :t]))
            assert (vals[u, :, t:] == 77.0).all()
            for now, was in ((codes, b0), (scales, b1)):
                assert torch.equal(now[u, :, :a], was[u, :, :a])
                assert torch.equal(now[u, :, a + t:], was[u, :, a + t:])


def test_append_special_values(rkv):
    """Every bf16 number once, in blocks of neighbours and in blocks of everything."""
    bits = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16)
    x = bits.view(BF).view(1, 1, 512, D)
    mixed = x.flatten()[torch.randperm(65536, generator=torch.Generator().manual_seed(4)).cuda()]
    y = mixed.view(1, 1, 512, D).contiguous()
    cache = rkv.kv4_cache(1, 1, 512)
    out = _ints([0])
    rkv.rkv_check_status(rkv.rkv_kv4_append(x.contiguous(), y, *cache, _ints([0]), out))
    for src, codes, scales in ((x, cache[0], cache[1]), (y, cache[2], cache[3])):
        wc, wsb = C.kv4_quantise(_f64(src))
        assert np.array_equal(_np(scales), wsb)
        assert np.array_equal(_np(codes), wc)


def test_append_in_place_length_and_bad_units(rkv):
    n, n_kv, cap, t = 5, 2, 32, 4
    new_k, new_v = _normal(5, n, n_kv, t, D), _normal(6, n, n_kv, t, D)
    cache = _filled_cache(rkv, n, n_kv, cap, 7)
    before = [x.clone() for x in cache]
    # full by one, negative length, too many new, negative new, fine
    length, news = _ints([29, -1, 3, 3, 28]), _ints([4, 4, 5, -1, 4])
    ws = rkv.rkv_kv4_append(new_k, new_v, *cache, length, length, new_len=news)
    with pytest.raises(rkv.RkvError) as e:
        rkv.rkv_check_status(ws)
    assert e.value.bits == 0x1
    assert length.tolist() == [29, -1, 3, 3, 32]
    for now, was in zip(cache, before):
        assert torch.equal(now[:4], was[:4]) and torch.equal(now[4, :, :28], was[4, :, :28])
    assert not torch.equal(cache[0][4], before[0][4])


@pytest.mark.parametrize("block", [16, 64])
def test_append_paged_is_the_same(rkv, block):
    n, n_kv, mb, t = 3, 2, 4, 21
    cap = mb * block
    table = torch.randperm(n * mb, generator=torch.Generator().manual_seed(8)).int().view(n, mb).cuda()
    flat = _filled_cache(rkv, n, n_kv, cap, 9)
    pools = [_to_pool(x, table, block) for x in flat]
    new_k, new_v = _normal(10, n, n_kv, t, D), _normal(11, n, n_kv, t, D)
    lens = _ints([0, block - 3, cap - t])
    a, b = torch.zeros_like(lens), torch.zeros_like(lens)
    rkv.rkv_check_status(rkv.rkv_kv4_append(new_k, new_v, *flat, lens, a))
    rkv.rkv_check_status(rkv.rkv_kv4_append_paged(new_k, new_v, *pools, table, lens, b))
    assert torch.equal(a, b)
    for x, pool in zip(flat, pools):
        assert torch.equal(_from_pool(pool, table), x)
        free = torch.ones(pool.shape[0], dtype=torch.bool)
        free[table.flatten().long().cpu()] = False
        assert (pool[free.cuda()] == 0xEE).all()  # no other block


# ------------------------------------------------------------------------------- 4-bit decode
def _kv4_case(rkv, n, n_kv, cap, lens, seed):
    """A cache whose rows below each length hold quantised values, garbage above."""
    cache = _filled_cache(rkv, n, n_kv, cap, seed)
    top = max(1, max(lens))
    zero, out = _ints([0] * n), _ints([0] * n)
    if max(lens):
        rkv.rkv_check_status(rkv.rkv_kv4_append(
            _normal(seed + 1, n, n_kv, top, D), _normal(seed + 2, n, n_kv, top, D), *cache, zero,
            out, new_len=_ints(lens)))
    return cache


def _check_decode(cache, lens, q, out, w0, w1, new=None, tag=""):
    """Outputs and weights of every unit against the oracle over the numbers the cache holds."""
    n, n_kv = cache[0].shape[:2]
    gqa = q.shape[1] // n_kv
    hq = _f64(q).reshape(n, n_kv, gqa, D)
    ho = _f64(out).reshape(n, n_kv, gqa, D)
    held = [_np(x) for x in cache]
    for u in range(n):
        for g in range(n_kv):
            t = lens[u]
            k = C.kv4_values(held[0][u, g, :t], held[1][u, g, :t])
            v = C.kv4_values(held[2][u, g, :t], held[3][u, g, :t])
            what = f"{tag} unit {u} head {g}"
            if t == 0:
                assert not ho[u, g].any(), what
            else:
                P.check_output(ho[u, g], hq[u, g], k, v, SCALE, True, 64 + t // 64, what)
            if w0 is not None:
                added = C.softmax_weights(hq[u, g], k, SCALE).sum(0)
                P.check_weights(_f64(w1[u, g, :t]), added, _f64(w0[u, g, :t]), hq[u, g], k, SCALE,
                                64 + t // 64, what + " weights")
                assert torch.equal(w1[u, g, t:], w0[u, g, t:]), what


@pytest.mark.parametrize("gqa", [1, 2, 4, 8])
@pytest.mark.parametrize("lens,cap", [([1], 1), ([0, 1, 2, 15], 16), ([16, 17, 127, 128], 129),
                                      ([1021, 300, 0], 1024), ([2500], 2500)])
def test_kv4_decode(rkv, gqa, lens, cap):
    n, n_kv = len(lens), 2
    cache = _kv4_case(rkv, n, n_kv, cap, lens, 20)
    q = _normal(30, 1, n, n_kv * gqa, D, spread=0.3)[0]
    for weights in (False, True):
        out = torch.full_like(q, float("nan"))
        w0 = torch.rand(n, n_kv, cap, device="cuda") if weights else None
        w1 = w0.clone() if weights else None
        rkv.rkv_check_status(rkv.rkv_kv4_decode(q, *cache, _ints(lens), SCALE, out, weights=w1))
        _check_decode(cache, lens, q, out, w0, w1)


@pytest.mark.parametrize("gqa,n,n_kv", [(4, 2, 2), (8, 1, 1), (1, 40, 8)])
@pytest.mark.parametrize("in_place", [False, True])
def test_kv4_decode_appends(rkv, gqa, n, n_kv, in_place):
    cap = 384
    lens = [(37 * u) % cap for u in range(n)]
    lens[0] = 255
    cache = _kv4_case(rkv, n, n_kv, cap, lens, 40)
    before = [x.clone() for x in cache]
    q = _normal(50, 1, n, n_kv * gqa, D)[0]
    nk, nv = _normal(51, n, n_kv, 1, D)[:, :, 0], _normal(52, n, n_kv, 1, D)[:, :, 0]
    nk, nv = nk.contiguous(), nv.contiguous()
    length = _ints(lens)
    out_len = length if in_place else torch.zeros_like(length)
    out, w0 = torch.empty_like(q), torch.zeros(n, n_kv, cap, device="cuda")
    w1 = w0.clone()
    ws = rkv.rkv_kv4_decode(q, *cache, length, SCALE, out, new_k=nk, new_v=nv, length_out=out_len,
                            weights=w1)
    rkv.rkv_check_status(ws)
    assert out_len.tolist() == [t + 1 for t in lens]
    for codes, scales, x in ((cache[0], cache[1], nk), (cache[2], cache[3], nv)):
        wc, wsb = C.kv4_quantise(_f64(x))
        for u, t in enumerate(lens):
            assert np.array_equal(_np(codes[u, :, t]), wc[u]) and np.array_equal(_np(scales[u, :, t]), wsb[u])
    for now, was in zip(cache, before):
        for u, t in enumerate(lens):
            assert torch.equal(now[u, :, :t], was[u, :, :t])
            assert torch.equal(now[u, :, t + 1:], was[u, :, t + 1:])
    _check_decode(cache, [t + 1 for t in lens], q, out, w0, w1)


@pytest.mark.parametrize("in_place", [False, True])
def test_kv4_decode_full_and_bad_lengths(rkv, in_place):
    n, n_kv, gqa, cap = 4, 2, 4, 200
    lens = [200, 260, -3, 10]
    held = [200, 200, 0, 11]
    cache = _kv4_case(rkv, n, n_kv, cap, [200, 200, 200, 200], 60)
    before = [x.clone() for x in cache]
    q = _normal(61, 1, n, n_kv * gqa, D)[0]
    nk = _normal(62, n, n_kv, 1, D)[:, :, 0].contiguous()
    length = _ints(lens)
    out_len = length if in_place else torch.zeros_like(length)
    out, w = torch.empty_like(q), torch.zeros(n, n_kv, cap, device="cuda")
    ws = rkv.rkv_kv4_decode(q, *cache, length, SCALE, out, new_k=nk, new_v=nk, length_out=out_len,
                            weights=w)
    with pytest.raises(rkv.RkvError) as e:
        rkv.rkv_check_status(ws)
    assert e.value.bits == 0x1
    assert out_len.tolist() == [200, 260, -3, 11]
    assert torch.equal(cache[0][:3], before[0][:3])
    _check_decode(cache, held, q, out, torch.zeros_like(w), w)


@pytest.mark.parametrize("block,gqa", [(16, 4), (64, 8), (256, 1)])
def test_kv4_decode_paged_is_the_same(rkv, block, gqa):
    n, n_kv, mb = 4, 2, 5
    cap = mb * block
    lens = [0, 1, cap - 1, block + 3]
    cache = _kv4_case(rkv, n, n_kv, cap, lens, 70)
    table = torch.randperm(n * mb, generator=torch.Generator().manual_seed(9)).int().view(n, mb).cuda()
    pools = [_to_pool(x, table, block) for x in cache]
    # entries past a unit's last block are never used
    for u, t in enumerate(lens):
        table[u, t // block + 1:] = 1 << 20
    q = _normal(71, 1, n, n_kv * gqa, D)[0]
    nk, nv = (_normal(s, n, n_kv, 1, D)[:, :, 0].contiguous() for s in (72, 73))
    res = []
    for paged in (False, True):
        out, w, ol = torch.empty_like(q), torch.ones(n, n_kv, cap, device="cuda"), _ints([0] * n)
        kw = dict(new_k=nk, new_v=nv, length_out=ol, weights=w)
        if paged:
            ws = rkv.rkv_kv4_decode_paged(q, *pools, table, _ints(lens), SCALE, out, **kw)
        else:
            ws = rkv.rkv_kv4_decode(q, *cache, _ints(lens), SCALE, out, **kw)
        rkv.rkv_check_status(ws)
        res.append((out, w, ol))
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_kv4_decode_paged_bad_entry(rkv):
    n, n_kv, block = 2, 1, 16
    table = _ints([[0, 1], [7, -1]])
    cache = [torch.zeros(2, n_kv, block, w, dtype=torch.uint8, device="cuda") for w in (64, 8, 64, 8)]
    q, out = _normal(75, 1, n, 2, D)[0], torch.empty(n, 2, D, dtype=BF, device="cuda")
    ws = rkv.rkv_kv4_decode_paged(q, *cache, table, _ints([20, 20]), SCALE, out)
    with pytest.raises(rkv.RkvError) as e:
        rkv.rkv_check_status(ws)
    assert e.value.bits == 0x10


def test_kv4_decode_growing_maximum(rkv):
    """Logits that rise along the sequence (every tile has a new maximum), fall, or hold one far
    above the rest; large values with scales near the top; queries of very different size."""
    n, n_kv, gqa, t = 4, 1, 4, 400
    g = torch.Generator(device="cuda").manual_seed(80)
    q = torch.randn(n, gqa, D, generator=g, device="cuda")
    ramp = torch.linspace(-1, 1, t, device="cuda")
    k = torch.randn(n, 1, t, D, generator=g, device="cuda") * 0.1
    k[0, 0] += ramp[:, None] * q[0, 0] * 3
    k[1, 0] -= ramp[:, None] * q[1, 1] * 3
    k[2, 0, 123] = q[2, 2] * 6
    k[3] *= 3000.0
    q[3] *= 2.0 ** -12
    q[3, 1] *= 2.0 ** 20
    q[3, 2, ::2] *= 2.0 ** -18
    v = torch.randn(n, 1, t, D, generator=g, device="cuda")
    v[2] *= 20000.0
    cache, out_len = rkv.kv4_cache(n, n_kv, t), _ints([0] * n)
    rkv.rkv_check_status(rkv.rkv_kv4_append(k.to(BF), v.to(BF), *cache, _ints([0] * n), out_len))
    q = q.to(BF)
    out, w = torch.empty_like(q), torch.zeros(n, n_kv, t, device="cuda")
    rkv.rkv_check_status(rkv.rkv_kv4_decode(q, *cache, out_len, SCALE, out, weights=w))
    _check_decode(cache, [t] * n, q, out, torch.zeros_like(w), w)


def test_kv4_decode_long_unit_splits(rkv):
    n, n_kv, gqa, cap = 1, 1, 4, 70001
    lens = [70000]
    cache = _kv4_case(rkv, n, n_kv, cap, lens, 90)
    q = _normal(91, 1, n, gqa, D, spread=0.2)[0]
    out, w0 = torch.empty_like(q), torch.rand(n, n_kv, cap, device="cuda")
    w1 = w0.clone()
    rkv.rkv_check_status(rkv.rkv_kv4_decode(q, *cache, _ints(lens), SCALE, out, weights=w1))
    _check_decode(cache, lens, q, out, w0, w1)


# ------------------------------------------------------------------------------- bf16 with weights
@pytest.mark.parametrize("gqa", [1, 2, 4, 8])
@pytest.mark.parametrize("lens,cap", [([1], 1), ([0, 1, 15, 16], 17), ([1000, 129, 5], 1024),
                                      ([40000], 40001)])
def test_dense_decode_weights(rkv, gqa, lens, cap):
    n, n_kv = len(lens), 2
    k, v = _normal(100, n, n_kv, cap, D), _normal(101, n, n_kv, cap, D)
    for u, t in enumerate(lens):  # rows past the length are not to be read into a result
        k[u, :, t:] = float("nan")
        v[u, :, t:] = float("inf")
    q = _normal(102, 1, n, n_kv * gqa, D, spread=0.3)[0]
    out, w0 = torch.full_like(q, float("nan")), torch.rand(n, n_kv, cap, device="cuda")
    w1 = w0.clone()
    rkv.rkv_check_status(rkv.rkv_dense_decode_weights(q, k, v, _ints(lens), SCALE, out, w1))
    hq, ho = _f64(q).reshape(n, n_kv, gqa, D), _f64(out).reshape(n, n_kv, gqa, D)
    for u, t in enumerate(lens):
        for g in range(n_kv):
            hk, hv = _f64(k[u, g, :t]), _f64(v[u, g, :t])
            if t == 0:
                assert not ho[u, g].any()
            else:
                P.check_output(ho[u, g], hq[u, g], hk, hv, SCALE, False, 64 + t // 64, f"{u} {g}")
            P.check_weights(_f64(w1[u, g, :t]), C.softmax_weights(hq[u, g], hk, SCALE).sum(0),
                            _f64(w0[u, g, :t]), hq[u, g], hk, SCALE, 64 + t // 64, f"{u} {g}")
            assert torch.equal(w1[u, g, t:], w0[u, g, t:])


def test_dense_decode_weights_bad_lengths(rkv):
    n, n_kv, gqa, cap = 2, 1, 2, 64
    k, v = _normal(105, n, n_kv, cap, D), _normal(106, n, n_kv, cap, D)
    q = _normal(107, 1, n, gqa, D)[0]
    outs = []
    for lens in ([65, -1], [64, 0]):
        out, w = torch.empty_like(q), torch.zeros(n, n_kv, cap, device="cuda")
        ws = rkv.rkv_dense_decode_weights(q, k, v, _ints(lens), SCALE, out, w)
        outs.append((out, w))
        if lens[0] > cap:
            with pytest.raises(rkv.RkvError) as e:
                rkv.rkv_check_status(ws)
            assert e.value.bits == 0x1
    assert all(torch.equal(a, b) for a, b in zip(*outs))


# ------------------------------------------------------------------------------- prompt
@pytest.mark.parametrize("n_kv,gqa,max_q,cap,news,lens", [
    (1, 1, 1, 1, [1], [1]),
    (2, 4, 1, 300, [1, 0, 1], [300, 77, 1]),
    (1, 3, 5, 200, [5, 2], [5, 199]),
    (2, 2, 100, 513, [100, 37, 99], [100, 513, 511]),
    (1, 4, 255, 600, [255, 1], [600, 600]),
    (1, 2, 256, 700, [256, 200, 3], [256, 700, 650]),
    (2, 1, 700, 700, [700, 301], [700, 400]),
    (1, 8, 333, 1500, [333], [1499]),
    (1, 64, 20, 300, [20], [299]),
])
def test_prompt_weights(rkv, n_kv, gqa, max_q, cap, news, lens):
    n = len(lens)
    k = _normal(110, n, n_kv, cap, D)
    q = _normal(111, n, n_kv * gqa, max_q, D, spread=0.2)
    for u in range(n):  # unused rows must not matter
        k[u, :, lens[u]:] = float("nan")
        q[u, :, news[u]:] = float("nan")
    w0 = torch.rand(n, n_kv, cap, device="cuda")
    w1 = w0.clone()
    ws = rkv.rkv_prompt_weights(q, _ints(news), k, _ints(lens), SCALE, w1)
    rkv.rkv_check_status(ws)
    for u in range(n):
        T, L = news[u], lens[u]
        for g in range(n_kv):
            hk = _f64(k[u, g, :L])
            hq = _f64(q[u, g * gqa:(g + 1) * gqa, :T])
            added = C.prompt_weights(hq, hk, SCALE) if T else np.zeros(L)
            P.check_weights(_f64(w1[u, g, :L]), added, _f64(w0[u, g, :L]), hq.reshape(-1, D), hk,
                            SCALE, 96 + L // 16 + gqa * T // 64, f"unit {u} head {g}")
            assert torch.equal(w1[u, g, L:], w0[u, g, L:])


def test_prompt_weights_in_chunks(rkv):
    """A prompt in chunks adds up to the prompt at once, and to its number of queries."""
    n, n_kv, gqa, L = 1, 2, 4, 900
    k, q = _normal(115, n, n_kv, L, D), _normal(116, n, n_kv * gqa, L, D, spread=0.2)
    whole, parts = torch.zeros(2, n, n_kv, L, device="cuda")
    rkv.rkv_check_status(rkv.rkv_prompt_weights(q, _ints([L]), k, _ints([L]), SCALE, whole))
    at = 0
    for t in (1, 299, 300, 17, 283):
        c = q[:, :, at:at + t].contiguous()
        at += t
        rkv.rkv_check_status(rkv.rkv_prompt_weights(c, _ints([t]), k, _ints([at]), SCALE, parts))
    assert at == L
    hk, hq = _f64(k[0, 0]), _f64(q[0, :gqa])
    P.check_weights(_f64(parts[0, 0]), C.prompt_weights(hq, hk, SCALE), np.zeros(L),
                    hq.reshape(-1, D), hk, SCALE, 96 + L // 16 + gqa * L // 64 + 5)
    assert torch.allclose(whole, parts, rtol=1e-4)
    assert abs(whole[0, 0].double().sum().item() - gqa * L) < 1e-3 * gqa * L


def test_prompt_weights_bad_units(rkv):
    n, n_kv, gqa, T, cap = 5, 1, 2, 10, 64
    k, q = _normal(117, n, n_kv, cap, D), _normal(118, n, n_kv * gqa, T, D)
    w = torch.zeros(n, n_kv, cap, device="cuda")
    ws = rkv.rkv_prompt_weights(q, _ints([11, 10, -1, 5, 10]), k, _ints([64, 9, 20, 65, 64]), SCALE, w)
    with pytest.raises(rkv.RkvError) as e:
        rkv.rkv_check_status(ws)
    assert e.value.bits == 0x3
    assert not w[:4].any() and w[4].all()


# ------------------------------------------------------------------------------- eviction
def _evict_case(n, n_kv, cap, lens, keep, seed, ties=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.exp(2 * torch.randn(n, n_kv, cap, generator=g, device="cuda"))
    if ties:
        w = torch.randint(0, 3, (n, n_kv, cap), generator=g, device="cuda").float()
    pos = torch.full((n, n_kv, cap), -1, dtype=I32, device="cuda")
    known = min(keep, cap)
    pos[..., :known] = torch.rand(n, n_kv, known + 50, generator=g, device="cuda").argsort(-1)[..., :known].int()
    return w, pos


@pytest.mark.parametrize("n,n_kv,cap,lens,keep,recent", [
    (1, 1, 2, [2], 1, 0),
    (1, 1, 2, [2], 1, 1),
    (3, 2, 100, [100, 65, 64], 64, 10),
    (4, 2, 100, [0, 1, 63, 100], 64, 64),
    (2, 3, 5000, [5000, 4097], 4096, 33),
    (2, 2, 5000, [4999, 700], 17, 5),
    (1, 2, 1100, [1100], 1024, 0),
    (1, 1, 40, [30], 50, 3),
])
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("kv4", [False, True])
def test_evict(rkv, n, n_kv, cap, lens, keep, recent, ties, kv4):
    w, pos = _evict_case(n, n_kv, cap, lens, keep, 120, ties)
    seen = [t + 50 for t in lens]
    if kv4:
        cache = _filled_cache(rkv, n, n_kv, cap, 121)
    else:
        cache = [_normal(122, n, n_kv, cap, D), _normal(123, n, n_kv, cap, D)]
    for in_place in (False, True):
        rows = [x.clone() for x in cache]
        length, win, pin = _ints(lens), w.clone(), pos.clone()
        if in_place:
            lo, wo, po = length, win, pin
        else:
            lo, wo, po = torch.zeros_like(length), torch.full_like(w, 5.0), torch.full_like(pos, 9)
        w_was, p_was = wo.clone(), po.clone()
        src = torch.full((n, n_kv, keep), -9, dtype=I32, device="cuda")
        call = rkv.rkv_evict_kv4 if kv4 else rkv.rkv_evict
        ws = call(*rows, length, win, pin, _ints(seen), keep, recent, lo, wo, po, src_rows=src)
        rkv.rkv_check_status(ws)
        assert lo.tolist() == [min(t, keep) for t in lens]
        for u, t in enumerate(lens):
            m = min(t, keep)
            for g in range(n_kv):
                want, at = C.evict(_f64(w[u, g, :t]), _np(pos[u, g, :t]), seen[u], keep, recent)
                assert src[u, g, :m].tolist() == want.tolist()
                assert (src[u, g, m:] == -1).all()
                ix = torch.tensor(want, device="cuda", dtype=torch.long)
                assert torch.equal(wo[u, g, :m], w[u, g, ix])
                assert po[u, g, :m].tolist() == list(at)
                assert (wo[u, g, m:t] == 0).all() and (po[u, g, m:t] == -1).all()
                assert torch.equal(wo[u, g, t:], w_was[u, g, t:])
                assert torch.equal(po[u, g, t:], p_was[u, g, t:])
                for now, was in zip(rows, cache):
                    assert torch.equal(now[u, g, :m].view(torch.uint8), was[u, g, ix].view(torch.uint8))
                    assert torch.equal(now[u, g, m:].view(torch.uint8), was[u, g, m:].view(torch.uint8))


@pytest.mark.parametrize("n,n_kv,cap,lens,keep,recent", [
    (40, 8, 300, [300 - 7 * u for u in range(40)], 100, 20),   # a CTA of its own for every SM
    (1, 2, 45000, [45000], 20000, 100),                        # more rows than shared memory holds
    (1, 1, 40960, [40959], 33, 32),
    (2, 1, 9000, [9000, 8999], 8998, 0),
])
@pytest.mark.parametrize("kv4", [False, True])
def test_evict_many_and_long(rkv, n, n_kv, cap, lens, keep, recent, kv4):
    w, pos = _evict_case(n, n_kv, cap, lens, keep, 125)
    w[:, :, ::3] = w[:, :, :1]  # many equal weights
    seen = [t + 50 for t in lens]
    cache = (_filled_cache(rkv, n, n_kv, cap, 126) if kv4 else
             [_normal(127, n, n_kv, cap, D), _normal(128, n, n_kv, cap, D)])
    rows = [x.clone() for x in cache]
    length, win, pin = _ints(lens), w.clone(), pos.clone()
    src = torch.full((n, n_kv, keep), -9, dtype=I32, device="cuda")
    call = rkv.rkv_evict_kv4 if kv4 else rkv.rkv_evict
    rkv.rkv_check_status(call(*rows, length, win, pin, _ints(seen), keep, recent, length, win, pin,
                              src_rows=src))
    assert length.tolist() == [min(t, keep) for t in lens]
    for u, t in enumerate(lens):
        m = min(t, keep)
        for g in range(n_kv):
            want, at = C.evict(_f64(w[u, g, :t]), _np(pos[u, g, :t]), seen[u], keep, recent)
            assert np.array_equal(_np(src[u, g, :m]), want)
            ix = torch.tensor(want, device="cuda", dtype=torch.long)
            assert torch.equal(win[u, g, :m], w[u, g, ix])
            assert np.array_equal(_np(pin[u, g, :m]), at)
            assert (win[u, g, m:t] == 0).all() and (pin[u, g, m:t] == -1).all()
            for now, was in zip(rows, cache):
                assert torch.equal(now[u, g, :m].view(torch.uint8), was[u, g, ix].view(torch.uint8))
                assert torch.equal(now[u, g, m:].view(torch.uint8), was[u, g, m:].view(torch.uint8))


@pytest.mark.parametrize("n,n_kv,cap,lens,keep", [
    (1, 1, 2047, [2047], 1000), (1, 1, 2048, [2048], 1), (3, 1, 4100, [4100, 33, 3000], 2999),
    (2, 1, 40000, [40000, 70], 60),                       # a unit that leaves most of its CTAs none
    (1, 3, 70001, [70001], 70000), (20, 1, 8191, [8191 - 31 * u for u in range(20)], 5000),
    (1, 1, 261888, [261888], 130000), (1, 1, 261889, [261889], 130000),  # the most rows of a cluster
    (160, 1, 41000, [41000 if u == 7 else u for u in range(160)], 500),
])
@pytest.mark.parametrize("equal", [False, True])
def test_evict_over_clusters(rkv, n, n_kv, cap, lens, keep, equal):
    w, pos = _evict_case(n, n_kv, cap, lens, keep, 135)
    if equal:
        w[:, :, 1::2] = w[:, :, :1]
    seen = [t + 50 for t in lens]
    k = torch.arange(n * n_kv * cap, device="cuda").view(n, n_kv, cap, 1).expand(-1, -1, -1, 8)
    rows = [torch.zeros(n, n_kv, cap, x, dtype=torch.uint8, device="cuda") for x in (64, 8, 64, 8)]
    rows[1].copy_((k >> torch.arange(0, 64, 8, device="cuda")) & 0xff)  # each row its own number
    was = rows[1].clone()
    length, win, pin = _ints(lens), w.clone(), pos.clone()
    recent = min(16, keep)
    rkv.rkv_check_status(rkv.rkv_evict_kv4(*rows, length, win, pin, _ints(seen), keep, recent, length, win,
                                           pin))
    assert length.tolist() == [min(t, keep) for t in lens]
    for u, t in enumerate(lens):
        m = min(t, keep)
        for g in range(n_kv):
            want, at = C.evict(_f64(w[u, g, :t]), _np(pos[u, g, :t]), seen[u], keep, recent)
            ix = torch.tensor(want, device="cuda", dtype=torch.long)
            assert torch.equal(win[u, g, :m], w[u, g, ix]) and np.array_equal(_np(pin[u, g, :m]), at)
            assert (win[u, g, m:t] == 0).all() and (pin[u, g, m:t] == -1).all()
            assert torch.equal(win[u, g, t:], w[u, g, t:]) and torch.equal(pin[u, g, t:], pos[u, g, t:])
            assert torch.equal(rows[1][u, g, :m], was[u, g, ix])
            assert torch.equal(rows[1][u, g, m:], was[u, g, m:])


def test_evict_special_weights(rkv):
    """Zeros of either sign tie, infinities and NaN are largest, the newest rows come first."""
    w = torch.tensor([0.0, -0.0, float("nan"), 1.0, float("inf"), 2.0, 0.0, 0.0], device="cuda").view(1, 1, 8)
    pos = torch.full((1, 1, 8), -1, dtype=I32, device="cuda")
    k, v = _normal(130, 1, 1, 8, D), _normal(131, 1, 1, 8, D)
    for keep, want in ((3, [6, 7, 2]), (4, [4, 7, 2, 6]), (6, [6, 7, 2, 3, 4, 5]),
                       (7, [0, 7, 2, 3, 4, 5, 6])):
        src = torch.empty(1, 1, keep, dtype=I32, device="cuda")
        lo, wo, po = _ints([0]), torch.empty_like(w), torch.empty_like(pos)
        rkv.rkv_check_status(rkv.rkv_evict(k.clone(), v.clone(), _ints([8]), w, pos, _ints([8]), keep,
                                           2, lo, wo, po, src_rows=src))
        assert sorted(src[0, 0].tolist()) == sorted(want), keep


def test_evict_bad_lengths(rkv):
    w, pos = _evict_case(2, 1, 32, [33, -1], 8, 132)
    k = _normal(133, 2, 1, 32, D)
    v = k.clone()
    lo, wo, po = _ints([0, 0]), torch.full_like(w, 5.0), torch.full_like(pos, 9)
    ws = rkv.rkv_evict(k, v, _ints([33, -1]), w, pos, _ints([33, 33]), 8, 2, lo, wo, po)
    with pytest.raises(rkv.RkvError) as e:
        rkv.rkv_check_status(ws)
    assert e.value.bits == 0x1 and lo.tolist() == [33, -1]
    assert (wo == 5.0).all() and (po == 9).all() and torch.equal(k, v)


# ------------------------------------------------------------------------------- together
@pytest.mark.parametrize("kv4", [True, False])
def test_generation_with_eviction(rkv, kv4):
    """A prompt in two chunks, then decode steps; the cache is shrunk whenever it has outgrown its
    budget. Every step is checked against the oracle over the rows the cache holds."""
    n, n_kv, gqa, keep, recent, slack, steps = 2, 2, 4, 96, 16, 8, 20
    prompt = [150, 131]
    cap = 160
    T = max(prompt)
    k, v = _normal(140, n, n_kv, T, D), _normal(141, n, n_kv, T, D)
    q = _normal(142, n, n_kv * gqa, T, D, spread=0.2)
    nk, nv = _normal(143, steps, n, n_kv, D), _normal(144, steps, n, n_kv, D)
    nq = _normal(145, steps, n, n_kv * gqa, D, spread=0.2)
    weights = torch.zeros(n, n_kv, cap, device="cuda")
    pos = torch.full((n, n_kv, cap), -1, dtype=I32, device="cuda")
    length, seen = _ints([0] * n), _ints(prompt)
    if kv4:
        cache = rkv.kv4_cache(n, n_kv, cap)
        kv_, vv_ = torch.zeros_like(k), torch.zeros_like(v)
        rkv.rkv_check_status(rkv.rkv_kv4_append(k, v, *cache, length, length, new_len=_ints(prompt),
                                                k_values=kv_, v_values=vv_))
        keys = kv_
    else:
        cache = [torch.zeros(n, n_kv, cap, D, dtype=BF, device="cuda") for _ in range(2)]
        cache[0][:, :, :T], cache[1][:, :, :T] = k, v
        length.copy_(_ints(prompt))
        keys = k
    # the prompt's weights, over the keys that the decode sees, in two chunks
    for a, b in ((0, 64), (64, T)):
        new = [min(b, p) - a for p in prompt]
        rkv.rkv_check_status(_prompt_into(rkv, q, keys, weights, a, b, new, prompt))
    for u, L in enumerate(prompt):
        hq, hk = _f64(q[u, :gqa, :L]), _f64(keys[u, 0, :L])
        P.check_weights(_f64(weights[u, 0, :L]), C.prompt_weights(hq, hk, SCALE), np.zeros(L),
                        hq.reshape(-1, D), hk, SCALE, 128, f"prompt {u}")
    # what each head's rows are, by position
    truth = [[list(range(p)) for _ in range(n_kv)] for p in prompt]
    for s in range(steps):
        if int(length.max()) > keep + slack:
            before = (weights.clone(), pos.clone(), length.tolist())
            call = rkv.rkv_evict_kv4 if kv4 else rkv.rkv_evict
            rkv.rkv_check_status(call(*cache, length, weights, pos, seen, keep, recent, length, weights, pos))
            for u in range(n):
                t = before[2][u]
                for g in range(n_kv):
                    src, at = C.evict(_f64(before[0][u, g, :t]), _np(before[1][u, g, :t]),
                                      int(seen[u]), keep, recent)
                    truth[u][g] = [truth[u][g][i] for i in src]
                    if t > keep:
                        assert truth[u][g] == list(at) == pos[u, g, :keep].tolist()
        w0 = weights.clone()
        out = torch.empty(n, n_kv * gqa, D, dtype=BF, device="cuda")
        if kv4:
            rkv.rkv_check_status(rkv.rkv_kv4_decode(nq[s], *cache, length, SCALE, out, new_k=nk[s],
                                                    new_v=nv[s], length_out=length, weights=weights))
        else:
            for u, t in enumerate(length.tolist()):
                cache[0][u, :, t], cache[1][u, :, t] = nk[s, u], nv[s, u]
            length += 1
            rkv.rkv_check_status(rkv.rkv_dense_decode_weights(nq[s], *cache, length, SCALE, out, weights))
        seen += 1
        for u in range(n):
            for g in range(n_kv):
                truth[u][g].append(prompt[u] + s)
                t = int(length[u])
                if kv4:
                    hk, hv = (C.kv4_values(_np(cache[i][u, g, :t]), _np(cache[i + 1][u, g, :t])) for i in (0, 2))
                else:
                    hk, hv = _f64(cache[0][u, g, :t]), _f64(cache[1][u, g, :t])
                # the rows are the tokens that they should be
                tok_k = torch.cat((keys[u, g, :prompt[u]], nk[:, u, g]))[truth[u][g]]
                want = _f64(tok_k)
                if kv4:
                    want = C.kv4_values(*C.kv4_quantise(want))
                assert np.array_equal(hk, want), (s, u, g)
                hq = _f64(nq[s, u, g * gqa:(g + 1) * gqa])
                P.check_output(_f64(out[u, g * gqa:(g + 1) * gqa]), hq, hk, hv, SCALE, kv4, 64, f"step {s}")
                P.check_weights(_f64(weights[u, g, :t]), C.softmax_weights(hq, hk, SCALE).sum(0),
                                _f64(w0[u, g, :t]), hq, hk, SCALE, 64, f"step {s}")


def _prompt_into(rkv, q, keys, weights, a, b, new, prompt):
    """Weights of queries [a, b) added to the first columns of a wider array."""
    T = keys.shape[2]
    w = weights[:, :, :T].contiguous()
    ws = rkv.rkv_prompt_weights(q[:, :, a:b].contiguous(), _ints(new), keys,
                                _ints([min(b, p) for p in prompt]), SCALE, w)
    weights[:, :, :T] = w
    return ws


# ------------------------------------------------------------------------------- streams, graphs
def test_side_stream_and_graph(rkv):
    """The calls run on the stream they are given, with a workspace of their own, and a captured
    step replays on new contents."""
    n, n_kv, gqa, cap = 2, 2, 4, 520
    cache = _kv4_case(rkv, n, n_kv, cap, [512, 300], 150)
    q = _normal(151, 1, n, n_kv * gqa, D)[0]
    nk, nv = (_normal(s, n, n_kv, 1, D)[:, :, 0].contiguous() for s in (152, 153))
    ref, w_ref, l_ref = torch.empty_like(q), torch.zeros(n, n_kv, cap, device="cuda"), _ints([512, 300])
    saved = [x.clone() for x in cache]
    for _ in range(2):
        rkv.rkv_check_status(rkv.rkv_kv4_decode(q, *cache, l_ref, SCALE, ref, new_k=nk, new_v=nv,
                                                length_out=l_ref, weights=w_ref))
    for x, y in zip(cache, saved):
        x.copy_(y)
    out, w, length = torch.empty_like(q), torch.zeros_like(w_ref), _ints([512, 300])
    ws = rkv.workspace(rkv.rkv_kv4_decode_workspace_bytes(n, n_kv, gqa, cap, True), "cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    rkv.rkv_kv4_decode(q, *cache, length, SCALE, out, new_k=nk, new_v=nv, length_out=length, weights=w,
                       stream=side)
    side.synchronize()
    for x, y in zip(cache, saved):
        x.copy_(y)
    w.zero_()
    length.copy_(_ints([512, 300]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rkv.rkv_kv4_decode(q, *cache, length, SCALE, out, new_k=nk, new_v=nv, length_out=length,
                           weights=w, ws=ws)
    assert length.tolist() == [512, 300]  # captured, not run
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    rkv.rkv_check_status(ws)
    assert torch.equal(out, ref) and torch.equal(w, w_ref) and torch.equal(length, l_ref)


def test_prompt_and_evict_in_a_graph(rkv):
    n, n_kv, gqa, L, keep = 1, 2, 4, 400, 256
    k, q = _normal(160, n, n_kv, L, D), _normal(161, n, n_kv * gqa, L, D, spread=0.2)
    v = _normal(162, n, n_kv, L, D)
    pos = torch.full((n, n_kv, L), -1, dtype=I32, device="cuda")
    res = []
    for captured in (False, True):
        kk, vv, w = k.clone(), v.clone(), torch.zeros(n, n_kv, L, device="cuda")
        lo, wo, po = _ints([0]), torch.zeros_like(w), pos.clone()
        ql, ln = _ints([L]), _ints([L])
        wp = rkv.workspace(rkv.rkv_prompt_weights_workspace_bytes(n, n_kv, gqa, L, L), "cuda")
        we = rkv.workspace(rkv.rkv_evict_workspace_bytes(n, n_kv, L, keep), "cuda")

        def step():
            rkv.rkv_prompt_weights(q, ql, kk, ln, SCALE, w, ws=wp)
            rkv.rkv_evict(kk, vv, ln, w, pos, ln, keep, 32, lo, wo, po, ws=we)
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        rkv.rkv_check_status(wp)
        rkv.rkv_check_status(we)
        res.append((kk, vv, w, lo, wo, po))
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_workspace_contents_do_not_matter(rkv):
    """One workspace for every call and shape, full of bytes but for its status word."""
    ws = torch.full((64 << 20,), 0xA5, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    for n, n_kv, gqa, cap in ((2, 2, 4, 300), (40, 2, 2, 700), (1, 1, 8, 20000)):
        lens = [cap - 1 - 3 * u for u in range(n)]
        cache = _kv4_case(rkv, n, n_kv, cap, lens, 170)
        q = _normal(171, 1, n, n_kv * gqa, D)[0]
        nk = _normal(172, n, n_kv, 1, D)[:, :, 0].contiguous()
        k, v = _normal(173, n, n_kv, cap, D), _normal(174, n, n_kv, cap, D)
        qp = _normal(175, n, n_kv * gqa, 50, D)
        pos = torch.full((n, n_kv, cap), -1, dtype=I32, device="cuda")
        res = []
        for shared in (False, True):
            w = ws if shared else None
            c = [x.clone() for x in cache]
            kk, vv = k.clone(), v.clone()
            out, wt, ln = torch.empty_like(q), torch.zeros(n, n_kv, cap, device="cuda"), _ints(lens)
            p, seen = pos.clone(), _ints(lens)
            o2, w2 = torch.empty_like(q), torch.zeros_like(wt)
            for call in (
                lambda: rkv.rkv_kv4_decode(q, *c, ln, SCALE, out, new_k=nk, new_v=nk, length_out=ln,
                                           weights=wt, ws=w),
                lambda: rkv.rkv_dense_decode_weights(q, kk, vv, seen, SCALE, o2, w2, ws=w),
                lambda: rkv.rkv_prompt_weights(qp, _ints([50] * n), kk, seen, SCALE, w2, ws=w),
                lambda: rkv.rkv_evict(kk, vv, seen, w2, p, seen, 100, 9, seen, w2, p, ws=w),
                lambda: rkv.rkv_evict_kv4(*c, ln, wt, pos, ln, 200, 9, ln, wt, p, ws=w),
            ):
                rkv.rkv_check_status(call())
            res.append((out, wt, ln, *c, o2, w2, kk, vv, seen, p))
        for a, b in zip(*res):
            assert torch.equal(a, b)


def test_rows_without_a_block_are_not_stored(rkv):
    n, n_kv, block, gqa = 2, 2, 16, 4
    pools = [torch.full((5, n_kv, block, w), 0x11, dtype=torch.uint8, device="cuda") for w in (64, 8, 64, 8)]
    table = _ints([[1, 2], [3, 9]])  # the second unit's second block is none
    lens = _ints([20, 15])
    q, out = _normal(180, 1, n, n_kv * gqa, D)[0], torch.empty(n, n_kv * gqa, D, dtype=BF, device="cuda")
    new, ln = _normal(181, n, n_kv, 3, D), torch.zeros_like(lens)
    first = [x[0].clone() for x in pools]
    ws = rkv.rkv_kv4_append_paged(new, new, *pools, table, lens, ln)
    with pytest.raises(rkv.RkvError) as e:
        rkv.rkv_check_status(ws)
    assert e.value.bits == 0x10 and ln.tolist() == [23, 18]
    row = new[:, :, 0].contiguous()
    ws = rkv.rkv_kv4_decode_paged(q, *pools, table, ln, SCALE, out, new_k=row, new_v=row, length_out=ln)
    with pytest.raises(rkv.RkvError) as e:
        rkv.rkv_check_status(ws)
    assert e.value.bits == 0x10 and ln.tolist() == [24, 19]
    for x, was in zip(pools, first):
        assert torch.equal(x[0], was) and (x[4] == 0x11).all()
        assert (x[3, :, :15] == 0x11).all()
    assert (pools[0][2, :, 4:8] != 0x11).any(-1).all() and (pools[0][3, :, 15] != 0x11).any()


def test_lengths_out_may_be_any_input(rkv):
    n, n_kv, cap, keep = 160, 3, 40, 8
    lens = [(7 * u) % (cap - 4) for u in range(n)]
    news = [u % 4 for u in range(n)]
    new = _normal(190, n, n_kv, 4, D)
    a, b = (rkv.kv4_cache(n, n_kv, cap) for _ in range(2))
    out, same = _ints([0] * n), _ints(news)
    rkv.rkv_check_status(rkv.rkv_kv4_append(new, new, *a, _ints(lens), out, new_len=_ints(news)))
    rkv.rkv_check_status(rkv.rkv_kv4_append(new, new, *b, _ints(lens), same, new_len=same))
    assert torch.equal(out, same) and out.tolist() == [x + y for x, y in zip(lens, news)]
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    w = torch.rand(n, n_kv, cap, device="cuda")
    pos = torch.full((n, n_kv, cap), -1, dtype=I32, device="cuda")
    res = []
    for alias in (False, True):
        k, v = _normal(191, n, n_kv, cap, D), _normal(192, n, n_kv, cap, D)
        seen, wo, po = _ints([x + 3 for x in lens]), w.clone(), pos.clone()
        lo = seen if alias else torch.zeros_like(seen)
        rkv.rkv_check_status(rkv.rkv_evict(k, v, _ints(lens), w, pos, seen, keep, 3, lo, wo, po))
        res.append((k, v, wo, po, lo))
    for x, y in zip(*res):
        assert torch.equal(x, y)
    assert res[0][4].tolist() == [min(x, keep) for x in lens]
