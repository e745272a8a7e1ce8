"""The cache calls at once on several streams, each with a workspace of its own: the results of calls one after
the other, bit for bit, every time."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128
SCALE = 1.0 / math.sqrt(D)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def test_calls_at_once():
    from sparse_kv_cache_snapkv_gb300 import rkv
    rkv.load()
    n, n_kv, gqa, cap, T = 4, 2, 4, 3000, 700
    k, v, q = _rand(1, n, n_kv, cap, D), _rand(2, n, n_kv, cap, D), _rand(3, n, n_kv * gqa, D)
    qp, lens = _rand(4, n, n_kv * gqa, T, D), [3000, 1, 2222, 700]
    ln, news = _ints(lens), _ints([min(T, t) for t in lens])
    w = torch.rand(n, n_kv, cap, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    pos = torch.full((n, n_kv, cap), -1, dtype=torch.int32, device="cuda")
    held = rkv.kv4_cache(n, n_kv, cap)
    rkv.rkv_check_status(rkv.rkv_kv4_append(k, v, *held, _ints([0] * n), torch.empty_like(ln), new_len=ln))

    def decode4(s):
        out, x = torch.empty_like(q), w.clone()
        ws = rkv.rkv_kv4_decode(q, *held, ln, SCALE, out, weights=x, stream=s)
        return ws, (out, x)

    def decode16(s):
        out, x = torch.empty_like(q), w.clone()
        ws = rkv.rkv_dense_decode_weights(q, k, v, ln, SCALE, out, x, stream=s)
        return ws, (out, x)

    def prompt(s):
        x = w.clone()
        return rkv.rkv_prompt_weights(qp, news, k, ln, SCALE, x, stream=s), (x,)

    def evict(s):
        kk, vv, x, p, m = k.clone(), v.clone(), w.clone(), pos.clone(), ln.clone()
        return rkv.rkv_evict(kk, vv, m, x, p, ln, 900, 64, m, x, p, stream=s), (kk, vv, x, p, m)

    def append(s):
        c, m = rkv.kv4_cache(n, n_kv, cap), _ints([0] * n)
        return rkv.rkv_kv4_append(k, v, *c, m, m, new_len=ln, stream=s), (*c, m)

    calls = (decode4, decode16, prompt, evict, append)
    streams = [torch.cuda.Stream() for _ in calls]
    want = []
    for call, s in zip(calls, streams):
        with torch.cuda.stream(s):
            want.append(call(s))
        torch.cuda.synchronize()
    for turn in range(25):
        got = []
        for i in range(len(calls)):
            j = (i + turn) % len(calls)
            with torch.cuda.stream(streams[j]):
                got.append((j, calls[j](streams[j])))
        torch.cuda.synchronize()
        for j, (ws, res) in got:
            rkv.rkv_check_status(ws)
            assert all(torch.equal(a, b) for a, b in zip(res, want[j][1])), (turn, calls[j].__name__)
