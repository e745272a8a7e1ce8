"""Packed attention whose waits run out, with calls right behind it on the stream: what a block that gave up had under way
(copies, products into tensor memory) has ended before the memory is another's."""
import pytest
import torch

from tests.test_gpu_serve_attention import SCALE, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", [1, 2, 3])
@pytest.mark.parametrize("news,lens", [([700, 65], [700, 1000]), ([64], [9000])])
def test_the_calls_behind_are_right(what, news, lens):
    from sparse_kv_cache_snapkv_gb300 import rkv
    c = Case(70 + what, news, lens)
    want, ws = c.call()
    rkv.rkv_check_status(ws)
    c.check(want)
    need = rkv.rkv_prompt_attention_workspace_bytes(c.n, c.n_kv, c.gqa, c.tokens)
    for limit in (1000, 20000):
        bad, good = rkv.workspace(need, "cuda"), rkv.workspace(need, "cuda")
        scrap, outs = torch.zeros_like(want), [torch.zeros_like(want) for _ in range(3)]
        rows = [t for u, T in enumerate(news) for t in range(c.starts[u], c.starts[u] + T)]
        for out in outs:
            rkv.rkv_testing_attention_wait_timeout(c.q, c.q_start, c.k, c.v, c.len, SCALE, scrap, what, limit, ws=bad)
            c.call(out=out, ws=good)
        rkv.rkv_check_status(good)
        with pytest.raises(rkv.RkvError) as e:
            rkv.rkv_check_status(bad)
        assert e.value.bits == 4
        for out in outs:
            assert torch.equal(out[rows], want[rows])
