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


def test_a_tile_without_rows_waits_as_long_as_an_item():
    """Items of one tile, then items of two: the second tile's warps are at the second item from the start, and wait for it
    longer than a step's limit. Only block 0, one load of which is never requested, gives up."""
    from sparse_kv_cache_snapkv_gb300 import rkv
    n_kv, cap, limit = 8, 51200, 200000  # 400 steps of an item: some 500 us; a step's limit of 200 us
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    some = -(-sms // n_kv)  # units whose items fill the GPU once
    news, lens = [1] * some + [64] * some, [cap] * some + [cap - 128] * some
    q_start = torch.tensor([sum(news[:u]) for u in range(2 * some + 1)], dtype=torch.int32, device="cuda")
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(sum(news), 4 * n_kv, 128, generator=g, device="cuda").bfloat16()
    k, v = (torch.empty(2 * some, n_kv, cap, 128, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in "kv")
    want, got = torch.zeros_like(q), torch.zeros_like(q)
    rkv.rkv_check_status(rkv.rkv_prompt_attention(q, q_start, k, v, length, SCALE, want))
    # the queries of block 0's first tile: the largest items come first, the units of one token among themselves by number
    ws = rkv.rkv_testing_attention_wait_timeout(q, q_start, k, v, length, SCALE, got, 1, limit)
    with pytest.raises(rkv.RkvError) as e:
        rkv.rkv_check_status(ws)
    assert e.value.bits == 4
    # block 0 has an item of each wave at most, and each is one unit's for one KV head
    wrong = (got != want).any(-1)
    lost = {(u, h // 4) for u in range(2 * some) for h in range(4 * n_kv)
            if wrong[int(q_start[u]):int(q_start[u + 1]), h].any()}
    assert 1 <= len(lost) <= 3, sorted(lost)
