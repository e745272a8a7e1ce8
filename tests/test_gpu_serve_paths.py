"""The serving step's calls together, on other streams, in graphs, with waits that run out, and what lies around their
workspaces and outputs."""
import math

import numpy as np
import pytest
import torch

from oracle import serve as S
from tests import serve_parity as P
from tests.test_gpu_serve_attention import Case, tree_masks

pytestmark = pytest.mark.gpu

D = 128
SCALE = 1.0 / math.sqrt(D)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _np(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------------------------------------ a request's life
class Serving:
    """A small engine: prompts, then drafted trees of which a path is accepted, then decode steps, on a paged cache."""

    def __init__(self, n, n_kv, gqa, block, most, blocks, seed):
        from sparse_kv_cache_snapkv_gb300 import rkv
        self.rkv, self.n, self.n_kv, self.hq, self.block, self.most = rkv, n, n_kv, n_kv * gqa, block, most
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.pools = [torch.full((blocks, n_kv, block, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        self.table = torch.full((n, most), -1, dtype=torch.int32, device="cuda")
        self.len, self.held, self.count = _ints([0] * n), _ints([0] * n), _ints([blocks])
        self.free = torch.randperm(blocks, generator=self.g, device="cuda").int()
        self.freq, self.mscale = rkv.rkv_rope_frequencies(D, 10000.0, "by_parts", factor=4.0, ctx=512)
        self.kept = [[] for _ in range(n)]  # (turned keys, values) of each request's tokens, in 64 bits

    def step(self, new, mask=None, depth=None, room=None):
        """New tokens of every request; returns (q as the attention sees it, starts, outputs)."""
        rkv, n, total = self.rkv, self.n, sum(new)
        room = room or total
        q_start, slots, positions = _ints([0] * (n + 1)), _ints([0] * room), _ints([0] * room)
        ws = rkv.rkv_reserve_slots(_ints(new), self.len, self.held, self.table, self.free, self.count, self.block, q_start,
                                   slots, positions, self.len, self.held, self.count)
        rkv.rkv_check_status(ws)
        if depth is not None:  # a drafted token stands behind its ancestors
            positions.copy_(_ints(depth + [0] * (room - total)))
        qkv = torch.randn(room, self.hq + 2 * self.n_kv, D, generator=self.g, device="cuda").bfloat16()
        q, k, v = qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.n_kv], qkv[:, self.hq + self.n_kv:]
        out, turned = (torch.full((room, self.hq, D), 768.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        rkv.rkv_check_status(rkv.rkv_rope_append(q, k, v, positions, self.freq.cuda(), slots, turned, *self.pools,
                                                 mscale=self.mscale))
        args = (self.table, self.len, SCALE, out)
        if mask is None:
            ws = rkv.rkv_prompt_attention_paged(turned, q_start, *self.pools, *args)
        else:
            ws = rkv.rkv_tree_attention_paged(turned, q_start, mask, *self.pools, *args)
        rkv.rkv_check_status(ws)
        at = q_start.tolist()
        assert at[-1] == total
        self.last = (k, v, positions)
        for u in range(n):
            rows = slice(at[u], at[u + 1])
            k64 = S.turn(_np(k[rows]), positions[rows].tolist(), self.freq.double().numpy(), False, self.mscale)
            # what the cache holds: the turned keys rounded to bf16
            k16 = torch.tensor(k64).to(torch.bfloat16).double().numpy()
            self.kept[u] += list(zip(k16, _np(v[rows])))
        return turned, at, out

    def check(self, turned, at, out, mask=None):
        for u in range(self.n):
            T, L = at[u + 1] - at[u], len(self.kept[u])
            if T == 0:
                continue
            assert L == int(self.len[u])
            k, v = (np.stack([x[i] for x in self.kept[u]], 1) for i in (0, 1))
            rows = slice(at[u], at[u + 1])
            sees = S.visible(T, L, None if mask is None else mask[rows].cpu().numpy())
            q = _np(turned[rows])
            ref, mag = S.attention(q, k, v, SCALE, sees)
            tol = P.attention_tolerance(q, k, SCALE, ref, mag)
            # a key on the border of two bf16 numbers may be the other one: the logits move by 2^-8 of a term's size
            # at one of its 128 dimensions in places; bounded by moving all of them
            moved = 2.0 ** -7 * np.abs(q).max() * np.abs(k).max() * SCALE * 2
            P.within(_np(out[rows]), ref, tol + moved * mag, f"request {u}")
        assert (out[at[-1]:] == 768.0).all()


def test_a_serving_engine():
    rng = np.random.default_rng(3)
    e = Serving(n=4, n_kv=2, gqa=4, block=16, most=40, blocks=90, seed=3)
    e.check(*e.step([150, 0, 33, 1], room=192))
    e.check(*e.step([0, 200, 64, 1]))
    for round_ in range(3):
        news = [8, 5, 0, 16]
        before = e.len.tolist()
        mask = torch.tensor(tree_masks(rng, news, 1), device="cuda")
        words = mask.cpu().numpy().astype(np.int64)[:, 0] & 0xFFFFFFFF
        ones = [bin(int(w)).count("1") for w in words]
        unit = [u for u, t in enumerate(news) for _ in range(t)]
        depth = [before[u] + o - 1 for u, o in zip(unit, ones)]
        turned, at, out = e.step(news, mask=mask, depth=depth)
        e.check(turned, at, out, mask=mask)
        # accept the path to the last drafted token of each request: its rows again, in place, and the length
        k, v, positions = e.last
        rows, slots = [], []
        table = e.table.tolist()
        for u in range(e.n):
            path = [i for i in range(news[u]) if news[u] and (int(words[at[u + 1] - 1]) >> i) & 1]
            for d, i in enumerate(path):
                rows.append(at[u] + i)
                p = before[u] + d
                slots.append(table[u][p // e.block] * e.block + p % e.block)
            tail = e.kept[u][before[u]:]
            e.kept[u] = e.kept[u][:before[u]] + [tail[i] for i in path]
            before[u] += len(path)
        idx = torch.tensor(rows, device="cuda")
        scrap = torch.empty(len(rows), e.hq, D, dtype=torch.bfloat16, device="cuda")
        e.rkv.rkv_check_status(e.rkv.rkv_rope_append(torch.zeros_like(scrap), k[idx].contiguous(), v[idx].contiguous(),
                                                     positions[idx], e.freq.cuda(), _ints(slots), scrap, *e.pools,
                                                     mscale=e.mscale))
        e.len.copy_(_ints(before))
        ws = e.rkv.rkv_release_blocks(e.len, e.held, e.table, e.free, e.count, e.block, e.held, e.count)
        e.rkv.rkv_check_status(ws)
        e.check(*e.step([1, 1, 1, 1]))  # a decode step
    e.len.zero_()
    e.rkv.rkv_check_status(e.rkv.rkv_release_blocks(e.len, e.held, e.table, e.free, e.count, e.block, e.held, e.count))
    assert int(e.count) == 90


def test_prompt_into_a_contiguous_cache_then_compress_and_decode():
    """Beside the calls that were there: the rows that rope_append stores are what stage 1 and the decodes read."""
    from sparse_kv_cache_snapkv_gb300 import rkv
    n, n_kv, gqa, T, cap = 2, 2, 4, 300, 400
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn(n * T, n_kv * gqa + 2 * n_kv, D, generator=g, device="cuda").bfloat16()
    q, k, v = qkv.split((n_kv * gqa, n_kv, n_kv), 1)
    kc, vc = (torch.zeros(n, n_kv, cap, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.arange(T, device="cuda").int().repeat(n)
    slots = (torch.arange(n, device="cuda").int()[:, None] * cap + torch.arange(T, device="cuda").int()).flatten()
    freq, _ = rkv.rkv_rope_frequencies()
    turned, out = (torch.empty(n * T, n_kv * gqa, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rkv.rkv_check_status(rkv.rkv_rope_append(q, k, v, pos, freq.cuda(), slots, turned, kc, vc))
    ln = _ints([T] * n)
    rkv.rkv_check_status(rkv.rkv_prompt_attention(turned, _ints([0, T, 2 * T]), kc, vc, ln, SCALE, out))
    # the last token's attention is what the decodes give for it
    last = turned.view(n, T, -1, D)[:, -1].contiguous()
    dense, decoded = torch.empty_like(last), out.view(n, T, -1, D)[:, -1]
    rkv.rkv_check_status(rkv.rkv_dense_decode(last, kc, vc, ln, SCALE, dense))
    assert (dense.float() - decoded.float()).abs().max() <= 2.0 ** -7 * vc.float().abs().max()
    # stage 1 takes the last window's queries by head
    window, keep = 32, 128
    q_win = turned.view(n, T, -1, D)[:, -window:].transpose(1, 2).contiguous()
    k_out, v_out = (torch.zeros(n, n_kv, keep, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kept, out_len = torch.zeros(n, n_kv, keep, dtype=torch.int32, device="cuda"), _ints([0] * n)
    rkv.rkv_check_status(rkv.rkv_snapkv_compress(kc, vc, ln, q_win, 7, keep, SCALE, k_out, v_out, kept, out_len))
    assert out_len.tolist() == [keep] * n
    for u in range(n):
        for h in range(n_kv):
            assert torch.equal(k_out[u, h], kc[u, h, kept[u, h].long()])


# ------------------------------------------------------------------------------------------------ streams, graphs
def _calls():
    """Every call with inputs of its own: functions of a stream that return (workspace, outputs)."""
    from sparse_kv_cache_snapkv_gb300 import rkv
    a, b = Case(31, [300, 64, 1], [300, 3000, 777]), Case(32, [64, 9], [9000, 80], words=2, block=64)
    x = torch.randn(500, 12, D, generator=torch.Generator(device="cuda").manual_seed(33), device="cuda").bfloat16()
    freq = rkv.rkv_rope_frequencies()[0].cuda()
    pos, slots = torch.arange(500, device="cuda").int(), torch.randperm(512, device="cuda")[:500].int()
    new, ln, held = _ints([5000, 1, 3000]), _ints([100, 0, 16]), _ints([7, 0, 1])
    free, count = torch.randperm(1200, device="cuda").int(), _ints([1000])

    def attention(c):
        def f(s, ws=None):
            out, ws = c.call(stream=s, ws=ws)
            return ws, (out,)
        return f

    def rope(s, ws=None):
        out = torch.zeros(500, 8, D, dtype=torch.bfloat16, device="cuda")
        kc, vc = (torch.zeros(8, 2, 64, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return rkv.rkv_rope_append(x[:, :8], x[:, 8:10], x[:, 10:], pos, freq, slots, out, kc, vc, ws=ws,
                                   stream=s), (out, kc, vc)

    def reserve(s, ws=None):
        t = torch.full((3, 400), 1199, dtype=torch.int32, device="cuda")  # (blocks held already are blocks)
        o = [torch.zeros(m, dtype=torch.int32, device="cuda") for m in (4, 9000, 9000, 3, 3, 1)]
        return rkv.rkv_reserve_slots(new, ln, held, t, free, count, 16, *o, ws=ws, stream=s), (t, *o)

    def release(s, ws=None):
        f, o = free.clone(), [torch.zeros(m, dtype=torch.int32, device="cuda") for m in (3, 1)]
        table = torch.arange(1200, device="cuda").int().view(3, 400)
        return rkv.rkv_release_blocks(_ints([0, 0, 0]), _ints([50, 0, 30]), table, f, count, 16, *o, ws=ws,
                                      stream=s), (f, *o)

    return attention(a), attention(b), rope, reserve, release


def test_calls_at_once_on_several_streams():
    from sparse_kv_cache_snapkv_gb300 import rkv
    calls = _calls()
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    want = []
    for call, s in zip(calls, streams):
        with torch.cuda.stream(s):
            ws, out = call(s)
            rkv.rkv_check_status(ws, stream=s)
            want.append(out)
    torch.cuda.synchronize()
    for _ in range(6):
        got = []
        for call, s in zip(calls, streams):
            with torch.cuda.stream(s):
                got.append(call(s))
        torch.cuda.synchronize()
        for (ws, out), ref in zip(got, want):
            rkv.rkv_check_status(ws)
            assert all(torch.equal(x, y) for x, y in zip(out, ref))


def test_captured_and_replayed_with_one_workspace():
    """Graphs that share a workspace, replayed one after the other, with inputs that change in place between."""
    from sparse_kv_cache_snapkv_gb300 import rkv
    a, b = Case(41, [200, 64], [200, 5000]), Case(42, [64, 2], [20000, 300], words=2)
    ws = rkv.workspace(max(rkv.rkv_prompt_attention_workspace_bytes(2, 2, 4, t) for t in (a.tokens, b.tokens)), "cuda")
    outs, graphs = [], []
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for c in (a, b):
            c.call(ws=ws)
            out = torch.full((c.tokens, 8, D), 768.0, dtype=torch.bfloat16, device="cuda")
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                c.call(out=out, ws=ws)
            outs.append(out)
            graphs.append(g)
        for seed in range(3):
            for c, g, out in zip((a, b), graphs, outs):
                c.q.copy_(torch.randn(c.q.shape, device="cuda").bfloat16())
                if seed == 1:  # other lengths: other pieces
                    c.len.copy_(_ints([c.lens[0], 77 if c is a else 100]))
                    c.lens = c.len.tolist()
                    c.news = [c.news[0], min(c.news[1], c.lens[1])]
                g.replay()
                s.synchronize()
                rkv.rkv_check_status(ws, stream=s)
                c.check(out)


def test_workspace_contents_do_not_matter_and_nothing_is_written_behind():
    from sparse_kv_cache_snapkv_gb300 import rkv
    for c in (Case(51, [64], [9000], words=2), Case(52, [500, 3, 70], [500, 3000, 100]),
              Case(53, [1] * 80, [50] * 80), Case(54, [64] * 70, [700] * 70, n_kv=1),
              Case(55, [3], [9000]), Case(56, [32], [20000], gqa=4, words=1), Case(57, [7, 4], [9000, 3000], gqa=11)):
        need = rkv.rkv_prompt_attention_workspace_bytes(c.n, c.n_kv, c.gqa, c.tokens)
        whole = torch.randint(0, 255, (need + 4096,), dtype=torch.uint8, device="cuda")
        behind = whole[need:].clone()
        whole[:256] = 0
        out, _ = c.call(ws=whole[:need])
        rkv.rkv_check_status(whole[:need])
        c.check(out)
        assert torch.equal(whole[need:], behind)
        with pytest.raises(rkv.RkvError):
            c.call(ws=whole[:need - 1])


@pytest.mark.parametrize("what", [1, 2, 3])
@pytest.mark.parametrize("limit", [1000, 10 ** 6])
def test_waits_that_run_out(what, limit):
    """One load of block 0 is never requested: the status says so, the context stays usable, the next call is right."""
    from sparse_kv_cache_snapkv_gb300 import rkv
    c = Case(60, [700, 65], [700, 1000])
    out = torch.zeros(c.tokens, 8, D, dtype=torch.bfloat16, device="cuda")
    ws = rkv.rkv_testing_attention_wait_timeout(c.q, c.q_start, c.k, c.v, c.len, SCALE, out, what, limit)
    with pytest.raises(rkv.RkvError) as e:
        rkv.rkv_check_status(ws)
    assert e.value.bits == 4
    out, ws = c.call()
    rkv.rkv_check_status(ws)
    c.check(out)


# ------------------------------------------------------------------------------------------------ far offsets
def test_attention_offsets_past_32_bits():
    """The last rows of a cache of more than 2^32 elements, contiguous and paged."""
    from sparse_kv_cache_snapkv_gb300 import rkv
    n, n_kv, cap, T, L = 5, 8, 900000, 40, 300
    k = torch.zeros(n, n_kv, cap, D, dtype=torch.bfloat16, device="cuda")  # 4.6e9 elements each
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    kk, vv = (torch.randn(n_kv, L, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(T, 32, D, generator=g, device="cuda").bfloat16()
    k[4, :, :L], v[4, :, :L] = kk, vv
    out, ref = torch.zeros_like(q), torch.zeros_like(q)
    rkv.rkv_check_status(rkv.rkv_prompt_attention(q, _ints([0, T]), kk[None], vv[None], _ints([L]), SCALE, ref))
    rkv.rkv_check_status(rkv.rkv_prompt_attention(q, _ints([0, 0, 0, 0, 0, T]), k, v, _ints([1, 0, 5, 0, L]), SCALE, out))
    assert torch.equal(out, ref)
    block = 4096
    pools = [x.view(-1)[: (x.numel() // (n_kv * block * D)) * n_kv * block * D].view(-1, n_kv, block, D) for x in (k, v)]
    last = pools[0].shape[0] - 1
    for pool, x in zip(pools, (kk, vv)):
        pool[last, :, :L] = x
    out.zero_()
    rkv.rkv_check_status(rkv.rkv_prompt_attention_paged(q, _ints([0, T]), *pools, _ints([[last]]), _ints([L]), SCALE, out))
    assert torch.equal(out, ref)
