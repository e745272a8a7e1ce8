"""Attention of packed tokens (prompts, chunks, drafted trees) against the float64 oracle."""
import math

import numpy as np
import pytest
import torch

from oracle import serve as S
from tests import serve_parity as P

pytestmark = pytest.mark.gpu

D = 128
SCALE = 1.0 / math.sqrt(D)
SENTINEL = 768.0  # (a bf16 number)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _np(t):
    return t.double().cpu().numpy()


def tree_masks(rng, news, words):
    """A random tree for every unit: a token's bits are its ancestors and itself."""
    rows = []
    for T in news:
        sees = np.zeros((T, 32 * words), dtype=bool)
        for j in range(T):
            p = j - 1 - int(rng.integers(0, 5))
            if p >= 0:
                sees[j] = sees[p]
            sees[j, j] = True
        rows.append(sees)
    bits = np.concatenate(rows) if rows else np.zeros((0, 32 * words), dtype=bool)
    w = (bits.reshape(len(bits), words, 32).astype(np.int64) << np.arange(32)).sum(-1)
    return np.where(w >= 2 ** 31, w - 2 ** 32, w).astype(np.int32)


class Case:
    """Packed q (a slice of rows that hold k and v as well), a cache whose rows behind the lengths hold NaN."""

    def __init__(self, seed, news, lens, n_kv=2, gqa=4, cap=None, block=0, words=0, front=0, behind=0, spread=1.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        n, hq = len(news), n_kv * gqa
        self.n, self.n_kv, self.gqa, self.news, self.lens, self.block = n, n_kv, gqa, news, lens, block
        cap = self.cap = cap or max(max(lens), 1)
        self.tokens = front + sum(news) + behind
        self.starts = [front + sum(news[:u]) for u in range(n + 1)]
        self.q_start, self.len = _ints(self.starts), _ints(lens)
        qkv = (normal(self.tokens, hq + 2 * n_kv, D) * spread).bfloat16()
        self.q = qkv[:, :hq]
        sigma = torch.exp(normal(n, n_kv, 1, D))
        k = (normal(n, n_kv, cap, D) * sigma).bfloat16()
        v = normal(n, n_kv, cap, D).bfloat16()
        for u, L in enumerate(lens):
            k[u, :, L:], v[u, :, L:] = math.nan, math.inf
        self.k, self.v, self.table = k, v, None
        self.dense = (k, v)
        if block:
            most = -(-cap // block)
            self.table = torch.randperm(n * most + 3, generator=g, device="cuda")[: n * most].int().view(n, most)
            pools = []
            for x in (k, v):
                pad = torch.full((n, n_kv, most * block, D), math.nan, dtype=torch.bfloat16, device="cuda")
                pad[:, :, :cap] = x
                pool = torch.full((n * most + 3, n_kv, block, D), math.nan, dtype=torch.bfloat16, device="cuda")
                pool[self.table.flatten().long()] = pad.unflatten(2, (most, block)).transpose(1, 2).flatten(0, 1)
                pools.append(pool)
            self.k, self.v = pools
            for u, L in enumerate(lens):  # blocks behind the last are never looked at
                self.table[u, -(-L // block):] = -5
        self.mask = None
        if words:
            m = np.zeros((self.tokens, words), dtype=np.int32)
            m[front:front + sum(news)] = tree_masks(rng, news, words)
            self.mask = torch.tensor(m, device="cuda")

    def call(self, out=None, **kw):
        from sparse_kv_cache_snapkv_gb300 import rkv
        if out is None:
            out = torch.full((self.tokens, self.n_kv * self.gqa, D), SENTINEL, dtype=torch.bfloat16, device="cuda")
        args = [self.q, self.q_start] + ([self.mask] if self.mask is not None else []) + [self.k, self.v]
        name = "rkv_tree_attention" if self.mask is not None else "rkv_prompt_attention"
        if self.block:
            args, name = args + [self.table], name + "_paged"
        ws = getattr(rkv, name)(*args, self.len, SCALE, out, **kw)
        return out, ws

    def check(self, out, skipped=()):
        got = _np(out)
        mine = np.zeros(self.tokens, dtype=bool)
        for u in range(self.n):
            a, T, L = self.starts[u], self.news[u], self.lens[u]
            if u in skipped or T == 0:
                continue
            mine[a:a + T] = True
            q = _np(self.q[a:a + T])
            k, v = _np(self.dense[0][u, :, :L]), _np(self.dense[1][u, :, :L])
            sees = S.visible(T, L, None if self.mask is None else self.mask[a:a + T].cpu().numpy())
            ref, mag = S.attention(q, k, v, SCALE, sees)
            P.within(got[a:a + T], ref, P.attention_tolerance(q, k, SCALE, ref, mag), f"unit {u}")
        assert (got[~mine] == SENTINEL).all()


def _checked(case, **kw):
    from sparse_kv_cache_snapkv_gb300 import rkv
    out, ws = case.call(**kw)
    rkv.rkv_check_status(ws)
    case.check(out)


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 300, 515])
def test_prompt_lengths(T):
    _checked(Case(T, [T], [T]))


@pytest.mark.parametrize("T,L", [(1, 1), (1, 128), (1, 129), (1, 1000), (5, 127), (5, 131), (64, 640), (65, 705),
                                 (100, 3000), (1, 9000), (130, 5003)])
def test_chunk_behind_cached_rows(T, L):
    _checked(Case(T + L, [T], [L], cap=L + 13))


@pytest.mark.parametrize("gqa,n_kv", [(1, 1), (1, 3), (2, 2), (3, 2), (4, 1), (5, 2), (6, 1), (7, 1), (8, 2), (12, 1),
                                      (16, 1), (33, 1), (64, 1)])
def test_groups(gqa, n_kv):
    _checked(Case(gqa, [150, 1, 37], [150, 260, 300], n_kv=n_kv, gqa=gqa))


@pytest.mark.parametrize("block", [1, 2, 8, 16, 32, 64, 128, 256, 512])
def test_paged_blocks(block):
    _checked(Case(block, [77, 0, 130, 1], [77, 5, 613, 1025], block=block))


def test_packed_ragged_batch_between_other_rows():
    news = [0, 70, 1, 0, 300, 2, 129, 0]
    lens = [0, 70, 400, 9, 301, 2, 1000, 0]
    _checked(Case(5, news, lens, n_kv=3, gqa=2, front=7, behind=11, cap=1111))


def test_many_units():
    rng = np.random.default_rng(1)
    news = [int(x) for x in rng.integers(0, 4, 2100)]
    lens = [t + int(x) for t, x in zip(news, rng.integers(0, 40, 2100))]
    _checked(Case(6, news, lens, n_kv=1, gqa=2))


def test_more_pairs_than_plan_threads():
    # 2304 pairs of tiles of one head: several rounds of the plan, and of every CTA
    _checked(Case(7, [2304], [2304], n_kv=1, gqa=64))


def test_large_scores_raise_the_reference():
    """Scores that grow along the keys: the running reference has to move up again and again."""
    c = Case(8, [300], [1500], n_kv=1, gqa=4)
    ramp = torch.linspace(0.05, 6.0, 1500, device="cuda")[None, None, :, None]
    c.k.copy_((c.k.float() * ramp).bfloat16())
    _checked(c)


def test_equal_scores():
    c = Case(9, [64], [4000], n_kv=1, gqa=1)
    c.k[0, :, :4000] = 0.0
    _checked(c)


@pytest.mark.parametrize("T,words,L", [(1, 1, 1), (1, 1, 300), (8, 1, 1021), (31, 1, 31), (32, 1, 160), (33, 2, 161),
                                       (64, 2, 1000), (65, 3, 1000), (100, 4, 228), (128, 4, 2000), (300, 10, 900),
                                       (1024, 32, 1100)])
def test_tree(T, words, L):
    _checked(Case(T + L, [T], [L], words=words))


@pytest.mark.parametrize("block", [0, 16, 64, 256])
def test_tree_batch(block):
    _checked(Case(11, [8, 1, 0, 33, 64, 17], [1008, 1, 40, 33, 700, 130], n_kv=2, gqa=4, words=2, block=block,
                  front=3, behind=5))


@pytest.mark.parametrize("base", [0, 1, 127, 128, 500])
def test_tree_rows_that_see_nothing(base):
    """Without cached rows an empty mask leaves a row empty: zeros. Bits from T on are ignored."""
    c = Case(12 + base, [70], [base + 70], words=3)
    c.mask[5] = 0
    c.mask[64:] = 0
    c.mask[20, 2] = -64  # tokens 70 .. 95: there are none
    out, ws = c.call()
    from sparse_kv_cache_snapkv_gb300 import rkv
    rkv.rkv_check_status(ws)
    c.check(out)
    if base == 0:
        assert (out[5] == 0).all() and (out[64:70] == 0).all()


def test_tree_of_all_bits_sees_every_drafted_row():
    c = Case(13, [40], [555], words=2)
    c.mask.fill_(-1)
    _checked(c)


def test_causal_mask_as_a_tree_is_the_prompt():
    c = Case(14, [60, 20], [700, 20], words=2)
    m = np.zeros((80, 2), dtype=np.int64)
    for i in range(80):
        t = i if i < 60 else i - 60
        for w in range(2):
            m[i, w] = ((1 << (t + 1)) - 1 >> (32 * w)) & 0xFFFFFFFF
    c.mask.copy_(torch.tensor(np.where(m >= 2 ** 31, m - 2 ** 32, m).astype(np.int32)))
    tree, _ = c.call()
    c.mask = None
    causal, _ = c.call()
    assert torch.equal(tree, causal)


@pytest.mark.parametrize("news,lens", [([64], [40000]), ([8, 1], [30000, 17]), ([16, 64, 1], [20000, 9000, 12345])])
@pytest.mark.parametrize("block", [0, 64])
def test_long_caches_are_cut(news, lens, block):
    """Few pairs of tiles over long caches: every CTA takes a part, and the parts are joined."""
    _checked(Case(15, news, lens, n_kv=2, gqa=4, words=2, block=block))
    _checked(Case(16, news, lens, n_kv=2, gqa=4, block=block))


def test_cut_items_join_the_same_way_each_time():
    c = Case(17, [64, 3], [50000, 2000], n_kv=8, gqa=4)
    first, _ = c.call()
    for _ in range(5):
        again, _ = c.call()
        assert torch.equal(first, again)


def test_contiguous_and_paged_agree_bit_for_bit():
    a = Case(18, [100, 1, 64], [1000, 3000, 64])
    b = Case(18, [100, 1, 64], [1000, 3000, 64], block=64)
    b.q = a.q
    for x, y in ((a.k, b.k), (a.v, b.v)):
        for u, L in enumerate(a.lens):
            for j in range(-(-L // 64)):
                e = min(64, L - 64 * j)
                y[b.table[u, j].long(), :, :e] = x[u, :, 64 * j: 64 * j + e]
    assert torch.equal(a.call()[0], b.call()[0])


def test_bad_units_are_skipped_and_reported():
    from sparse_kv_cache_snapkv_gb300 import rkv
    news, lens = [50, 20, 30], [50, 200, 30]
    for what, bits in (("long", 1), ("negative", 1), ("few", 2), ("order", 2), ("behind", 2)):
        c = Case(19, news, lens, cap=256)
        skipped = (1,)
        if what == "long":
            c.len[1] = 257
        elif what == "negative":
            c.len[1] = -1
        elif what == "few":
            c.len[1] = 19
        elif what == "order":
            c.q_start[1], skipped = 80, (0, 1)  # unit 0: 80 tokens for 50 rows; unit 1: 80 .. 70
        else:
            c.q_start[3], skipped = 101, (2,)   # a token behind the last
        out, ws = c.call()
        with pytest.raises(rkv.RkvError) as e:
            rkv.rkv_check_status(ws)
        assert e.value.bits == bits, what
        c.check(out, skipped=skipped)


def test_tree_of_more_tokens_than_bits_is_skipped():
    from sparse_kv_cache_snapkv_gb300 import rkv
    c = Case(20, [33, 4], [50, 60], words=1 + 1)
    c.mask = c.mask[:, :1].contiguous()
    out, ws = c.call()
    with pytest.raises(rkv.RkvError) as e:
        rkv.rkv_check_status(ws)
    assert e.value.bits == 2
    c.check(out, skipped=(0,))


def test_bad_table_entries_are_reported():
    """An entry outside the pool: block 0 is read in its place, by the tokens that see it alone."""
    from sparse_kv_cache_snapkv_gb300 import rkv
    for bad in (-1, 10 ** 6):
        c = Case(21, [10, 10], [300, 200], block=64)
        c.table[0, 1] = bad
        c.k[0], c.v[0] = 0.0, 0.0
        out, ws = c.call()
        with pytest.raises(rkv.RkvError) as e:
            rkv.rkv_check_status(ws)
        assert e.value.bits == 0x10
        own = set(c.table[1, :4].tolist())
        if 0 not in own:
            got = _np(out)[10:20]
            q, k, v = _np(c.q[10:20]), _np(c.dense[0][1, :, :200]), _np(c.dense[1][1, :, :200])
            ref, mag = S.attention(q, k, v, SCALE, S.visible(10, 200))
            P.within(got, ref, P.attention_tolerance(q, k, SCALE, ref, mag), "the other unit")
