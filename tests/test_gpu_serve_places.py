"""Block tables and slots kept on the GPU, and rotary positions stored by slot, against the oracle."""
import numpy as np
import pytest
import torch

from oracle import serve as S
from tests import serve_parity as P

pytestmark = pytest.mark.gpu

D = 128


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _np(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------------------------------------ reserve, release
class Pool:
    """A pool with some blocks held by units, the others on the free stack in some order."""

    def __init__(self, seed, lens, block, max_blocks, spare, extra=None):
        rng = np.random.default_rng(seed)
        self.block, self.max_blocks, self.n = block, max_blocks, len(lens)
        self.len = list(lens)
        self.held = [-(-max(t, 0) // block) + (extra[u] if extra else 0) for u, t in enumerate(lens)]
        self.num = sum(self.held) + spare
        order = [int(x) for x in rng.permutation(self.num)]
        self.table = [[-9] * max_blocks for _ in lens]
        for u, h in enumerate(self.held):
            self.table[u][:h], order = order[:h], order[h:]
        self.count = len(order)
        self.free = order + [-3] * (self.num - len(order))

    def reserve(self, new, room, alias=False, ws=None, stream=None, fix=None):
        from sparse_kv_cache_snapkv_gb300 import rkv
        n = self.n
        t = dict(new=_ints(new), len=_ints(self.len), held=_ints(self.held), table=_ints(self.table),
                 free=_ints(self.free), count=_ints([self.count]))
        if fix:
            fix(t)
        q_start, slots, positions = (torch.full((m,), 99, dtype=torch.int32, device="cuda") for m in (n + 1, room, room))
        outs = ([t["len"], t["held"], t["count"]] if alias else
                [torch.full_like(t[k], 55) for k in ("len", "held", "count")])
        ws = rkv.rkv_reserve_slots(t["new"], t["len"], t["held"], t["table"], t["free"], t["count"], self.block, q_start,
                                   slots, positions, *outs, ws=ws, stream=stream)
        try:
            bits = rkv.rkv_check_status(ws)
        except rkv.RkvError as e:
            bits = e.bits
        got = dict(q_start=q_start, slots=slots, positions=positions, table=t["table"], len=outs[0], held=outs[1])
        got = {k: v.tolist() for k, v in got.items()}
        got["free_count"] = int(outs[2])
        assert t["free"].tolist() == self.free if not fix else True
        return got, bits

    def expect(self, new, room):
        return S.reserve(new, self.len, self.held, self.table, self.free, self.count, self.block, room)


def _same(pool, new, room, bits=0, **kw):
    got, b = pool.reserve(new, room, **kw)
    want, wb = pool.expect(new, room)
    assert got == want
    assert b == wb == bits


@pytest.mark.parametrize("block", [1, 3, 16, 64])
@pytest.mark.parametrize("alias", [False, True])
def test_reserve(block, alias):
    lens = [0, 1, block, block + 1, 5 * block, 100, 37]
    new = [5, 0, 1, block - 1, 0, 33, 3 * block + 1]
    _same(Pool(block, lens, block, 200, 400), new, sum(new) + 9, alias=alias)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 1000, 1024, 1025, 3000])
def test_reserve_one_token_of_each(n):
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, 70, n)]
    _same(Pool(n, lens, 16, 8, n), [1] * n, n)


@pytest.mark.parametrize("room", [8192, 8193, 30000])
def test_reserve_prompts(room):
    """Both sides of the size from which a second kernel places the tokens."""
    new = [0, 4000, 1, 2500, 0, 1600, 0]
    lens = [10, 0, 64, 100, 0, 5000, 0]
    _same(Pool(3, lens, 64, 128, 300), new, room)


def test_reserve_uses_held_blocks_first():
    lens = [10, 0, 40]
    _same(Pool(4, lens, 16, 32, 20, extra=[3, 2, 0]), [70, 33, 1], 120)


def test_reserve_nothing():
    _same(Pool(5, [3, 0], 16, 4, 0), [0, 0], 7)


def test_reserve_without_enough_blocks():
    # 6 free: the first needs 4, the second 3 (not served), the third 1 (counted behind it: not served), the fourth none
    _same(Pool(6, [0, 0, 16, 17], 16, 8, 6), [64, 48, 1, 2], 200, bits=0x20)


def test_reserve_the_last_block():
    _same(Pool(7, [0, 5], 16, 8, 3), [48, 11], 59)


@pytest.mark.parametrize("new,bits", [([5, -1, 3], 1), ([5, 2 ** 31 - 1, 3], 1), ([5, 200, 3], 1), ([60, 60, 10], 1)])
def test_reserve_refuses_units(new, bits):
    """A negative count, sums past 31 bits, more than a unit's table, more tokens than there is room for."""
    _same(Pool(8, [1, 2, 3], 16, 8, 40), new, 100, bits=bits)


def test_reserve_with_bad_state():
    p = Pool(9, [1, 2, 3], 16, 8, 40)
    p.len[1] = -4
    _same(p, [1, 1, 1], 3, bits=1)
    p = Pool(9, [1, 2, 3], 16, 8, 40)
    p.held[2] = 9
    _same(p, [1, 1, 1], 3, bits=1)
    p = Pool(9, [1, 20, 3], 16, 8, 40)
    p.held[1] = 1  # 20 tokens need two blocks
    _same(p, [1, 1, 1], 3, bits=0x10)
    p = Pool(9, [1, 20, 3], 16, 8, 40)
    p.table[1][1] = p.num
    _same(p, [1, 1, 1], 3, bits=0x10)
    p = Pool(9, [1, 16, 3], 16, 8, 40)
    p.free[p.count - 1] = -1
    _same(p, [1, 20, 1], 30, bits=0x10)
    for count in (-1, 10 ** 6):
        p = Pool(9, [1, 16, 3], 16, 8, 40)
        p.count = count
        _same(p, [1, 1, 1], 3, bits=0x30)


def _release(p, length, alias=False):
    from sparse_kv_cache_snapkv_gb300 import rkv
    held, count, free, table = _ints(p.held), _ints([p.count]), _ints(p.free), _ints(p.table)
    h, c = (held, count) if alias else (torch.full_like(held, 55), torch.full_like(count, 55))
    ws = rkv.rkv_release_blocks(_ints(length), held, table, free, count, p.block, h, c)
    try:
        bits = rkv.rkv_check_status(ws)
    except rkv.RkvError as e:
        bits = e.bits
    assert table.tolist() == p.table
    return dict(free_blocks=free.tolist(), held=h.tolist(), free_count=int(c)), bits


@pytest.mark.parametrize("n,max_blocks", [(1, 8), (7, 16), (33, 16), (1025, 7), (1025, 9), (3000, 20)])
@pytest.mark.parametrize("alias", [False, True])
def test_release(n, max_blocks, alias):
    rng = np.random.default_rng(n)
    p = Pool(n, [int(x) for x in rng.integers(0, 16 * max_blocks + 1, n)], 16, max_blocks, 5)
    length = [int(t * f) for t, f in zip(p.len, rng.choice([0.0, 0.4, 1.0, 2.0], n))]
    got, bits = _release(p, length, alias)
    want, wb = S.release(length, p.held, p.table, p.free, p.count, 16)
    assert got == want and bits == wb == 0


def test_release_with_bad_state():
    for change, length, bits in ((None, [0, -1, 5], 1), ("held", [0, 0, 0], 1), ("count", [0, 0, 0], 0x10),
                                 ("negative", [0, 0, 0], 0x10), ("entry", [0, 0, 0], 0x10)):
        p = Pool(10, [40, 50, 60], 16, 8, 3)
        if change == "held":
            p.held[1] = 9
        elif change == "count":
            p.count += 1  # one block more than there is
        elif change == "negative":
            p.count = -2
        elif change == "entry":
            p.table[0][0] = 1000
        got, b = _release(p, length)
        want, wb = S.release(length, p.held, p.table, p.free, p.count, 16)
        assert got == want and b == wb == bits, change


def test_blocks_go_round():
    """Requests come, grow, are cut and end; no block is ever held twice, and all come back."""
    from sparse_kv_cache_snapkv_gb300 import rkv
    rng = np.random.default_rng(11)
    n, block, most, num = 20, 16, 12, 150
    length, held, count = _ints([0] * n), _ints([0] * n), _ints([num])
    table, free = torch.full((n, most), -1, dtype=torch.int32, device="cuda"), _ints(list(rng.permutation(num)))
    q_start, slots, positions = _ints([0] * (n + 1)), _ints([0] * 600), _ints([0] * 600)
    ws = rkv.workspace(rkv.rkv_reserve_slots_workspace_bytes(n), "cuda")
    for step in range(60):
        add = [int(x) if t + x <= most * block else 0 for x, t in zip(rng.choice([0, 1, 1, 20], n), length.tolist())]
        rkv.rkv_reserve_slots(_ints(add), length, held, table, free, count, block, q_start, slots, positions, length, held,
                              count, ws=ws)
        try:
            rkv.rkv_check_status(ws)
        except rkv.RkvError as e:
            assert e.bits == 0x20
        if step % 3 == 2:
            cut = torch.tensor(rng.choice([0.0, 0.5, 1.0], n), device="cuda")
            length.copy_((length * cut).int())
            rkv.rkv_release_blocks(length, held, table, free, count, block, held, count, ws=ws)
            rkv.rkv_check_status(ws)
        owned = [b for u, h in enumerate(held.tolist()) for b in table[u, :h].tolist()]
        assert sorted(owned + free[: int(count)].tolist()) == list(range(num))
    length.zero_()
    rkv.rkv_release_blocks(length, held, table, free, count, block, held, count, ws=ws)
    assert int(count) == num and sorted(free.tolist()) == list(range(num))


# ------------------------------------------------------------------------------------------------ rotary positions
def _rope(seed, tokens, hq, n_kv, rot=128, interleaved=False, mscale=1.0, block=16, blocks=None, positions=None,
          slots=None, inplace=False, base=10000.0, fused=True):
    from sparse_kv_cache_snapkv_gb300 import rkv
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    blocks = blocks or -(-tokens // block) + 2
    if fused:
        x = normal(tokens, hq + 2 * n_kv, D)
        q, k, v = x[:, :hq], x[:, hq:hq + n_kv], x[:, hq + n_kv:]
    else:
        q, k, v = normal(tokens, hq, D), normal(tokens, n_kv, D), normal(tokens, n_kv, D)
    if positions is None:
        positions = torch.randint(0, 100000, (tokens,), generator=g, device="cuda").tolist()
    if slots is None:
        slots = torch.randperm(blocks * block, generator=g, device="cuda")[:tokens].tolist()
    freq, _ = rkv.rkv_rope_frequencies(rot, base)
    kc, vc = normal(blocks, n_kv, block, D), normal(blocks, n_kv, block, D)
    q64, k64, v64, kw, vw = _np(q), _np(k), _np(v), _np(kc), _np(vc)
    q_out = q if inplace else torch.full((tokens, hq, D), 777.0, dtype=torch.bfloat16, device="cuda")
    before = _np(q_out)
    ws = rkv.rkv_rope_append(q, k, v, _ints(positions), freq.cuda(), _ints(slots), q_out, kc, vc, interleaved=interleaved,
                             mscale=mscale)
    try:
        bits = rkv.rkv_check_status(ws)
    except rkv.RkvError as e:
        bits = e.bits
    f = freq.double().numpy()
    there = np.array([0 <= s < blocks * block for s in slots])
    refq, refk = S.turn(q64, positions, f, interleaved, mscale), S.turn(k64, positions, f, interleaved, mscale)
    tolq, tolk = (P.turn_tolerance(x, positions, f, interleaved, mscale, r) for x, r in ((q64, refq), (k64, refk)))
    got = _np(q_out)
    P.within(got[there], refq[there], tolq[there], "q")
    assert (got[~there] == before[~there]).all()
    kg, vg = _np(kc), _np(vc)
    ktol = np.zeros(kw.shape)
    for t in np.flatnonzero(there):
        b, r = divmod(slots[t], block)
        kw[b, :, r], ktol[b, :, r], vw[b, :, r] = refk[t], tolk[t], v64[t]
    P.within(kg, kw, ktol, "k")
    assert (vg == vw).all()
    return bits


@pytest.mark.parametrize("tokens", [1, 2, 7, 64, 333, 5000])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(tokens, interleaved):
    assert _rope(tokens, tokens, 8, 2, interleaved=interleaved) == 0


@pytest.mark.parametrize("rot", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_of_part_of_the_head(rot, interleaved):
    assert _rope(rot, 37, 4, 2, rot=rot, interleaved=interleaved, mscale=1.25) == 0


@pytest.mark.parametrize("hq,n_kv", [(1, 1), (3, 1), (5, 2), (32, 8), (64, 1), (7, 7), (130, 3)])
def test_rope_heads(hq, n_kv):
    assert _rope(hq, 21, hq, n_kv) == 0
    assert _rope(hq, 21, hq, n_kv, fused=False) == 0


@pytest.mark.parametrize("block", [1, 3, 64, 1000])
def test_rope_blocks(block):
    """Any number of rows in a block: a contiguous cache is one with blocks of its capacity."""
    assert _rope(block, 50, 4, 2, block=block) == 0


def test_rope_of_far_and_negative_positions():
    far = [0, 1, -1, 2 ** 20, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321]
    for interleaved in (False, True):
        assert _rope(1, len(far), 4, 2, positions=far, interleaved=interleaved) == 0


def test_rope_in_place():
    assert _rope(2, 100, 8, 2, inplace=True, fused=False) == 0


def test_rope_leaves_out_tokens_without_a_place():
    slots = [5, -1, 40, -2 ** 31, 0, 47]
    assert _rope(3, 6, 4, 2, slots=slots, blocks=3) == 0
    assert _rope(3, 6, 4, 2, slots=[5, 48, 40, 2 ** 31 - 1, 0, 47], blocks=3) == 0x10


def test_rope_many_tokens_fill_the_card():
    assert _rope(4, 40000, 4, 1, block=64) == 0


def test_rope_offsets_past_32_bits():
    """A pool of more than 2^32 elements: rows at its end."""
    from sparse_kv_cache_snapkv_gb300 import rkv
    n_kv, block, blocks = 8, 1024, 4200  # 4.4e9 elements
    kc = torch.zeros(blocks, n_kv, block, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    x = torch.randn(3, 12, D, device="cuda").bfloat16()
    slots = [blocks * block - 1, 4100 * block + 5, 0]
    out = torch.zeros(3, 4, D, dtype=torch.bfloat16, device="cuda")
    freq, _ = rkv.rkv_rope_frequencies()
    x = torch.cat((x, torch.randn(3, 8, D, device="cuda").bfloat16()), 1)
    rkv.rkv_check_status(rkv.rkv_rope_append(x[:, :4], x[:, 4:12], x[:, 12:20], _ints([0, 0, 0]), freq.cuda(),
                                             _ints(slots), out, kc, vc))
    for t, s in enumerate(slots):
        assert torch.equal(kc[s // block, :, s % block], x[t, 4:12])  # position 0: as they are
        assert torch.equal(vc[s // block, :, s % block], x[t, 12:20])
    assert int((kc != 0).any(-1).sum()) == 24
