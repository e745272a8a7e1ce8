"""Measured cases of a serving step around the cache: block tables and slots reserved for a batch of requests, rotary
positions with the new rows stored by slot, causal attention of packed prompts over the cache, and attention of a tree
of drafted tokens over it.

`run` computes a case in its plain form (elementary torch operations), or, where `own` is true, calls the library.
`exact` gives the same outputs in 64 bits, written apart from the plain form.

Packed arrays are token-major, [tokens][heads][128]; unit u has the tokens q_start[u] .. q_start[u + 1] - 1. Caches are
[n][n_kv][cap][128], or pools [blocks][n_kv][block][128] with a block table [n][max_blocks]. A slot is block * rows of a
block + row (of the first kind: unit * cap + row); -1 is no place.
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
DEV = "cuda"
OPS = ("prompt_attention", "tree_attention", "rope_append", "slots")


# ----------------------------------------------------------------------------------------------- cases
def _case(name, op, **kw):
    c = {"op": op, "n": 1, "n_kv": 8, "gqa": 4, "cap": 4096, "tokens": 1, "ragged": False, "block": 0, "rot": 128,
         "interleaved": False, "far": 1, "release": False}
    assert set(kw) <= set(c)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the smallest prompt: one request of a few dozen tokens, where the call's own cost counts
        _case("prompt_short", "prompt_attention", cap=77, tokens=77),
        # one layer of a prompt of 8192
        _case("prompt_8k", "prompt_attention", cap=8192, tokens=8192),
        # a batch of prompts of different lengths, packed, on a paged cache
        _case("prompt_packed", "prompt_attention", n=16, cap=2048, tokens=2047, ragged=True, block=64),
        # chunks of prompts behind cached tokens, 8 query heads to a KV head, on a paged cache
        _case("prompt_chunks", "prompt_attention", n=3, n_kv=4, gqa=8, cap=20480, tokens=509, ragged=True, block=128),
        # the smallest tree: eight drafted tokens over a short cache
        _case("tree_short", "tree_attention", cap=1021, tokens=8),
        # a ragged batch of trees of up to 32 tokens on a paged cache
        _case("tree_batch", "tree_attention", n=32, cap=20480, tokens=32, ragged=True, block=64),
        # one long sequence: the split over the sequence has to fill the card
        _case("tree_long", "tree_attention", cap=131071, tokens=64),
        # one decode step of a batch: one new token of each request
        _case("rope_step", "rope_append", n=64, cap=4096, ragged=True, block=16),
        # the rows of a batch of prompts
        _case("rope_prompts", "rope_append", n=16, cap=4096, tokens=4095, ragged=True, block=64),
        # half of the head in the interleaved order, chunks far along a long context
        _case("rope_far", "rope_append", n=2, n_kv=4, gqa=8, cap=1500, tokens=1111, ragged=True, rot=64,
              interleaved=True, far=1000),
        # a decode step's places for 256 requests
        _case("slots_step", "slots", n=256, cap=8192, tokens=1, ragged=True, block=16),
        # places for a batch of prompts
        _case("slots_prompts", "slots", n=64, cap=40960, tokens=32768, ragged=True, block=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(OPS)
    n, n_kv, gqa = _log(rng, 1, 32), rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 8))
    ragged, block = rng.random() < 0.5, rng.choice((0, 16, 64, 128))
    if op == "prompt_attention":
        n = _log(rng, 1, 16)
        cap = _log(rng, 1, min(131072, (1 << 20) // (n * n_kv)))
        tokens = _log(rng, 1, max(1, min(cap, (1 << 30) // (n * n_kv * gqa * cap))))
        return _case(None, op, n=n, n_kv=n_kv, gqa=gqa, cap=cap, tokens=tokens, ragged=ragged, block=block)
    if op == "tree_attention":
        cap = _log(rng, 1, min(131072, (1 << 21) // (n * n_kv)))
        return _case(None, op, n=n, n_kv=n_kv, gqa=gqa, cap=cap, tokens=_log(rng, 1, min(cap, 64)), ragged=ragged,
                     block=block)
    if op == "rope_append":
        cap = _log(rng, 1, 1 << 15) // n + 1
        return _case(None, op, n=n, n_kv=n_kv, gqa=gqa, cap=cap, tokens=_log(rng, 1, cap), ragged=ragged, block=block,
                     rot=rng.choice((32, 64, 96, 128, 128)), interleaved=rng.random() < 0.5, far=rng.choice((1, 1, 100)))
    n, cap = _log(rng, 1, 1024), _log(rng, 16, 40960)
    tokens = _log(rng, 1, min(cap, max(1, (1 << 20) // n)))
    return _case(None, op, n=n, cap=cap, tokens=tokens, ragged=ragged, block=rng.choice((16, 32, 64, 128)),
                 release=rng.random() < 0.3)


def _news(case):
    """New tokens of each unit."""
    n, most = case["n"], case["tokens"]
    return [max(1, most * (u * 5 % n + 1) // n) for u in range(n)] if case["ragged"] else [most] * n


def _lens(case):
    """Tokens of each unit with its new ones: the capacity, or spread between a quarter of it and all of it."""
    n, cap = case["n"], case["cap"]
    got = [cap // 4 + (cap - cap // 4) * (u * 7 % n + 1) // n for u in range(n)] if case["ragged"] else [cap] * n
    return [max(k, t) for k, t in zip(got, _news(case))]


def _max_blocks(case):
    return -(-case["cap"] // case["block"])


def work(case):
    n, n_kv, gqa, op = case["n"], case["n_kv"], case["gqa"], case["op"]
    news, lens = _news(case), _lens(case)
    tokens = sum(news)
    if op in ("prompt_attention", "tree_attention"):
        # (each drafted token sees the cached ones and, of its tree, a path: counted as its own token)
        pairs = sum(t * (k - t) + (t * (t + 1) // 2 if op == "prompt_attention" else t) for t, k in zip(news, lens))
        return {"bytes": 512 * n_kv * (sum(lens) + gqa * tokens), "flops": 512 * pairs * n_kv * gqa}
    if op == "rope_append":
        return {"bytes": 512 * tokens * (n_kv * gqa + 2 * n_kv) + 8 * tokens,
                "flops": 3 * tokens * case["rot"] * n_kv * (gqa + 1)}
    new_blocks = sum(-(-k // case["block"]) for k in lens) - sum(-(-(k - t) // case["block"]) for t, k in zip(news, lens))
    if case["release"]:
        return {"bytes": 16 * n + 8 * new_blocks, "flops": 4 * n}
    return {"bytes": 24 * n + 8 * tokens + 8 * new_blocks, "flops": 4 * tokens}


# ----------------------------------------------------------------------------------------------- inputs
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _frequencies(rot, far):
    """base^(-2 i / rot); for long contexts the slow ones are divided by `far`, the fast ones kept, with a ramp between."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 500000.0 ** (-2 * i / rot)
    turns = 8192 * f / (2 * math.pi)  # over the context that the slow ones were made for
    keep = ((turns - 1) / (4 - 1)).clamp(0, 1)
    return (f * keep + f / far * (1 - keep)).float().to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    n, n_kv, gqa, cap, op, block = (case[k] for k in ("n", "n_kv", "gqa", "cap", "op", "block"))
    news, lens, hq = _news(case), _lens(case), n_kv * gqa
    normal = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    tokens = sum(news)
    s = {"case": dict(case), "len": _ints(lens), "new_len": _ints(news), "most": max(news)}
    s["q_start"] = torch.cat((_ints([0]), s["new_len"].cumsum(0))).int()
    if op == "slots":
        most, before = _max_blocks(case), s["len"] - s["new_len"]
        # a pool with a tenth more blocks than these requests need; which are free is a matter of history
        blocks = int(sum(-(-k // block) for k in lens) * 1.1) + 1
        perm = torch.randperm(blocks, generator=g, device=DEV).int()
        after = (s["len"] + block - 1) // block
        s["held"] = after if case["release"] else (before + block - 1) // block
        first = s["held"].cumsum(0) - s["held"]
        j = torch.arange(most, device=DEV)
        there = j < s["held"][:, None]
        at = (first[:, None] + j).clamp(max=blocks - 1)
        s["table"] = torch.where(there, perm[at], torch.full((), -1, dtype=torch.int32, device=DEV))
        used = int(s["held"].sum())
        s["free_blocks"] = torch.full((blocks,), -1, dtype=torch.int32, device=DEV)
        s["free_blocks"][: blocks - used] = perm[used:]
        s["free_count"] = _ints([blocks - used])
        s["held_out"], s["free_count_out"] = torch.zeros_like(s["held"]), torch.zeros_like(s["free_count"])
        if case["release"]:  # a third of the requests have ended, the others were cut back by some tokens
            cut = torch.rand(n, generator=g, device=DEV)
            s["len"] = torch.where(cut < 1 / 3, torch.zeros_like(s["len"]), (s["len"] * cut).int())
        else:
            s["len"] = before
            s["len_out"], s["starts"] = torch.zeros_like(before), torch.zeros_like(s["q_start"])
            room = -(-tokens // 64) * 64  # a batch padded to a multiple of 64
            s["slots"], s["positions"] = (torch.zeros(room, dtype=torch.int32, device=DEV) for _ in range(2))
        return s
    # what the projections left: queries, keys and values side by side
    sigma = torch.exp(normal(n, n_kv, 1, D))  # keys have channels of very different size
    s["qkv"] = normal(tokens, (hq + 2 * n_kv) * D).bfloat16()
    if block:
        most = _max_blocks(case)
        s["table"] = torch.randperm(n * most, generator=g, device=DEV).int().view(n, most)
    rows, blocks = (block, n * most) if block else (cap, n)
    s["k"], s["v"] = (torch.empty(blocks, n_kv, rows, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for b in range(0, blocks, 256):  # (in parts: the numbers are made in 32 bits)
        e = min(blocks, b + 256)
        s["k"][b:e], s["v"][b:e] = normal(e - b, n_kv, rows, D).bfloat16(), normal(e - b, n_kv, rows, D).bfloat16()
    if block:
        for u in range(n):
            s["k"][s["table"][u].long()] *= sigma[u].bfloat16()
    else:
        s["k"] *= sigma.bfloat16()
    s["q_out"] = torch.zeros(tokens, hq, D, dtype=torch.bfloat16, device=DEV)
    if op == "rope_append":
        unit = torch.repeat_interleave(torch.arange(n, device=DEV), s["new_len"].long())
        at = torch.arange(tokens, device=DEV) - s["q_start"][unit] + (s["len"] - s["new_len"])[unit]
        place = s["table"][unit, at // block].long() * block + at % block if block else unit * cap + at
        s["slots"] = place.int()
        s["positions"] = (at + 1000 * (case["far"] - 1)).int()
        s["inv_freq"] = _frequencies(case["rot"], case["far"])
        s["mscale"] = 0.1 * math.log(case["far"]) + 1.0
    if op == "tree_attention":
        # every token hangs on one of the few before it; a row's bits are its ancestors and itself
        most = case["tokens"]
        parent = torch.arange(most, device=DEV) - 1 - torch.randint(0, 6, (n, most), generator=g, device=DEV)
        sees = torch.zeros(n, most, -(-most // 32) * 32, dtype=torch.bool, device=DEV)
        units = torch.arange(n, device=DEV)
        for j in range(most):
            p = parent[:, j]
            sees[:, j] = sees[units, p.clamp(min=0)] & (p >= 0)[:, None]
            sees[:, j, j] = True
        bits = (sees.unflatten(-1, (-1, 32)).long() << torch.arange(32, device=DEV)).sum(-1)
        bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int()
        s["mask"] = bits[torch.arange(most, device=DEV) < s["new_len"][:, None]].contiguous()
    return s


# ----------------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if op == "slots":
        return _release(s) if s["case"]["release"] else _reserve(s)
    return _rope(s) if op == "rope_append" else _attention(s)


def _workspace(s, size):
    """The workspace that a program keeps from one call to the next."""
    if "ws" not in s:
        from sparse_kv_cache_snapkv_gb300 import rkv
        s["ws"] = rkv.workspace(size(), DEV)
    return s["ws"]


def _split(s):
    hq, n_kv = s["case"]["n_kv"] * s["case"]["gqa"], s["case"]["n_kv"]
    x = s["qkv"].unflatten(-1, (-1, D))
    return x[:, :hq], x[:, hq : hq + n_kv], x[:, hq + n_kv :]


def _reserve(s):
    block = s["case"]["block"]
    if own:
        from sparse_kv_cache_snapkv_gb300 import rkv
        rkv.rkv_reserve_slots(s["new_len"], s["len"], s["held"], s["table"], s["free_blocks"], s["free_count"], block,
                              s["starts"], s["slots"], s["positions"], s["len_out"], s["held_out"], s["free_count_out"],
                              ws=_workspace(s, lambda: rkv.rkv_reserve_slots_workspace_bytes(s["case"]["n"])))
        return [s[k] for k in ("starts", "slots", "positions", "table", "len_out", "held_out", "free_count_out")]
    length, new, held, table, free = s["len"].long(), s["new_len"].long(), s["held"].long(), s["table"], s["free_count"].long()
    start = torch.cat((torch.zeros_like(new[:1]), new.cumsum(0)))
    need = ((length + new + block - 1) // block - held).clamp(min=0)
    upto = need.cumsum(0)
    served = (need == 0) | (upto <= free)
    j = torch.arange(table.shape[1], device=DEV) - held[:, None]
    fresh = (j >= 0) & (j < need[:, None]) & served[:, None]
    source = (free - 1 - (upto - need)[:, None] - j).clamp(min=0, max=s["free_blocks"].shape[0] - 1)
    table.copy_(torch.where(fresh, s["free_blocks"][source], table))
    t = torch.arange(s["slots"].shape[0], device=DEV)
    unit = torch.searchsorted(start[1:].contiguous(), t, right=True).clamp(max=new.shape[0] - 1)
    at = length[unit] + t - start[unit]
    placed = (t < start[-1]) & served[unit]
    blocks = table[unit, (at // block).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(placed, blocks * block + at % block, -1).int()
    positions = torch.where(placed, at, 0).int()
    return [start.int(), slots, positions, table, torch.where(served, length + new, length).int(),
            torch.where(served, held + need, held).int(), (free - torch.where(served, need, 0).sum()).int()]


def _release(s):
    block = s["case"]["block"]
    if own:
        from sparse_kv_cache_snapkv_gb300 import rkv
        rkv.rkv_release_blocks(s["len"], s["held"], s["table"], s["free_blocks"], s["free_count"], block, s["held_out"],
                               s["free_count_out"],
                               ws=_workspace(s, lambda: rkv.rkv_release_blocks_workspace_bytes(s["case"]["n"])))
        return [s["free_blocks"], s["held_out"], s["free_count_out"]]
    held, table, free = s["held"].long(), s["table"], s["free_count"].long()
    keep = torch.minimum((s["len"].long() + block - 1) // block, held)
    give = held - keep
    j = torch.arange(table.shape[1], device=DEV)
    back = (j >= keep[:, None]) & (j < held[:, None])
    at = free + (give.cumsum(0) - give)[:, None] + j - keep[:, None]
    s["free_blocks"][at[back]] = table[back]
    return [s["free_blocks"], keep.int(), (free + give.sum()).int()]


def _rope(s):
    case, (q, k, v) = s["case"], _split(s)
    if own:
        from sparse_kv_cache_snapkv_gb300 import rkv
        rkv.rkv_rope_append(q, k, v, s["positions"], s["inv_freq"], s["slots"], s["q_out"], s["k"], s["v"],
                            interleaved=case["interleaved"], mscale=s["mscale"],
                            ws=_workspace(s, lambda: rkv.rkv_rope_append_workspace_bytes()))
        return [s["q_out"], s["k"], s["v"]]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = (f(angle).float()[:, None] * s["mscale"] for f in (torch.cos, torch.sin))
    half = case["rot"] // 2
    order = torch.arange(case["rot"], device=DEV)
    order = order.view(half, 2).T if case["interleaved"] else order.view(2, half)  # first and second of each pair

    def rotated(x):
        y = x.float()
        a, b = y[..., order[0]], y[..., order[1]]
        y[..., order[0]], y[..., order[1]] = a * cos - b * sin, b * cos + a * sin
        return y.bfloat16()

    rows = s["k"].shape[2]
    at = s["slots"].long()
    s["q_out"].copy_(rotated(q))
    s["k"][at // rows, :, at % rows] = rotated(k)
    s["v"][at // rows, :, at % rows] = v
    return [s["q_out"], s["k"], s["v"]]


def _attention(s):
    case, q = s["case"], _split(s)[0]
    n, n_kv, gqa, paged, tree = case["n"], case["n_kv"], case["gqa"], bool(case["block"]), case["op"] == "tree_attention"
    if own:
        from sparse_kv_cache_snapkv_gb300 import rkv
        size = lambda: rkv.rkv_prompt_attention_workspace_bytes(n, n_kv, gqa, q.shape[0])  # noqa: E731
        call = getattr(rkv, f"rkv_{case['op']}" + ("_paged" if paged else ""))
        mask, table = ((s["mask"],) if tree else ()), ((s["table"],) if paged else ())
        call(q, s["q_start"], *mask, s["k"], s["v"], *table, s["len"], SCALE, s["q_out"], ws=_workspace(s, size))
        return s["q_out"]
    flat = (lambda x: x[s["table"].long()].transpose(1, 2).flatten(2, 3)) if paged else lambda x: x  # noqa: E731
    k, v = flat(s["k"]).float(), flat(s["v"]).float()
    length, new = s["len"].long()[:, None], s["new_len"].long()[:, None]
    i, j = torch.arange(s["most"], device=DEV), torch.arange(k.shape[2], device=DEV)
    mine = i < new
    token = (s["q_start"][:-1].long()[:, None] + i).clamp(max=q.shape[0] - 1)
    x = q[token].float().unflatten(2, (n_kv, gqa)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(x, k.transpose(-1, -2)).unflatten(2, (gqa, -1))  # [n][n_kv][gqa][most][rows]
    x *= SCALE
    drafted = j - (length - new)  # [n][rows]: number among the new tokens
    if tree:
        bits = (s["mask"][token][..., None] >> torch.arange(32, device=DEV)) & 1
        bits = bits.flatten(-2)  # [n][most][32 words]
        at = drafted.clamp(min=0, max=bits.shape[-1] - 1)[:, None].expand(-1, i.shape[0], -1)
        sees = (drafted < 0)[:, None] | (bits.gather(2, at).bool() & (drafted < new)[:, None])
    else:
        sees = drafted[:, None] <= i[:, None]
    sees = sees & mine[..., None] & (j < length)[:, None]
    x.masked_fill_(~sees[:, None, None], -math.inf)
    x -= x.amax(-1, keepdim=True).clamp(min=-1e30)
    x.exp_()
    x /= x.sum(-1, keepdim=True).clamp(min=1e-30)
    v = torch.where((j < length)[:, None, :, None], v, torch.zeros((), device=DEV))
    o = torch.matmul(x.flatten(2, 3), v).unflatten(2, (gqa, -1)).permute(0, 3, 1, 2, 4).flatten(2, 3)
    s["q_out"][token[mine]] = o[mine].bfloat16()
    return s["q_out"]


# ----------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    if case["op"] == "slots":
        return None  # whole numbers
    s = prepare(case, seed)
    n, n_kv, gqa, block = case["n"], case["n_kv"], case["gqa"], case["block"]
    hq, starts = n_kv * gqa, s["q_start"].tolist()
    rows = s["qkv"].double().view(s["qkv"].shape[0], -1, D)
    out = torch.zeros(rows.shape[0], hq, D, dtype=torch.float64, device=DEV)
    if case["op"] == "rope_append":
        # each pair as a complex number, turned by its angle
        angle = s["positions"].double()[:, None] * s["inv_freq"].double()
        turn = torch.polar(torch.full_like(angle, s["mscale"]), angle)[:, None]
        rot, x = case["rot"], rows[:, : hq + n_kv]
        if case["interleaved"]:
            z = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
            y = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2 : rot].contiguous()) * turn
            y = torch.cat((z.real, z.imag), -1)
        y = torch.cat((y, x[..., rot:]), -1)
        k, v = s["k"].double(), s["v"].double()
        for t, slot in enumerate(s["slots"].tolist() if rows.shape[0] <= 4096 else ()):
            k[slot // k.shape[2], :, slot % k.shape[2]] = y[t, hq:]
            v[slot // k.shape[2], :, slot % k.shape[2]] = rows[t, hq + n_kv :]
        return [y[:, :hq], k, v] if rows.shape[0] <= 4096 else [y[:, :hq], None, None]
    for u, (length, new) in enumerate(zip(s["len"].tolist(), s["new_len"].tolist())):
        a = starts[u]
        j = torch.arange(length, device=DEV)
        for g in range(n_kv):
            if block:
                k, v = (s[m][s["table"][u].long(), g].flatten(0, 1)[:length].double() for m in "kv")
            else:
                k, v = (s[m][u, g, :length].double() for m in "kv")
            for i in range(0, new, 2048):
                e = min(new, i + 2048)
                if case["op"] == "tree_attention":
                    sees = torch.ones(e - i, length, dtype=torch.bool, device=DEV)
                    word = s["mask"][a + i : a + e].long()
                    for d in range(new):
                        sees[:, length - new + d] = (word[:, d // 32] >> (d % 32)) & 1 == 1
                else:
                    sees = j <= length - new + torch.arange(i, e, device=DEV)[:, None]
                for h in range(g * gqa, (g + 1) * gqa):
                    x = (rows[a + i : a + e, h] @ k.T) * SCALE
                    p = torch.softmax(x.masked_fill(~sees, -math.inf), -1)
                    out[a + i : a + e, h] = p @ v
    return out
