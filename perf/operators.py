"""Measured cases of the cache operators: a cache held in 4 bits (append, decode), decode steps and prompts that
accumulate each cached token's attention weight, and eviction by that weight.

`run` computes a case in its plain form (elementary torch operations in 32 bits), or, where `own` is true, calls
the library. `exact` gives the same outputs in 64 bits, written apart from the plain form.

Layouts (head_dim 128): caches [n][n_kv][cap][...]; a 4-bit row is 64 bytes of e2m1 codes (dimension 2 j in the low
half of byte j) and 8 ue5m3 scale bytes, one for 16 dimensions (byte b stands for the fp16 number with bits b << 7).
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
DEV = "cuda"
OPS = ("kv4_append", "kv4_decode", "dense_decode_weights", "prompt_weights", "evict")
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # e2m1
MAX_SCALE_BYTE = 226  # 10240: six times it is the largest fp16-representable product of a code and a scale
MAX_VALUE = 61440.0


# ----------------------------------------------------------------------------------------------- cases
def _case(name, op, **kw):
    c = {"op": op, "n": 1, "n_kv": 8, "gqa": 4, "cap": 4096, "ragged": False, "tokens": 0, "append": False,
         "weights": False, "block": 0, "keep": 0, "recent": 0, "kv4": False}
    assert set(kw) <= set(c)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a prompt of one layer of a batch goes to the 4-bit cache, ragged, with the values it stands for handed
        # back for the prompt's own attention
        _case("append_prompts", "kv4_append", n=16, cap=8192, tokens=8190, ragged=True),
        # one decode step's new token of every layer and sequence: a latency-bound call
        _case("append_token", "kv4_append", n=64, cap=2048, tokens=1, ragged=True),
        # the smallest decode call: one layer, one sequence, a short cache
        _case("kv4_short", "kv4_decode", cap=1021),
        # a batch of 32 units with 32K tokens each; the step appends its token and accumulates weights
        _case("kv4_batch_32k", "kv4_decode", n=32, cap=32768, append=True, weights=True),
        # a serving engine's ragged batch on a paged cache, 8 query heads to a KV head
        _case("kv4_paged_ragged", "kv4_decode", n=16, n_kv=4, gqa=8, cap=20480, ragged=True, block=64, append=True),
        # one long sequence: the split over the sequence has to fill the card
        _case("kv4_long", "kv4_decode", cap=131071, weights=True),
        # one layer of a small model at 4K
        _case("dense_small", "dense_decode_weights", n_kv=2, cap=4096, weights=True),
        # a ragged batch up to 32K tokens in bf16
        _case("dense_ragged", "dense_decode_weights", n=16, cap=32768, ragged=True, weights=True),
        # the prompt of one layer: every query against every key before it
        _case("prompt_8k", "prompt_weights", cap=8192, tokens=8192),
        # a chunk of a prompt behind cached tokens, ragged, two sequences
        _case("prompt_chunk", "prompt_weights", n=2, n_kv=2, cap=2500, tokens=509, ragged=True),
        # a 4096-row budget that decode steps have outgrown by 256, every layer of a 32-layer model
        _case("evict_steps", "evict", n=32, cap=4352, keep=4096, recent=256),
        # a prompt shrunk to a budget, in the 4-bit cache
        _case("evict_prompt_kv4", "evict", n=4, cap=32768, keep=4096, recent=512, kv4=True, ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(OPS)
    n, n_kv, gqa = _log(rng, 1, 32), rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 4, 8))
    ragged = rng.random() < 0.5
    rows = lambda most: _log(rng, 1, max(1, min(131072, most // (n * n_kv))))  # noqa: E731
    if op == "kv4_append":
        cap = rows(1 << 20)
        return _case(None, op, n=n, n_kv=n_kv, cap=cap, tokens=_log(rng, 1, cap), ragged=ragged)
    if op == "kv4_decode":
        return _case(None, op, n=n, n_kv=n_kv, gqa=gqa, cap=rows(1 << 23), ragged=ragged, append=rng.random() < 0.5,
                     weights=rng.random() < 0.5, block=rng.choice((0, 0, 16, 128)))
    if op == "dense_decode_weights":
        return _case(None, op, n=n, n_kv=n_kv, gqa=gqa, cap=rows(1 << 21), ragged=ragged, weights=True)
    if op == "prompt_weights":
        n = _log(rng, 1, 4)
        cap = _log(rng, 1, int(math.sqrt((1 << 31) // (n * n_kv * gqa))))
        return _case(None, op, n=n, n_kv=n_kv, gqa=gqa, cap=cap, tokens=_log(rng, 1, cap), ragged=ragged)
    cap = max(2, rows(1 << 20))
    keep = _log(rng, 1, cap - 1)
    return _case(None, op, n=n, n_kv=n_kv, cap=cap, keep=keep, recent=rng.randint(0, keep), kv4=rng.random() < 0.5,
                 ragged=ragged)


def _lens(case):
    """Rows in the cache of each unit before the call: full, or spread between a quarter of the capacity and all of it."""
    n, room = case["n"], case["tokens"] if case["op"] == "kv4_append" else 1 if case["append"] else 0
    top = max(0, case["cap"] - room)
    if not case["ragged"]:
        return [top] * n
    low = top // 4 if case["op"] != "evict" else min(top, case["keep"] // 2)
    return [low + (top - low) * (u * 7 % n + 1) // n for u in range(n)]


def _news(case):
    """New tokens (append) or queries (prompt) of each unit."""
    n, most = case["n"], case["tokens"]
    if not case["ragged"]:
        return [most] * n
    got = [max(1, most * (u * 5 % n + 1) // n) for u in range(n)]
    return [min(t, k) for t, k in zip(got, _lens(case))] if case["op"] == "prompt_weights" else got


def work(case):
    n_kv, gqa, lens = case["n_kv"], case["gqa"], _lens(case)
    heads = case["n"] * n_kv
    if case["op"] == "kv4_append":
        rows = n_kv * sum(_news(case))
        return {"bytes": rows * (512 + 144 + 512), "flops": rows * 256 * 3}
    if case["op"] == "kv4_decode":
        rows = n_kv * (sum(lens) + (case["n"] if case["append"] else 0))
        extra = heads * (512 + 144) if case["append"] else 0
        return {"bytes": rows * (144 + (8 if case["weights"] else 0)) + extra + heads * gqa * 512, "flops": rows * 512 * gqa}
    if case["op"] == "dense_decode_weights":
        rows = n_kv * sum(lens)
        return {"bytes": rows * (512 + 8) + heads * gqa * 512, "flops": rows * 512 * gqa}
    if case["op"] == "prompt_weights":
        news = _news(case)
        pairs = sum(t * (k - t) + t * (t + 1) // 2 for t, k in zip(news, lens))
        keys = n_kv * sum(lens)
        return {"bytes": keys * (256 + 8) + n_kv * gqa * sum(news) * 256, "flops": 256 * pairs * n_kv * gqa}
    keep, row = case["keep"], 144 if case["kv4"] else 512
    total = moved = 0
    for k in lens:
        total += k * 8 + min(k, keep) * 8
        if k > keep:  # about as many rows below `keep` lose their place as the share that goes
            moved += keep * (k - keep) // k
    return {"bytes": n_kv * (total + moved * 2 * row), "flops": n_kv * sum(lens)}


# ----------------------------------------------------------------------------------------------- inputs
def _table():
    """The numbers that the scale bytes 0 .. MAX_SCALE_BYTE stand for (exact in 32 bits)."""
    b = torch.arange(MAX_SCALE_BYTE + 1, device=DEV)
    e, m = b // 8, (b % 8).float()
    return torch.where(e == 0, m * 2.0 ** -17, (8 + m) * torch.exp2((e - 18).float()))


def _quantise(x):
    """[.., 128] -> codes [.., 64] and scales [.., 8], uint8. Comparisons of numbers of few bits, exact in 32."""
    x = x.float()
    x = torch.where(x == x, x, torch.zeros((), device=x.device)).clamp(-MAX_VALUE, MAX_VALUE)
    a = x.abs().unflatten(-1, (8, 16))
    table = _table()
    mids = (table[1:] + table[:-1]) * 3.0  # six times the midpoints of neighbouring scales
    amax = a.amax(-1)
    b = torch.bucketize(amax, mids)
    at = mids[b.clamp(max=MAX_SCALE_BYTE - 1)]
    b = b + ((amax == at) & (b % 2 == 1) & (b < MAX_SCALE_BYTE))  # a tie goes to the even byte
    s = table[b].unsqueeze(-1)
    code = ((a > 0.25 * s).int() + (a >= 0.75 * s).int() + (a > 1.25 * s).int() + (a >= 1.75 * s).int()
            + (a > 2.5 * s).int() + (a >= 3.5 * s).int() + (a > 5.0 * s).int())
    code = torch.where(s > 0, code, torch.zeros_like(code)).flatten(-2) + 8 * torch.signbit(x).int()
    codes = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
    return codes.contiguous(), b.to(torch.uint8).contiguous()


def _values(codes, scales):
    """[.., 64] codes and [.., 8] scales -> [.., 128] in 32 bits (exact)."""
    lut = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    table = torch.cat((_table(), torch.zeros(256 - MAX_SCALE_BYTE - 1, device=codes.device)))
    return (lut[pair.int()].unflatten(-1, (8, 16)) * table[scales.int()].unsqueeze(-1)).flatten(-2)


def _pools(case, x, table):
    """[n][n_kv][cap][w] -> a pool [blocks][n_kv][block][w] whose blocks are in the order of `table`."""
    n, n_kv, cap, w = x.shape
    block, most = case["block"], table.shape[1]
    pad = torch.zeros(n, n_kv, most * block, w, dtype=x.dtype, device=x.device)
    pad[:, :, :cap] = x
    pool = torch.empty(n * most, n_kv, block, w, dtype=x.dtype, device=x.device)
    pool[table.flatten().long()] = pad.unflatten(2, (most, block)).transpose(1, 2).flatten(0, 1)
    return pool


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    n, n_kv, gqa, cap, op = case["n"], case["n_kv"], case["gqa"], case["cap"], case["op"]
    normal = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    s = {"case": dict(case), "len": _ints(_lens(case))}
    sigma = torch.exp(normal(n, n_kv, 1, D))  # keys have channels of very different size
    rows = lambda u, t: ((normal(n_kv, t, D) * sigma[u]).bfloat16(), normal(n_kv, t, D).bfloat16())  # noqa: E731

    if op in ("kv4_decode", "kv4_append") or case["kv4"]:
        for k, w in (("k_codes", 64), ("k_scales", 8), ("v_codes", 64), ("v_scales", 8)):
            s[k] = torch.zeros(n, n_kv, cap, w, dtype=torch.uint8, device=DEV)
        if op != "kv4_append":
            for u in range(n):
                k, v = rows(u, cap)
                s["k_codes"][u], s["k_scales"][u] = _quantise(k)
                s["v_codes"][u], s["v_scales"][u] = _quantise(v)
    else:
        s["k"] = torch.empty(n, n_kv, cap, D, dtype=torch.bfloat16, device=DEV)
        s["v"] = torch.empty_like(s["k"])
        for u in range(n):
            s["k"][u], s["v"][u] = rows(u, cap)

    if op == "kv4_append":
        t = case["tokens"]
        s["new_len"] = _ints(_news(case))
        s["new_k"] = (normal(n, n_kv, t, D) * sigma).bfloat16()
        s["new_v"] = normal(n, n_kv, t, D).bfloat16()
        s["k_values"], s["v_values"] = torch.zeros_like(s["new_k"]), torch.zeros_like(s["new_v"])
        s["len_out"] = torch.zeros_like(s["len"])
    if op in ("kv4_decode", "dense_decode_weights"):
        s["q"] = normal(n, n_kv * gqa, D).bfloat16()
        s["out"] = torch.zeros_like(s["q"])
        s["new_k"] = s["new_v"] = s["len_out"] = None
        if case["append"]:
            s["new_k"] = (normal(n, n_kv, D) * sigma[:, :, 0]).bfloat16()
            s["new_v"] = normal(n, n_kv, D).bfloat16()
            s["len_out"] = torch.zeros_like(s["len"])
    room = cap
    if case["block"]:
        most = -(-cap // case["block"])
        room = most * case["block"]
        s["table"] = torch.randperm(n * most, generator=g, device=DEV).int().view(n, most)
        for k in ("k_codes", "k_scales", "v_codes", "v_scales"):
            s[k] = _pools(case, s[k], s["table"])
    if op == "prompt_weights":
        s["q"] = normal(n, n_kv * gqa, case["tokens"], D).bfloat16()
        s["q_len"] = _ints(_news(case))
        del s["v"]
    s["weights"] = None
    if case["weights"] or op in ("prompt_weights", "evict"):  # rows past a sequence hold zero
        # what was accumulated before: a long history for an eviction, the queries of a few tokens for the others (a
        # prompt's or chunk's own rows have none yet)
        before = s["len"] - s["q_len"] if op == "prompt_weights" else s["len"]
        held = torch.arange(room, device=DEV) < before[:, None, None]
        few = 1.0 if op == "evict" else gqa / before.clamp(min=1).float()[:, None, None]
        s["weights"] = torch.where(held, torch.exp(2.0 * normal(n, n_kv, room)) * few, torch.zeros((), device=DEV))
    if op == "evict":
        # rows kept by an earlier eviction know their positions; those appended since do not (-1)
        known = min(case["keep"], cap)
        s["seen"] = s["len"] + 1000
        first = torch.rand(n, n_kv, known + 1000, generator=g, device=DEV).argsort(-1)[..., :known]
        s["pos"] = torch.full((n, n_kv, cap), -1, dtype=torch.int32, device=DEV)
        s["pos"][..., :known] = first.int()
        over = (s["len"] > case["keep"])[:, None, None] & (torch.arange(cap, device=DEV) < known)
        s["pos"] = torch.where(over, s["pos"], torch.full_like(s["pos"], -1))
        s["len_out"] = torch.zeros_like(s["len"])
        s["weights_out"], s["pos_out"] = torch.zeros_like(s["weights"]), torch.full_like(s["pos"], -1)
        s["src_rows"] = torch.zeros(n, n_kv, case["keep"], dtype=torch.int32, device=DEV)
    if own:
        from sparse_kv_cache_snapkv_gb300 import rkv
        size = {"kv4_append": lambda: rkv.rkv_kv4_append_workspace_bytes(n),
                "kv4_decode": lambda: rkv.rkv_kv4_decode_workspace_bytes(n, n_kv, gqa, room, s["weights"] is not None),
                "dense_decode_weights": lambda: rkv.rkv_dense_decode_weights_workspace_bytes(n, n_kv, gqa, cap),
                "prompt_weights": lambda: rkv.rkv_prompt_weights_workspace_bytes(n, n_kv, gqa, case["tokens"], cap),
                "evict": lambda: rkv.rkv_evict_workspace_bytes(n, n_kv, cap, case["keep"])}[op]()
        s["ws"] = rkv.workspace(size, DEV)
    return s


# ----------------------------------------------------------------------------------------------- one pass
def run(s):
    return {"kv4_append": _append, "kv4_decode": _decode, "dense_decode_weights": _decode, "prompt_weights": _prompt,
            "evict": _evict}[s["case"]["op"]](s)


def _append(s):
    if own:
        from sparse_kv_cache_snapkv_gb300 import rkv
        rkv.rkv_kv4_append(s["new_k"], s["new_v"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["len"],
                           s["len_out"], new_len=s["new_len"], k_values=s["k_values"], v_values=s["v_values"], ws=s["ws"])
        return {"k_values": s["k_values"], "v_values": s["v_values"], "len": s["len_out"]}
    t = torch.arange(s["new_k"].shape[2], device=DEV)
    new = t < s["new_len"][:, None]
    u, j = new.nonzero(as_tuple=True)
    at = s["len"][u] + j
    for name in ("k", "v"):
        codes, scales = _quantise(s["new_" + name][u, :, j])
        s[name + "_codes"][u, :, at] = codes
        s[name + "_scales"][u, :, at] = scales
        s[name + "_values"][u, :, j] = _values(codes, scales).bfloat16()
    return {"k_values": s["k_values"], "v_values": s["v_values"], "len": s["len"] + s["new_len"]}


def _attend(q, k, v, length):
    """softmax(scale q k^T) v over the first `length` rows, and the probabilities; all in 32 bits."""
    n, n_kv, cap, _ = k.shape
    there = torch.arange(cap, device=DEV) < length[:, None]
    x = torch.matmul(q.float().view(n, n_kv, -1, D), k.transpose(-1, -2)) * SCALE
    x = torch.where(there[:, None, None], x, torch.full((), -math.inf, device=DEV))
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p, torch.where(there[:, None, :, None], v, torch.zeros((), device=DEV)))
    return o.reshape(n, -1, D), p.sum(2)


def _decode(s):
    case = s["case"]
    if own:
        from sparse_kv_cache_snapkv_gb300 import rkv
        if case["op"] == "dense_decode_weights":
            rkv.rkv_dense_decode_weights(s["q"], s["k"], s["v"], s["len"], SCALE, s["out"], s["weights"], ws=s["ws"])
        elif case["block"]:
            rkv.rkv_kv4_decode_paged(s["q"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["table"], s["len"],
                                     SCALE, s["out"], new_k=s["new_k"], new_v=s["new_v"], length_out=s["len_out"],
                                     weights=s["weights"], ws=s["ws"])
        else:
            rkv.rkv_kv4_decode(s["q"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["len"], SCALE, s["out"],
                               new_k=s["new_k"], new_v=s["new_v"], length_out=s["len_out"], weights=s["weights"], ws=s["ws"])
        return [x for x in (s["out"], s["weights"], s["len_out"]) if x is not None]
    length = s["len"]
    units = torch.arange(case["n"], device=DEV)
    if case["append"]:
        at = s["len"].long()
        for name in ("k", "v"):
            codes, scales = _quantise(s["new_" + name])
            for field, x in (("_codes", codes), ("_scales", scales)):
                if case["block"]:
                    s[name + field][s["table"][units, at // case["block"]].long(), :, at % case["block"]] = x
                else:
                    s[name + field][units, :, at] = x
        length = length + 1
    if case["op"] == "dense_decode_weights":
        k, v = s["k"].float(), s["v"].float()
    else:
        flat = (lambda x: x[s["table"].long()].transpose(1, 2).flatten(2, 3)) if case["block"] else lambda x: x  # noqa: E731
        k = _values(flat(s["k_codes"]), flat(s["k_scales"]))
        v = _values(flat(s["v_codes"]), flat(s["v_scales"]))
    out, w = _attend(s["q"], k, v, length)
    s["out"].copy_(out)
    if s["weights"] is not None:
        s["weights"] += w
    return [x for x in (s["out"], s["weights"], length if case["append"] else None) if x is not None]


def _prompt(s):
    if own:
        from sparse_kv_cache_snapkv_gb300 import rkv
        rkv.rkv_prompt_weights(s["q"], s["q_len"], s["k"], s["len"], SCALE, s["weights"], ws=s["ws"])
        return s["weights"]
    n, n_kv, cap, _ = s["k"].shape
    t = s["q"].shape[2]
    x = torch.matmul(s["q"].float().view(n, n_kv, -1, D), s["k"].float().transpose(-1, -2)).view(n, n_kv, -1, t, cap)
    x *= SCALE
    i, j = torch.arange(t, device=DEV)[:, None], torch.arange(cap, device=DEV)
    last = (s["len"] - s["q_len"])[:, None, None] + i
    seen = (j <= last) & (i < s["q_len"][:, None, None])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    x -= x.amax(-1, keepdim=True).clamp(min=-1e30)
    x.exp_()
    x /= x.sum(-1, keepdim=True).clamp(min=1e-30)
    s["weights"] += x.sum((2, 3))
    return s["weights"]


def _evict(s):
    names = ("k_codes", "k_scales", "v_codes", "v_scales") if s["case"]["kv4"] else ("k", "v")
    keep, recent = s["case"]["keep"], s["case"]["recent"]
    if own:
        from sparse_kv_cache_snapkv_gb300 import rkv
        call = rkv.rkv_evict_kv4 if s["case"]["kv4"] else rkv.rkv_evict
        call(*[s[m] for m in names], s["len"], s["weights"], s["pos"], s["seen"], keep, recent, s["len_out"],
             s["weights_out"], s["pos_out"], src_rows=s["src_rows"], ws=s["ws"])
        return [s[m] for m in names] + [s["len_out"], s["weights_out"], s["pos_out"], s["src_rows"]]
    n, n_kv, cap = s["weights"].shape
    row = torch.arange(cap, device=DEV)
    length, seen = s["len"][:, None, None], s["seen"][:, None, None]
    held, over = row < length, length > keep
    pos = torch.where(s["pos"] >= 0, s["pos"], seen - (length - row).int())
    inf = torch.full((), math.inf, device=DEV)
    key = torch.where(held & (pos >= seen - recent), inf, torch.where(held, s["weights"], -inf))
    order = key.sort(dim=-1, descending=True, stable=True).indices
    chosen = torch.zeros(n, n_kv, cap, dtype=torch.bool, device=DEV).scatter_(2, order[..., :keep], True)
    free = ~chosen[..., :keep]
    movers = torch.where(chosen & (row >= keep), row, cap).sort(-1).values[..., :keep]
    movers = movers.gather(2, (free.cumsum(-1) - 1).clamp(min=0, max=movers.shape[-1] - 1))
    src = torch.where(over, torch.where(free, movers, row[:keep]), row[:keep])
    src_rows = torch.where(src < torch.minimum(length, torch.full_like(length, keep)), src, -1)
    src_rows = torch.where(over, src, src_rows).int()
    src = src.clamp(max=cap - 1)
    # eviction moves rows as they are; a 4-bit row's bytes come back as bytes
    moved = []
    for m in names:
        x = s[m].clone()
        x[:, :, :keep] = s[m].gather(2, src[..., None].expand(-1, -1, -1, x.shape[-1]))
        moved.append(x)
    weights, pos_out = s["weights_out"].clone(), s["pos_out"].clone()
    weights[..., :keep] = torch.where(held[..., :keep], s["weights"].gather(2, src), weights[..., :keep])
    kept_pos = torch.where(over, pos.gather(2, src), s["pos"][..., :keep])
    pos_out[..., :keep] = torch.where(held[..., :keep], kept_pos.int(), pos_out[..., :keep])
    weights[..., keep:] = torch.where(held[..., keep:], torch.zeros_like(weights[..., keep:]), weights[..., keep:])
    pos_out[..., keep:] = torch.where(held[..., keep:], -1, pos_out[..., keep:])
    return moved + [s["len"].clamp(max=keep), weights, pos_out, src_rows]


# ----------------------------------------------------------------------------------------------- in 64 bits
def _number(code, scale_byte):
    """The number of an e2m1 code and a scale byte, from the fields of the two formats."""
    code, b = code.long(), scale_byte.long()
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
    se, sm = b >> 3, (b & 7).double()
    s = torch.where(se == 0, sm / 8 * 2.0 ** -14, (1 + sm / 8) * torch.exp2((se - 15).double()))
    return torch.where((code & 8) > 0, -mag, mag) * s


def _row64(codes, scales):
    low, high = codes & 15, codes >> 4
    pair = torch.stack((low, high), -1).flatten(-2)
    return _number(pair, scales.repeat_interleave(16, -1))


def _nearest64(x):
    """The value that a 4-bit row holds for x: the nearest scale to amax / 6, then the nearest code, ties to even."""
    x = x.double()
    a = x.abs().unflatten(-1, (8, 16)).clamp(max=MAX_VALUE)
    want = a.amax(-1, keepdim=True) / 6
    e = torch.floor(torch.log2(want.clamp(min=2.0 ** -14)))
    step = torch.exp2(e - 3)
    s = (torch.round(want / step) * step).clamp(max=10240.0)
    y = a / torch.where(s > 0, s, torch.ones_like(s))
    unit = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = (torch.round(y / unit) * unit).clamp(max=6.0) * s
    return torch.copysign(y.flatten(-2), x)


def _weights64(q, k, mask):
    """softmax rows of q [R, 128] against k [L, 128] under mask [R, L], in 64 bits."""
    x = (q.double() @ k.double().T) * SCALE
    x = x.masked_fill(~mask, -math.inf)
    return torch.softmax(x, -1).nan_to_num(0.0)


def exact(case, seed):
    s = prepare(case, seed)
    n, n_kv, gqa, keep = case["n"], case["n_kv"], case["gqa"], case["keep"]
    lens = s["len"].tolist()
    if case["op"] == "kv4_append":
        k, v = torch.zeros_like(s["new_k"]).double(), torch.zeros_like(s["new_v"]).double()
        for u, t in enumerate(s["new_len"].tolist()):
            k[u, :, :t], v[u, :, :t] = _nearest64(s["new_k"][u, :, :t]), _nearest64(s["new_v"][u, :, :t])
        return {"k_values": k, "v_values": v, "len": None}
    if case["op"] in ("kv4_decode", "dense_decode_weights"):
        out = torch.zeros(n, n_kv * gqa, D, dtype=torch.float64, device=DEV)
        w = None if s["weights"] is None else s["weights"].double()
        for u, t in enumerate(lens):
            for g in range(n_kv):
                if case["op"] == "dense_decode_weights":
                    k, v = s["k"][u, g, :t].double(), s["v"][u, g, :t].double()
                else:
                    if case["block"]:
                        cat = lambda x: x[s["table"][u].long(), g].flatten(0, 1)[:t]  # noqa: E731,B023
                    else:
                        cat = lambda x: x[u, g, :t]  # noqa: E731,B023
                    k, v = _row64(cat(s["k_codes"]), cat(s["k_scales"])), _row64(cat(s["v_codes"]), cat(s["v_scales"]))
                if case["append"]:
                    k, v = torch.cat((k, _nearest64(s["new_k"][u, g])[None])), torch.cat((v, _nearest64(s["new_v"][u, g])[None]))
                heads = slice(g * gqa, (g + 1) * gqa)
                p = _weights64(s["q"][u, heads], k, torch.ones(gqa, k.shape[0], dtype=torch.bool, device=DEV))
                out[u, heads] = p @ v
                if w is not None:
                    w[u, g, : k.shape[0]] += p.sum(0)
        got = [out] if w is None else [out, w]
        return got + [None] if case["append"] else got
    if case["op"] == "prompt_weights":
        w = s["weights"].double()
        for u, (t, length) in enumerate(zip(s["q_len"].tolist(), lens)):
            j = torch.arange(length, device=DEV)
            for h in range(n_kv * gqa):
                for a in range(0, t, 4096):
                    i = torch.arange(a, min(t, a + 4096), device=DEV)[:, None]
                    p = _weights64(s["q"][u, h, a : a + i.shape[0]], s["k"][u, h // gqa, :length], j <= length - t + i)
                    w[u, h // gqa, :length] += p.sum(0)
        return w
    # eviction: the same rows, one (unit, head) at a time on the host
    names = ("k_codes", "k_scales", "v_codes", "v_scales") if case["kv4"] else ("k", "v")
    weights, pos = s["weights"].double().cpu(), s["pos"].cpu()
    w_out, p_out = s["weights_out"].double().cpu(), s["pos_out"].cpu()
    source = torch.full((n, n_kv, case["cap"]), -1, dtype=torch.int64)
    seen = s["seen"].tolist()
    for u, length in enumerate(lens):
        for g in range(n_kv):
            w, p = weights[u, g, :length], pos[u, g, :length].clone()
            rows = torch.arange(length)
            if length > keep:
                p = torch.where(p < 0, seen[u] - length + rows, p)
                safe = p >= seen[u] - case["recent"]
                order = torch.argsort(torch.where(safe, math.inf, w), descending=True, stable=True)[:keep]
                mask = torch.zeros(length, dtype=torch.bool)
                mask[order] = True
                place = rows[:keep].clone()
                place[~mask[:keep]] = rows[keep:][mask[keep:]]
                source[u, g, :keep] = place
                w_out[u, g, :keep], w_out[u, g, keep:length] = w[place], 0
                p_out[u, g, :keep], p_out[u, g, keep:length] = p[place].int(), -1
            else:
                source[u, g, :length] = rows
                w_out[u, g, :length], p_out[u, g, :length] = w, p
    at = torch.where(source < 0, torch.arange(case["cap"]), source)
    if keep < case["cap"]:
        at[..., keep:] = torch.arange(keep, case["cap"])
    at = at.to(DEV)[..., None]
    moved = [s[m].gather(2, at.expand(-1, -1, -1, s[m].shape[-1])) for m in names]
    return moved + [s["len"].clamp(max=keep), w_out, p_out, source[..., :keep].int()]
