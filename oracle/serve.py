"""Oracle of a serving step around the cache (places, rotary positions, attention of packed tokens): numpy in
float64 and Python integers, written from the definitions in include/rkv.h, without the library's arithmetic.
"""
from __future__ import annotations

import math

import numpy as np

from .cache import softmax_weights


def reserve(new_len, length, held, table, free_blocks, free_count, block, max_tokens):
    """What rkv_reserve_slots leaves: a dict of its outputs (table included) and the status bits it sets."""
    num_blocks, max_blocks = len(free_blocks), len(table[0])
    table = [list(t) for t in table]
    room = free_count if 0 <= free_count <= num_blocks else 0
    bits = 0 if room == free_count else 0x10
    start, starts, asked, taken = 0, [], 0, 0
    slots, positions = [-1] * max_tokens, [0] * max_tokens
    len_out, held_out = list(length), list(held)
    for u, (add, have, own) in enumerate(zip(new_len, length, held)):
        starts.append(min(start, 2 ** 31 - 1))
        mine = start
        start += max(add, 0)
        if add < 0 or have < 0 or not 0 <= own <= max_blocks or have + add > max_blocks * block:
            bits |= 0x1
            continue
        if own < -(-have // block):
            bits |= 0x10
            continue
        if start > max_tokens:
            bits |= 0x1
            continue
        need = max(0, -(-(have + add) // block) - own)
        asked += need
        if need and asked > room:
            bits |= 0x20
            continue
        for j in range(need):
            table[u][own + j] = free_blocks[room - 1 - taken - j]
        taken += need
        len_out[u], held_out[u] = have + add, own + need
        for i in range(add):
            b = table[u][(have + i) // block]
            if 0 <= b < num_blocks:
                slots[mine + i], positions[mine + i] = b * block + (have + i) % block, have + i
            else:
                bits |= 0x10
    starts.append(min(start, 2 ** 31 - 1))
    return dict(q_start=starts, slots=slots, positions=positions, table=table, len=len_out, held=held_out,
                free_count=free_count - taken), bits


def release(length, held, table, free_blocks, free_count, block):
    """What rkv_release_blocks leaves, and the status bits."""
    num_blocks, max_blocks = len(free_blocks), len(table[0])
    bits, back, held_out = 0, [], list(held)
    for u, (have, own) in enumerate(zip(length, held)):
        if have < 0 or not 0 <= own <= max_blocks:
            bits |= 0x1
            continue
        keep = min(own, -(-have // block))
        back += list(table[u][keep:own])
        held_out[u] = keep
    free = list(free_blocks)
    if not 0 <= free_count <= num_blocks or len(back) > num_blocks - free_count:
        return dict(free_blocks=free, held=list(held), free_count=free_count), bits | 0x10
    if any(not 0 <= b < num_blocks for b in back):
        bits |= 0x10
    free[free_count:free_count + len(back)] = back
    return dict(free_blocks=free, held=held_out, free_count=free_count + len(back)), bits


def frequencies(kind, rot, base, factor=1.0, ctx=0, fast=32.0, slow=1.0):
    """inv_freq [rot / 2] and mscale."""
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "plain":
        return np.array(f), 1.0
    if kind == "linear":
        return np.array(f) / factor, 1.0
    if kind == "base":
        b = base * factor ** (rot / (rot - 2))
        return np.array([b ** (-2.0 * i / rot) for i in range(rot // 2)]), 1.0
    out = []
    for i, x in enumerate(f):
        if kind in ("by_parts", "by_whole_parts"):
            # pair numbers at which a pair turns `fast` and `slow` times within ctx
            first, last = (rot / 2 * math.log(ctx / (2 * math.pi * t)) / math.log(base) for t in (fast, slow))
            if kind == "by_whole_parts":
                first, last = (min(max(e, 0), rot - 1) for e in (math.floor(first), math.ceil(last)))
                last += 0.001 * (first == last)
            share = 1 - min(max((i - first) / (last - first), 0.0), 1.0)
        else:
            share = min(max((ctx * x / (2 * math.pi) - slow) / (fast - slow), 0.0), 1.0)
        out.append(x * share + x / factor * (1 - share))
    return np.array(out), 1.0 if kind == "smooth" else 0.1 * math.log(factor) + 1


def turn(x, positions, inv_freq, interleaved, mscale=1.0):
    """x [tokens, heads, 128] at its positions."""
    x = np.asarray(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    # whole turns are dropped in extended precision: a far position's angle has few bits behind the point
    w = np.asarray(positions, dtype=np.longdouble)[:, None] * f.astype(np.longdouble)
    two_pi = np.longdouble("6.283185307179586476925286766559005768")
    w = (w - np.round(w / two_pi) * two_pi).astype(np.float64)
    z = mscale * np.exp(1j * w)[:, None]
    half, y = len(f), x.copy()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    t = (x[..., a] + 1j * x[..., b]) * z
    y[..., a], y[..., b] = t.real, t.imag
    return y


def visible(T, L, mask=None):
    """[T, L]: which of a unit's L rows each of its T new tokens sees (mask [T, words] of 32-bit words)."""
    j = np.arange(L)
    if mask is None:
        return j[None] <= L - T + np.arange(T)[:, None]
    words = np.asarray(mask, dtype=np.int64) & 0xFFFFFFFF
    sees = np.ones((T, L), dtype=bool)
    for d in range(T):
        sees[:, L - T + d] = (words[:, d // 32] >> (d % 32)) & 1 == 1
    return sees


def attention(q, k, v, scale, sees):
    """out [T, Hq, 128], and the sums of |p v| beside it, of q [T, Hq, 128] over k, v [n_kv, L, 128]."""
    T, hq, d = q.shape
    gqa = hq // k.shape[0]
    out, mag = np.zeros((T, hq, d)), np.zeros((T, hq, d))
    for h in range(hq):
        p = softmax_weights(q[:, h], k[h // gqa], scale, sees)
        vv = np.asarray(v[h // gqa], dtype=np.float64)
        out[:, h], mag[:, h] = p @ vv, p @ np.abs(vv)
    return out, mag
