"""The README's step of a serving engine runs, and its outputs are the attention of what it stored."""
import math
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_readme_serving_step():
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), flags=re.S)
    code = [b for b in blocks if "rkv_reserve_slots" in b]
    assert len(code) == 1
    from sparse_kv_cache_snapkv_gb300 import rkv
    n, n_kv, hq, block, most, scale = 3, 2, 8, 16, 20, 1 / math.sqrt(128)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    new = [100, 1, 33]
    tokens = sum(new)
    v = dict(rkv=rkv, torch=torch, n=n, n_kv=n_kv, hq=hq, block=block, scale=scale, new_len=ints(new),
             length=ints([0] * n), held=ints([0] * n), table=torch.full((n, most), -1, dtype=torch.int32, device="cuda"),
             free=torch.randperm(40, device="cuda").int(), count=ints([40]), q_start=ints([0] * (n + 1)),
             slots=ints([0] * tokens), positions=ints([0] * tokens),
             qkv=torch.randn(tokens, hq + 2 * n_kv, 128, device="cuda").bfloat16(),
             q_turned=torch.zeros(tokens, hq, 128, dtype=torch.bfloat16, device="cuda"),
             out=torch.zeros(tokens, hq, 128, dtype=torch.bfloat16, device="cuda"),
             k_pool=torch.zeros(40, n_kv, block, 128, dtype=torch.bfloat16, device="cuda"),
             v_pool=torch.zeros(40, n_kv, block, 128, dtype=torch.bfloat16, device="cuda"))
    exec(code[0], v)
    assert v["length"].tolist() == new and int(v["count"]) == 40 - 7 - 1 - 3
    at = [0, 100, 101, 134]
    for u in range(n):
        rows = slice(at[u], at[u + 1])
        k, w = (v[p][v["table"][u, : int(v["held"][u])].long()].transpose(0, 1).flatten(1, 2)[:, : new[u]].float()
                for p in ("k_pool", "v_pool"))
        q = v["q_turned"][rows].float().unflatten(1, (n_kv, -1))
        x = torch.einsum("tgcd,gld->gctl", q, k) * scale
        x = x.masked_fill(torch.ones(new[u], new[u], dtype=torch.bool, device="cuda").triu(1), -math.inf).softmax(-1)
        ref = torch.einsum("gctl,gld->tgcd", x, w).flatten(1, 2)
        # (two bf16 roundings, of the weights and of the outputs, and fp32 products on both sides)
        mag = torch.einsum("gctl,gld->tgcd", x, w.abs()).flatten(1, 2)
        assert ((v["out"][rows].float() - ref).abs() <= 2.0 ** -7 * mag + 2.0 ** -7 * ref.abs()).all()
