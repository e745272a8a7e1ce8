"""The README's example of a 4-bit cache that is evicted from runs as it stands."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(__file__), "..", "README.md")


def test_readme_example_of_a_shrinking_cache():
    from sparse_kv_cache_snapkv_gb300 import rkv
    with open(README) as f:
        code = [c for c in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "kv4_cache" in c]
    assert len(code) == 1
    n, n_kv, gqa, D, T, keep, steps = 2, 2, 4, 128, 700, 456, 513
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    prompt_len = torch.tensor([700, 300], dtype=torch.int32, device="cuda")
    q_t = r(n, n_kv * gqa, D)
    names = dict(rkv=rkv, torch=torch, n=n, n_kv=n_kv, cap=T + 256, keep=keep, steps=steps, scale=D ** -0.5,
                 k=r(n, n_kv, T, D), v=r(n, n_kv, T, D), q=r(n, n_kv * gqa, T, D), prompt_len=prompt_len,
                 length=torch.zeros_like(prompt_len), q_t=q_t, k_t=r(n, n_kv, D), v_t=r(n, n_kv, D),
                 out=torch.full_like(q_t, float("nan")))
    exec(code[0], names)
    torch.cuda.synchronize()
    # 256 steps, an eviction, 256 more, another, one more
    assert names["length"].tolist() == [keep + 1, keep + 1]
    assert names["seen"].tolist() == [1213, 813]
    assert torch.isfinite(names["out"]).all() and (names["weights"] >= 0).all()
