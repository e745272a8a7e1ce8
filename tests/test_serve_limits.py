"""Counts of units near the end of 32 bits: refused before any launch, with a workspace size of 0. (The kernels' loops over
the units step by a block's or a grid's threads in 32 bits, and the plan's pairs are counted in them.) No GPU needed."""
import pytest

from tests.test_serve_contract import CALLS, lib  # noqa: F401

TOP = 2 ** 31 - 1
MOST = 2 ** 30


@pytest.mark.parametrize("n", [MOST + 1, TOP - 4096, TOP - 1024, TOP - 1])
def test_too_many_units(lib, n):  # noqa: F811
    assert lib.rkv_reserve_slots_workspace_bytes(n) == 0
    assert lib.rkv_release_blocks_workspace_bytes(n) == 0
    for gqa, tokens in ((1, 9), (64, 2 ** 24), (64, 1)):
        assert lib.rkv_prompt_attention_workspace_bytes(n, 1, gqa, tokens) == 0, (gqa, tokens)
    for name in ("rkv_reserve_slots", "rkv_release_blocks", "rkv_prompt_attention_paged", "rkv_tree_attention_paged"):
        ok, _ = CALLS[name]
        assert getattr(lib, name)(*{**ok, "n": n}.values()) == 1, name


def test_as_many_units_as_there_may_be(lib):  # noqa: F811
    """Sizes are those of their formulas' order, and do not fall on the way there."""
    for size, per in ((lib.rkv_reserve_slots_workspace_bytes, 16), (lib.rkv_release_blocks_workspace_bytes, 16),
                      (lambda n: lib.rkv_prompt_attention_workspace_bytes(n, 1, 64, 2 ** 24), 68)):
        last = 0
        for n in (1, 2 ** 20, 2 ** 29, MOST - 1, MOST):
            got = size(n)
            assert max(last, per * n) <= got <= per * n + 2 ** 31, n
            last = got
