"""Attention of packed tokens at the largest scores that it promises: scale log2(e) q . k up to 2^28 in magnitude, where fp32
holds them to 16. All numbers below are exact in bf16, and their products and sums in fp32.

Equal scores s: the reference is s rounded, and the numerators are 2^r with one r, |r| <= 8, for all keys: rounded to bf16
by one common factor within 2^-8, in fp32 sums of at most L additions within 2^-23 each; the division and the rounding of
the result to bf16 add 2^-22 and 2^-8. So outputs are the mean of the visible values, within
2^-7 |mean| + (2^-15 + 2 L 2^-23) mean |v|. With one key twice as far up the others' numerators are 0: its value alone,
within 2^-7 of it and what is left of the bound above.
"""
import numpy as np
import pytest

from oracle import serve as S
from tests.test_gpu_serve_attention import SCALE, Case

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


def _case(**kw):
    c = Case(**kw)
    c.q.fill_(2.0 ** 11)
    for u, L in enumerate(c.lens):
        c.k[u, :, :L] = 1.5 * 2.0 ** 12
    assert 2 ** 27 < 128 * 1.5 * 2.0 ** 23 * SCALE * LOG2E < 2 ** 28
    return c


def _run(c):
    from sparse_kv_cache_snapkv_gb300 import rkv
    out, ws = c.call()
    rkv.rkv_check_status(ws)
    return out.double().cpu().numpy()


CASES = {"prompt": dict(news=[140], lens=[1000]), "tree": dict(news=[40], lens=[300], words=2),
         "cut": dict(news=[20], lens=[20000])}


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("name", sorted(CASES))
def test_equal_scores(name, sign):
    c = _case(seed=1, **CASES[name])
    c.k *= sign
    got, T, L = _run(c), c.news[0], c.lens[0]
    sees = S.visible(T, L, None if c.mask is None else c.mask.cpu().numpy()).astype(np.float64)
    sees /= sees.sum(1, keepdims=True)
    for h in range(8):
        v = c.v[0, h // 4, :L].double().cpu().numpy()
        ref, mag = sees @ v, sees @ np.abs(v)
        err = np.abs(got[:, h] - ref)
        assert (err <= 2.0 ** -7 * np.abs(ref) + (2.0 ** -15 + 2 * L * 2.0 ** -23) * mag).all(), (h, err.max())


@pytest.mark.parametrize("at", [0, 31, 32, 127, 128, 700])
@pytest.mark.parametrize("low", [0.5, -1.0])
def test_one_key_far_above(at, low):
    c = _case(seed=2, **CASES["prompt"])
    c.k[:, :, : c.lens[0]] *= low
    c.k[0, :, at] = 1.5 * 2.0 ** 12
    got, T, L = _run(c), c.news[0], c.lens[0]
    for h in range(8):
        v = c.v[0, h // 4, at].double().cpu().numpy()
        err = np.abs(got[:, h] - v)
        assert (err <= (2.0 ** -7 + 2.0 ** -15) * np.abs(v) + 2.0 ** -30).all(), (h, err.max())
