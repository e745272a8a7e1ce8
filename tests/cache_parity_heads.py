"""Tolerances of the cache decodes per query head, from the kernels' arithmetic.

As tests/cache_parity.py, but each head is held to its own logits' size: A_h = scale log2(e)
max_t sum_c |q_hc k_tc|, eps_h = 260 u A_h, and a head's probabilities are within
    e_h = 2 (2 ln 2 eps_h + 2^-22) + terms u
of the true ones, relatively. `check_decode` refuses a case whose e_h is above MOST, so that no
case passes because its tolerance is wider than its values.

Output: p enters the product with V as the sum of two numbers of the product's type. Two fp16
numbers hold it within 2^-11 2^-11 = 2^-22 of itself, or within 2^-25 of 2^7 p where the second
leaves the normal numbers: 2^-32 of the largest p, at most T 2^-31 max|v| over T tokens after the
division by l (the joins' rescaling is exact to u, counted in `terms`). Two bf16 numbers: 2^-16. So
    (e_h + terms u + 2^-22 or 2^-16) sum_t p_t |v_t| + T 2^-31 max|v| (4 bits) + 2^-8 |ref|.
"""
import numpy as np

from oracle import cache as C
from tests.cache_parity import LN2, U32

MOST = 0.05


def head_errors(q, k, scale, terms):
    """e_h of every row of q [R, d] against k [T, d]."""
    a = np.abs(np.asarray(q, dtype=np.float64)) @ np.abs(np.asarray(k, dtype=np.float64)).T
    eps = 260 * U32 * a.max(1) * scale / LN2
    return 2 * (2 * LN2 * eps + 2.0 ** -22) + terms * U32


def check_decode(out, added, q, k, v, scale, kv4, terms, what, most=MOST):
    """Outputs [G, d] and weights [T] (that began at zero; None: not asked for) of one KV group."""
    k, v = np.asarray(k, dtype=np.float64), np.asarray(v, dtype=np.float64)
    e = head_errors(q, k, scale, terms)
    assert (e < most).all(), f"{what}: a tolerance of {e.max():.2e} shows nothing"
    p = C.softmax_weights(q, k, scale)
    ref, mag = p @ v, p @ np.abs(v)
    tol = (e[:, None] + terms * U32 + (2.0 ** -22 if kv4 else 2.0 ** -16)) * mag
    tol = tol + 2.0 ** -8 * np.abs(ref) + (v.shape[0] * 2.0 ** -31 * np.abs(v).max() if kv4 else 0) + 1e-30
    _within(out, ref, tol, what)
    if added is not None:
        w = p.sum(0)
        _within(added, w, ((e[:, None] + terms * U32) * p).sum(0) + 2 * U32 * w + 1e-30, what + " weights")


def _within(got, ref, tol, what):
    err = np.abs(np.asarray(got, dtype=np.float64) - ref)
    over = err / tol
    assert (err <= tol).all(), (f"{what}: {(~(err <= tol)).sum()} of {err.size} outside, worst "
                                f"{np.nanmax(over):.2f} tolerances at {np.unravel_index(np.nanargmax(over), err.shape)}")
