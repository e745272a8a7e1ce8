"""Tolerances of the cache calls against the float64 oracle, derived from the kernels' arithmetic.

u = 2^-24 is half a step of fp32 (relative), 2^-11 of fp16, 2^-8 of bf16; the hardware exponential
is within 2^-22 of 2^x, relatively, besides the rounding of its argument.

Logit (log2 domain): 128 exact products (of bf16 numbers, or of exact 4-bit values and queries
scaled by a power of two) summed in fp32 in any order, a sum on the tensor core being within 2 u,
then one multiplication: within eps = 260 u A of the true one, A = scale log2(e) sum_c |q_c k_c|.
(4 bits: queries below 2^-25 of their head's largest lose up to 2^-33 of it, far inside eps.)

Probability p = 2^(s - m) / l. The numerator and each term of l are off, relatively, by
ln 2 (eps + u |s - m|) + 2^-22, and u |s - m| <= 2 u A < eps; l has `terms` additions of its own. So
    e_p = 2 (2 ln 2 eps_max + 2^-22) + terms u,
eps_max from the largest A of the call. A weight is a sum of p over queries and heads, in up to
`terms` additions, added to what was there:  (e_p + terms u) w + 2 u (w + before).

Output: sum_t p_t v_t, with p rounded for the product: to fp16 (4 bits) by 2^-11 of a value, or
2^-25 where 2^7 p leaves the normal numbers: 2^-32 of the largest p, hence at most T 2^-31 max|v|
over T tokens after the division by l; to two bf16 numbers otherwise, by 2^-16. The sum has at most
`terms` roundings and the result is rounded to bf16:
    (e_p + terms u + 2^-11 or 2^-16) sum_t p_t |v_t| + T 2^-31 max|v| (4 bits) + 2^-8 |ref|.
"""
import numpy as np

from oracle import cache as C

U32 = 2.0 ** -24
LN2 = float(np.log(2.0))


def probability_error(q, k, scale, terms):
    a = np.abs(np.asarray(q, dtype=np.float64)) @ np.abs(np.asarray(k, dtype=np.float64)).T
    eps = 260 * U32 * (a.max() if a.size else 0.0) * scale / LN2
    return 2 * (2 * LN2 * eps + 2.0 ** -22) + terms * U32


def _within(got, ref, tol, what):
    err = np.abs(np.asarray(got, dtype=np.float64) - ref)
    bad = ~(err <= tol)
    if bad.any():
        worst = int(np.argmax(np.where(np.isfinite(err), err - tol, np.inf)))
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; worst {err.flat[worst]:.3e}"
                             f" (tolerance {tol.flat[worst]:.3e}, ref {ref.flat[worst]:.4e}) at {worst}")


def check_weights(got, added, before, q, k, scale, terms, what="weights"):
    """got = before + added within the bound (q [R, d], k [T, d] of the group)."""
    added, before = np.asarray(added, dtype=np.float64), np.asarray(before, dtype=np.float64)
    tol = (probability_error(q, k, scale, terms) + terms * U32) * added
    _within(got, before + added, tol + 2 * U32 * np.abs(before + added) + 1e-30, what)


def check_output(got, q, k, v, scale, kv4, terms, what="output"):
    """got [G, d] against the softmax attention of q over k, v [T, d] (the numbers held)."""
    p = C.softmax_weights(q, k, scale)
    v = np.asarray(v, dtype=np.float64)
    ref, mag = p @ v, p @ np.abs(v)
    tol = (probability_error(q, k, scale, terms) + terms * U32 + (2.0 ** -11 if kv4 else 2.0 ** -16)) * mag
    tol = tol + 2.0 ** -8 * np.abs(ref) + 1e-30
    if kv4 and v.size:
        tol = tol + v.shape[0] * 2.0 ** -31 * np.abs(v).max()
    _within(got, ref, tol, what)
