"""Tolerances of the serving step's calls against the float64 oracle, derived from the kernels' arithmetic.

u = 2^-24 is half a step of fp32 (relative), 2^-8 of bf16; the hardware exponential is within 2^-22 of 2^x,
relatively, besides the rounding of its argument.

Attention. A logit (log2 domain) is a sum of 128 exact products of bf16 numbers on the tensor core, each
addition within 2 u, times a constant: within eps = 260 u A of the true one, A = scale log2(e) sum_c |q_c k_c|.
The exponent s - m is one multiply-add: off by another u |s - m| <= u (2 A + 16). So a numerator is off,
relatively, by ln 2 (eps + u (2 A + 16)) + 2^-22; raising the reference m and joining parts multiply by further
exponentials, each within 2^-21 with its rounding: fewer than 2^7 of them, 2^-14. The divisor is a sum of such
numbers in fp32, of at most L additions. P enters the product with V rounded to bf16 (2^-8); that product's sum has
L additions within 2 u, and the result is divided and rounded to bf16:
    (2 ln 2 (eps + u (2 A + 16)) + 2^-21 + 2^-13 + 3 L u + 2^-8) sum_j p_j |v_j| + 2^-8 |ref|.

Rotary positions. The angle is a fraction of a turn: the frequency's is within 2^-53 of it (relative, double), so
2^-53 |pos| f / (2 pi) turns, the upper 32 bits lose 2^-32, their conversion 2^-25, and sincospi is within 2 u:
    e = 2 pi (2^-53 |pos| f / (2 pi) + 2^-24.5) + 2 u.
Each output is a sum of two products (fp32; mscale times the cosine is rounded too): within (e + 4 u) mscale (|a| +
|b|) and rounded to bf16: 2^-8 |ref|.
"""
import numpy as np

U32 = 2.0 ** -24
LN2 = float(np.log(2.0))


def within(got, ref, tol, what):
    got = np.asarray(got, dtype=np.float64)
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    if bad.any():
        at = int(np.argmax(np.where(np.isfinite(err), err - tol, np.inf)))
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; worst {err.flat[at]:.3e} (tolerance "
                             f"{tol.flat[at]:.3e}, ref {ref.flat[at]:.4e}) at {np.unravel_index(at, ref.shape)}")


def attention_tolerance(q, k, scale, ref, mag):
    """q [T, Hq, 128], k [n_kv, L, 128], ref and mag [T, Hq, 128]; a bound for each query head of its own."""
    gqa, L = q.shape[1] // k.shape[0], k.shape[1]
    e = np.zeros((1, q.shape[1], 1))
    for h in range(q.shape[1]):
        a = np.abs(q[:, h]) @ np.abs(k[h // gqa]).T
        a = (a.max() if a.size else 0.0) * scale / LN2
        e[0, h, 0] = 2 * LN2 * (260 * U32 * a + U32 * (2 * a + 16)) + 2.0 ** -21 + 2.0 ** -13
    return (e + 3 * L * U32 + 2.0 ** -8) * mag + 2.0 ** -8 * np.abs(ref) + 1e-30


def turn_tolerance(x, positions, inv_freq, interleaved, mscale, ref):
    half = len(inv_freq)
    pos = np.abs(np.asarray(positions, dtype=np.float64))[:, None]
    e = 2 * np.pi * (2.0 ** -53 * pos * np.abs(inv_freq) / (2 * np.pi) + 2.0 ** -24.5) + 2 * U32
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    both = np.abs(x[..., a]) + np.abs(x[..., b])
    tol = np.zeros(x.shape)
    tol[..., a] = tol[..., b] = ((e + 4 * U32) * abs(mscale))[:, None] * both
    tol[..., :2 * half] += 2.0 ** -8 * np.abs(ref[..., :2 * half]) + 2.0 ** -133
    return tol
