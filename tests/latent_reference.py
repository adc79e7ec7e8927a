"""Plain 64-bit forms of the rotary, latent-store and latent-attention operators, and how far a kernel's
outputs may be from them.  Inputs are float64 arrays of bf16 values."""

import numpy as np


def bf16(x):
    """float64 values of x rounded to bf16 (nearest, ties to even)."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def rotate(x, positions, inv_freq, interleaved, magnitude=1.0):
    """(y, bound): x [n, heads, dim] with its first 2 len(inv_freq) elements rotated, and the error of a bf16 result:
    its rounding, 2^-8 of it; and of the fp32 sums, |x1| + |x2| times 2^-20: angles are off by up to 2^-25 turns (the
    fraction's 24 bits), 2^-22.3 radians, and sines, cosines, products and sums by 2^-23 or less each."""
    rot = 2 * len(inv_freq)
    a = np.asarray(positions, np.float64)[:, None] * inv_freq
    c, s = (magnitude * f(a)[:, None, :] for f in (np.cos, np.sin))
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y, slack = x.copy(), np.zeros_like(x)
    x1, x2 = x[..., first], x[..., second]
    y[..., first], y[..., second] = x1 * c - x2 * s, x2 * c + x1 * s
    slack[..., first] = slack[..., second] = (np.abs(x1) + np.abs(x2)) * abs(magnitude) * 2.0 ** -20
    return y, slack


def normalise(c, weight, eps):
    """(y, slack): a row c * weight / sqrt(mean(c^2) + eps); the fp32 form is off by a few of its 24 bits' steps,
    the sum's included (all its terms are positive): 2^-20 of the value."""
    y = c / np.sqrt((c * c).mean(-1, keepdims=True) + eps) * weight
    return y, np.abs(y) * 2.0 ** -20


def attend(q, rows, latent, scale, seen):
    """(o, bound): attention of q [n, heads, width] over rows [keys, width], values their first `latent` elements, query
    i over the first seen[i] rows.

    The kernel's errors: its output's rounding, 2^-8 of the result; a weight's rounding to bf16, 2^-8 of the weight,
    which moves the result by at most sum_j p_j 2^-8 |v_j - o|, for the sum that divides takes the rounded weights; a logit,
    an fp32 sum of `width` products, off by at most (width + 4) 2^-24 sum |q_i k_i| times the scale, and so ln w_j (of
    this key and of the others), with the exponential's 2^-21 beside it; the fp32 sums over the keys and their
    rescaling, 2^-24 of sum p |v| a key, at most."""
    n, heads, width = q.shape
    o, bound = np.zeros((n, heads, latent)), np.zeros((n, heads, latent))
    for i in range(n):
        m = int(seen[i])
        if m <= 0:
            continue
        k, v = rows[:m], rows[:m, :latent]
        s = q[i] @ k.T * scale                                     # [heads, m]
        w = np.exp(s - s.max(-1, keepdims=True))
        p = w / w.sum(-1, keepdims=True)
        o[i] = p @ v
        logit = ((width + 4) * 2.0 ** -24 * scale) * (np.abs(q[i]) @ np.abs(k).T).max(-1)
        err = 2.0 ** -8 + 2 * logit + 2.0 ** -21
        # sum_j p_j |v_j - o| <= sum_j p_j |v_j| + |o|, and exactly where the keys are few
        if m <= 512:
            spread = np.stack([p[h] @ np.abs(v - o[i, h]) for h in range(heads)])
        else:
            spread = p @ np.abs(v) + np.abs(o[i])
        bound[i] = 2.0 ** -8 * np.abs(o[i]) + err[:, None] * spread + (m + 8) * 2.0 ** -24 * (p @ np.abs(v)) + 1e-37
    return o, bound
