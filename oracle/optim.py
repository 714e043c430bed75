"""One AdamW step over a list of tensors -- oracle, TEST INFRASTRUCTURE ONLY.

Decoupled weight decay, bias-corrected moments, the clip of the global norm, in float64; the 8-bit
moments' grid and their stochastic rounding from the definition (a float of few bits, rounded up
where its place between two grid values and the element's random number reach the next one).
The pages name few-bit optimizer states without a format ("FTDD-03" teaching script, decision 3);
the format read here is stated in the functions.
"""

import numpy as np

BLOCK = 256


def hash32(x):
    """The 32-bit mixer whose constants C. Wellons, "Prospecting for Hash Functions" (2018), gives."""
    x = np.asarray(x, dtype=np.uint64) & 0xFFFFFFFF
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x7FEB352D)) & np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x846CA68B)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def element_bits(seed, t, e):
    """32 random bits of element numbers e at step t."""
    e = np.asarray(e, dtype=np.uint64)
    word = int(hash32(int(hash32(seed & 0xFFFFFFFF)) + t))
    hi = ((e >> np.uint64(32)) * np.uint64(0x9E3779B1)) & np.uint64(0xFFFFFFFF)
    return hash32(((e & np.uint64(0xFFFFFFFF)) ^ hi) + np.uint64(word))


def grid(mantissa, codes, top_code):
    """Values of codes 0..codes-1: code top_code is 1.0, each below the next lower float of
    `mantissa` bits, code 0 is 0."""
    c = np.arange(codes, dtype=np.int64)
    k = 127 * 2 ** mantissa - top_code + c
    v = 2.0 ** (k // 2 ** mantissa - 127) * (1 + (k % 2 ** mantissa) / 2 ** mantissa)
    v[0] = 0.0
    return v


M_GRID = grid(3, 128, 127)
V_GRID = grid(4, 256, 255)


def encode(x, values, r16, never_zero):
    """(codes, distance of the decision from a tie in steps, step) of x in [0, 1]: between neighbouring values lo
    and hi above 0, hi where (x - lo) / (hi - lo) + r16 / 65536 >= 1; below the least value, that
    value where r16 / 65536 < x / least (never_zero: wherever x > 0)."""
    lo = np.clip(np.searchsorted(values, x, side="right") - 1, 0, len(values) - 2)
    frac = (x - values[lo]) / (values[lo + 1] - values[lo])
    place = frac + r16 / 65536.0 - 1.0
    place = np.where(lo > 0, place, 1.0 if never_zero else frac - r16 / 65536.0)
    up = np.where(lo > 0, place >= 0, (place > 0) & (x > 0))
    return lo + up, np.abs(place), values[lo + 1] - values[lo]


def decode(code, values, scale):
    return values[code] * np.repeat(scale, BLOCK)[: len(code)]


def blocks_of(sizes):
    return [-(-n // BLOCK) for n in sizes]


def step(p, g, m, v, t, lr, b1, b2, eps, wd, factor):
    """One tensor (flat float64 arrays): (p', m', v', magnitude of m', magnitude of the move), the
    magnitudes with the two terms of m', which may cancel, in absolute value."""
    g = g * factor
    m_mag = np.abs(b1 * m) + np.abs((1 - b1) * g)
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    over = (1 - b1 ** t) * (np.sqrt(v / (1 - b2 ** t)) + eps)
    return p - lr * wd * p - lr * m / over, m, v, m_mag, abs(lr) * m_mag / over


def clip_factor(grads, grad_scale, max_norm):
    """(norm of the scaled gradients, factor on the gradients)."""
    norm = float(np.sqrt(sum(float(np.sum(np.square(np.asarray(g, np.float64)))) for g in grads)))
    norm *= abs(grad_scale)
    clip = min(1.0, max_norm / (norm + 1e-6)) if max_norm else 1.0
    return norm, grad_scale * clip
