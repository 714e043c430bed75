"""Residual updates with their RMS norms, and rotary positions -- oracle, TEST INFRASTRUCTURE ONLY.

Plain definitions in float64 ("Unsloth vs QLoRA vs Liger-Kernel", section 2: RMSNorm and RoPE are
among the hand-differentiated ops)::

    a  = y r_y (w_post + o),  r_y = (mean(y^2) + eps)^(-1/2)      (a = y without w_post)
    h' = res h + br gate a
    n  = h' r_h (w_pre + o),  r_h = (mean(h'^2) + eps)^(-1/2)

The backward is written from the Jacobian of x / rms(x) row by row, apart from the library's
formulas.  Every gradient comes with a magnitude: the sum of the absolute values that are added
for it, to which a bound on the rounding of an fp32 evaluation is proportional.

Rotary angles are in extended precision (64-bit mantissa): position x frequency / 2 pi, of which
the fraction of a turn is kept.
"""

import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def rstd(x, eps):
    x = _f64(x)
    return (np.mean(x * x, axis=1) + eps) ** -0.5


def update(h, y, w_post, gate, eps, res, br, o):
    """(h', magnitude, r_y or None) before rounding to the stored type; gate broadcasts."""
    h, y, w_post, gate = _f64(h), _f64(y), _f64(w_post), _f64(gate)
    r = None
    a = y
    if w_post is not None:
        r = rstd(y, eps)
        a = y * r[:, None] * (w_post + o)
    if gate is not None:
        a = a * gate
    return res * h + br * a, np.abs(res * h) + np.abs(br * a), r


def norm(h_stored, w_pre, eps, o):
    """(n before rounding, r_h) of h' as stored."""
    h = _f64(h_stored)
    r = rstd(h, eps)
    return h * r[:, None] * (_f64(w_pre) + o), r


def _norm_bwd(x, r, w, d, d_mag):
    """Gradient of sum(d * (w x r)), r = rms^-1 of each row of x: the row's Jacobian is
    r (I - (x r)(x r)^T / D).  Returns (dx, its magnitude, dw, its magnitude)."""
    unit = x * r[:, None]
    z, z_mag = d * w, d_mag * np.abs(w)
    D = x.shape[1]
    dx = np.stack([ri * (zi - ui * (ui @ zi) / D) for ri, zi, ui in zip(r, z, unit)]) \
        if len(x) else np.zeros_like(x)
    mag = r[:, None] * (z_mag + np.abs(unit) * np.mean(z_mag * np.abs(unit), axis=1,
                                                       keepdims=True))
    return dx, mag, np.sum(d * unit, axis=0), np.sum(d_mag * np.abs(unit), axis=0)


def backward(dn, dh_out, h_out, y, r_pre, r_post, w_pre, w_post, gate, res, br, o):
    """dict of name -> (gradient, magnitude): dh, dy, dw_pre, dw_post, dgate (whole, before any sum
    over what the gate is broadcast along)."""
    dn, dh_out, h_out, y = _f64(dn), _f64(dh_out), _f64(h_out), _f64(y)
    w_pre, w_post, gate = _f64(w_pre), _f64(w_post), _f64(gate)
    out = {}
    G = dh_out if dh_out is not None else np.zeros_like(h_out)
    G_mag = np.abs(G)
    if w_pre is not None:
        dx, mag, dw, dw_mag = _norm_bwd(h_out, _f64(r_pre), w_pre + o, dn, np.abs(dn))
        G, G_mag = G + dx, G_mag + mag
        out["dw_pre"] = (dw, dw_mag)
    out["dh"] = (res * G, abs(res) * G_mag)
    if y is None:
        return out
    E, E_mag = br * G, abs(br) * G_mag
    a = y if w_post is None else y * _f64(r_post)[:, None] * (w_post + o)
    if gate is not None:
        out["dgate"] = (E * a, E_mag * np.abs(a))
        E, E_mag = E * gate, E_mag * np.abs(gate)
    if w_post is None:
        out["dy"] = (E, E_mag)
    else:
        dy, mag, dw, dw_mag = _norm_bwd(y, _f64(r_post), w_post + o, E, E_mag)
        out["dy"], out["dw_post"] = (dy, mag), (dw, dw_mag)
    return out


def frequencies(rd, base, scaling=None):
    """(radians per position of each pair in extended precision, factor on the values)."""
    L = np.longdouble
    i = np.arange(0, rd, 2).astype(L)
    f = L(base) ** (-i / rd)
    if scaling is None:
        return f, 1.0
    kind, s = scaling["kind"], L(scaling["factor"])
    two_pi = L("6.283185307179586476925286766559")
    if kind == "linear":
        return f / s, 1.0
    if kind == "base":
        return (L(base) * s ** (L(rd) / (rd - 2))) ** (-i / rd), 1.0
    n = L(scaling["original"])
    if kind == "bands":
        turns = n * f / two_pi
        out = []
        for fi, t in zip(f, turns):
            if t <= scaling["low"]:
                out.append(fi / s)
            elif t >= scaling["high"]:
                out.append(fi)
            else:
                keep = (t - L(scaling["low"])) / (L(scaling["high"]) - L(scaling["low"]))
                out.append((1 - keep) * fi / s + keep * fi)
        return np.array(out), 1.0
    assert kind == "ramp"

    def index(turns):  # the (fractional) pair that makes this many turns in the original length
        return float(rd * np.log(n / (turns * two_pi)) / (2 * np.log(L(base))))
    lo, hi = max(np.floor(index(scaling["fast"])), 0), min(np.ceil(index(scaling["slow"])), rd - 1)
    slow = np.clip((np.arange(rd // 2) - lo) / max(hi - lo, 1e-3), 0, 1).astype(L)
    return f * (1 - slow) + f / s * slow, 0.1 * float(np.log(s)) + 1.0


def rope(x, positions, f, scale, rd, interleaved, inverse):
    """x [M, heads, hd] -> (turned, magnitude), positions [M] (python or numpy integers)."""
    x = _f64(x)
    two_pi = np.longdouble("6.283185307179586476925286766559")
    turns = np.array([int(p) for p in positions], dtype=np.longdouble)[:, None] * (f / two_pi)
    angle = ((turns - np.floor(turns)) * two_pi).astype(np.float64)[:, None, :]
    c, s = np.cos(angle) * scale, np.sin(angle) * scale * (-1 if inverse else 1)
    first, second = (slice(0, rd, 2), slice(1, rd, 2)) if interleaved else \
        (slice(0, rd // 2), slice(rd // 2, rd))
    a, b = x[..., first], x[..., second]
    out, mag = x.copy(), np.zeros_like(x)
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    mag[..., first] = mag[..., second] = (np.abs(a) + np.abs(b)) * abs(scale)
    return out, mag
