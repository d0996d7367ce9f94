"""Element-wise comparison against bounds that are derived, not chosen: see oracle/operators.py
for attention; `norm_rope_bounds` for the query/key preparation."""
import math

import numpy as np
import torch

from oracle import operators as ops

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half_step(dtype):
    """Half a step of a type, relative to the value."""
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def check(name, got, want, tol):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fin = np.isfinite(want)
    assert (np.isfinite(got) == fin).all() and (got[~fin] == want[~fin]).all(), name
    off, tol = np.abs(got[fin] - want[fin]), np.broadcast_to(tol, want.shape)[fin]
    assert (off <= tol).all(), f"{name}: {(off / np.maximum(tol, 1e-300)).max():.3g} of its bound"


def norm_rope_bounds(x, w, inv_freq, positions, u, eps, interleaved, rope_scale, dy=None):
    """Bound of y, or given dy of (dx, dw). fp32 arithmetic in units of F = 2^-24: the mean of
    squares adds d / 8 + 8 positive terms in any order and the root is off by two steps; an angle
    is off by half a step of a phase of at most half a turn (pi F), by the table's 2^-53 of the
    frequency times the position, and the phase's 32 bits (2 pi 2^-33); sin, cos and the products
    take a few steps more."""
    F, d, half = ops.F32, x.shape[-1], len(inv_freq)
    e_norm = 0.0 if w is None else (d / 8 + 20) * F
    ang = np.zeros(x.shape[:1] + (1,) + x.shape[2:])
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    per = np.abs(positions.astype(np.float64))[:, None, :, None] * np.asarray(inv_freq) * 2.0 ** -51
    ang[..., ia] = ang[..., ib] = per + math.pi * F + 2.0 ** -30 + 8 * F

    def turned(z, dz):
        """Bound of a rotation of z, known to dz."""
        m, dm = np.abs(z), dz.copy()
        pair, dpair = m.copy(), dz.copy()
        pair[..., ia] = pair[..., ib] = rope_scale * (m[..., ia] + m[..., ib])
        dpair[..., ia] = dpair[..., ib] = rope_scale * (dm[..., ia] + dm[..., ib])
        return pair * ang + dpair

    small = 2.0 ** -25 if 2.0 ** -12 < u < 2.0 ** -9 else 1e-38
    if dy is None:
        r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        n = x if w is None else x * r * w
        y = ops.norm_rope(x, w, inv_freq, positions, eps, interleaved, rope_scale)
        return turned(n, np.abs(n) * e_norm) + 1.01 * u * np.abs(y) + small
    dx, dw = ops.norm_rope(x, w, inv_freq, positions, eps, interleaved, rope_scale, dy)
    ddn = turned(dy, np.zeros_like(dy))
    if w is None:
        return ddn + 1.01 * u * np.abs(dx) + small, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dn = ops.norm_rope(dy, None, inv_freq, -positions, 0.0, interleaved, rope_scale)
    g, dg, ax = np.abs(dn * w), ddn * np.abs(w), np.abs(x)
    mean = lambda a: a.mean(-1, keepdims=True)
    tol = r * (dg + ax * r * r * mean(dg * ax)) \
        + 3 * e_norm * r * (g + ax * r * r * mean(g * ax)) + 1.01 * u * np.abs(dx) + small
    n = x.size // d
    dw_tol = (ddn * ax * r).sum((0, 1, 2)) + (e_norm + (n / 8 + 96) * F) * \
        (np.abs(dn) * ax * r).sum((0, 1, 2)) + 1e-38
    return tol, dw_tol
