"""64-bit CPU versions, from the definitions, of the operators around causal attention: span
attention (any key range per row, capped scores, distance bias) with its gradients, new tokens
over a paged cache, and per-head norm with rotary positions. Slow and plain; independent of the
CUDA path.

The attention functions also return error bounds. A 16-bit kernel rounds P (and dS) to its type
and its outputs once; `u` is half a step of that type relative to the value. With E_ij the
absolute error of a score in fp32 (accumulation of the dot product, cap, bias and exponent
arithmetic), the bounds follow term by term:

    |d out|  <= (u + 2 E) P |V| + u |out|
    |d dV|   <= (u + 2 E)^T P^T |dO| + u |dV|
    |d dS|   <= (3 u + 2 E) |dS| + P f (|dO| . |d out|)       f the cap's derivative; D is formed
                                                             from the rounded out
    |d dQ|   <= scale |d dS| |K| + u |dQ|,   |d dK| likewise
"""
from __future__ import annotations

import math

import numpy as np

F32 = 2.0 ** -24


def score_parts(q, k, scale, softcap=0.0, slope=0.0, offset=None):
    """One head's scores [Sq, Skv] before the mask, the cap's derivative, and a bound of their
    fp32 error."""
    Sq, Skv, d = q.shape[0], k.shape[0], q.shape[1]
    s = scale * (q @ k.T)
    err = (d + 8) * F32 * scale * (np.abs(q) @ np.abs(k).T)
    f = np.ones_like(s)
    if softcap:
        t = np.tanh(s / softcap)
        s, f = softcap * t, 1.0 - t * t
        err = err + softcap * 2.0 ** -20       # 1 - 2 / (1 + e^2x): a few fp32 steps of 1
    if slope:
        offset = Skv - Sq if offset is None else offset
        dist = np.abs(np.arange(Sq)[:, None] + offset - np.arange(Skv)[None, :])
        s = s - slope * dist
        err = err + 4 * F32 * np.abs(slope * dist)
    # scaling to base 2, subtracting the maximum, the exponential itself
    err = err + 8 * F32 * (np.abs(s) + np.abs(s).max(initial=0.0) + 1.0)
    return s, f, err


def span_head(q, k, v, begin, end, scale, softcap=0.0, slope=0.0, dout=None, u=0.0, offset=None):
    """One (query head, key/value head) pair: dict of out, lse, their bounds out_tol, lse_tol
    and, given dout, dq, dk, dv and theirs."""
    Sq, Skv = q.shape[0], k.shape[0]
    s, f, err = score_parts(q, k, scale, softcap, slope, offset)
    j = np.arange(Skv)
    ok = (j >= np.maximum(begin, 0)[:, None]) & (j < np.minimum(end, Skv)[:, None])
    s = np.where(ok, s, -np.inf)
    err = np.where(ok, err, 0.0)
    any_ok = ok.any(axis=1)
    m = np.where(any_ok, s.max(axis=1, initial=-np.inf), 0.0)
    e = np.exp(s - m[:, None])
    l = e.sum(axis=1)
    p = e / np.where(any_ok, l, 1.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(any_ok, m + np.log(np.where(any_ok, l, 1.0)), -np.inf)
    out = p @ v
    # fp16 probabilities below its smallest normal step: absolute 2^-25 of a sum >= 1
    tiny = Skv * 2.0 ** -25 * np.abs(v).max(initial=0.0) if u < 2.0 ** -9 else 0.0
    out_tol = (p * (u + 2 * err)) @ np.abs(v) + u * np.abs(out) * 1.01 + tiny * 1.01 + 1e-30
    lse_tol = 2 * err.max(axis=1, initial=0.0) + 4 * F32 * np.abs(np.where(any_ok, lse, 0.0)) + 1e-7
    res = dict(out=out, lse=lse, out_tol=out_tol, lse_tol=lse_tol)
    if dout is None:
        return res
    dp = dout @ v.T
    D = (dout * out).sum(axis=1, keepdims=True)
    ds = p * f * (dp - D)
    d_tol = (np.abs(dout) * out_tol).sum(axis=1, keepdims=True)
    dp_tol = (q.shape[1] + 8) * F32 * (np.abs(dout) @ np.abs(v).T)
    ds_tol = (3 * u + 2 * err) * np.abs(ds) * 1.02 + p * f * (d_tol + dp_tol) * 1.02
    if u < 2.0 ** -9:       # fp16: probabilities and dS below its smallest normal step
        ds_tol = ds_tol + np.where(ok, 2.0 ** -25 * (np.abs(dp) + np.abs(D) + 1.0), 0.0)
    acc = (Sq + Skv) * F32   # fp32 sums over rows or keys
    dq, dk, dv = scale * ds @ k, scale * ds.T @ q, p.T @ dout
    aq, ak = np.abs(q), np.abs(k)
    sub = 2.0 ** -25 if u < 2.0 ** -9 else 0.0
    res.update(
        dq=dq, dk=dk, dv=dv,
        dq_tol=scale * (ds_tol + acc * np.abs(ds)) @ ak + 1.01 * u * np.abs(dq) + sub + 1e-30,
        dk_tol=scale * (ds_tol + acc * np.abs(ds)).T @ aq + 1.01 * u * np.abs(dk) + sub + 1e-30,
        dv_tol=(p * (u + 2 * err + acc)).T @ np.abs(dout) + np.where(ok, sub, 0.0).T @ np.abs(dout)
        + 1.01 * u * np.abs(dv) + sub + 1e-30)
    return res


def span_attention(q, k, v, begin, end, scale, softcap=0.0, slopes=None, dout=None, u=0.0):
    """Every head of [B, Hq, Sq, d] queries; gradients of shared heads are summed."""
    B, Hq, Sq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out = {}

    def put(name, b, h, x, add=False):
        shape = (B, Hkv if name[:2] in ("dk", "dv") else Hq) + x.shape
        a = out.setdefault(name, np.zeros(shape))
        a[b, h] = a[b, h] + x if add else x

    for b in range(B):
        for h in range(Hq):
            r = span_head(q[b, h], k[b, h // G], v[b, h // G], begin[b], end[b], scale, softcap,
                          0.0 if slopes is None else float(slopes[h]),
                          None if dout is None else dout[b, h], u)
            for name, x in r.items():
                shared = name[:2] in ("dk", "dv")
                put(name, b, h // G if shared else h, x, add=shared)
    return out


def ragged_attention(q, k_cache, v_cache, block_table, seq_lens, scale, window=0, softcap=0.0,
                     slopes=None, u=0.0):
    """New tokens q [B, Hq, Sq, d] over pages [num_blocks, Hkv, block_size, d]."""
    B, Hq, Sq, d = q.shape
    nb, Hkv, bs = k_cache.shape[:3]
    G = Hq // Hkv
    res = {n: np.zeros((B, Hq, Sq, d)) for n in ("out", "out_tol")}
    res.update({n: np.full((B, Hq, Sq), -np.inf) for n in ("lse", "lse_tol")})
    for b in range(B):
        n = min(max(int(seq_lens[b]), 0), block_table.shape[1] * bs)
        pos = n - Sq + np.arange(Sq)
        end = np.maximum(pos + 1, 0)
        begin = np.maximum(end - window, 0) if window else np.zeros(Sq, int)
        first = max(0, n - Sq + 1 - window) if window else 0
        K, V = np.zeros((2, Hkv, n, d))
        for j in range(first, n):
            page = block_table[b, j // bs]
            if 0 <= page < nb:
                K[:, j], V[:, j] = k_cache[page, :, j % bs], v_cache[page, :, j % bs]
        for h in range(Hq):
            if n == 0:
                continue
            r = span_head(q[b, h], K[h // G], V[h // G], begin, end, scale, softcap,
                          0.0 if slopes is None else float(slopes[h]), u=u, offset=n - Sq)
            for name in res:
                res[name][b, h] = r[name]
    return res


def norm_rope(x, w, inv_freq, positions, eps=1e-6, interleaved=False, rope_scale=1.0, dy=None):
    """x [B, H, S, d], positions [B, S]: y, or given dy (dx, dw)."""
    d, half = x.shape[-1], len(inv_freq)
    a = np.zeros((len(positions), positions.shape[1], half))
    for i, f in enumerate(inv_freq):    # whole turns removed in extended precision
        turns = positions.astype(np.longdouble) * (np.longdouble(f) / (2 * np.longdouble(math.pi)))
        a[..., i] = 2 * math.pi * (turns - np.round(turns)).astype(np.float64)
    c, s = rope_scale * np.cos(a)[:, None], rope_scale * np.sin(a)[:, None]
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)

    def turn(z, s):
        y = z.copy()
        y[..., ia] = c * z[..., ia] - s * z[..., ib]
        y[..., ib] = s * z[..., ia] + c * z[..., ib]
        return y

    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if dy is None:
        return turn(x if w is None else x * r * w, s)
    dn = turn(dy, -s)
    if w is None:
        return dn, None
    g = dn * w
    return r * (g - x * r * r * (g * x).mean(-1, keepdims=True)), (dn * x * r).sum((0, 1, 2))
