"""The 64-bit versions of the span, ragged and query/key-preparation operators against
differences, against the causal oracle and against closed forms (CPU)."""
import math

import numpy as np
import pytest

import oracle
from oracle import operators as ops


def rng_inputs(seed, Sq, Skv, d=8):
    r = np.random.default_rng(seed)
    return r.normal(size=(Sq, d)), r.normal(size=(Skv, d)), r.normal(size=(Skv, d)), \
        r.normal(size=(Sq, d))


@pytest.mark.parametrize("softcap,slope", [(0.0, 0.0), (1.5, 0.0), (0.0, 0.3), (2.0, 0.1)])
def test_span_gradients_match_differences(softcap, slope):
    q, k, v, do = rng_inputs(3, 5, 7)
    begin, end = np.array([0, 2, 3, -4, 0]), np.array([3, 2, 7, 99, 1])   # row 1 sees nothing
    f = lambda q, k, v: (ops.span_head(q, k, v, begin, end, 0.4, softcap, slope)["out"] * do).sum()
    got = ops.span_head(q, k, v, begin, end, 0.4, softcap, slope, dout=do)
    h = 1e-6
    for name, args, at in (("dq", (q, k, v), 0), ("dk", (q, k, v), 1), ("dv", (q, k, v), 2)):
        num = np.zeros_like(args[at])
        for i in np.ndindex(num.shape):
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[at][i] += h
            lo[at][i] -= h
            num[i] = (f(*hi) - f(*lo)) / (2 * h)
        # central differences: third derivative times h^2 and rounding 1e-16 / h
        assert np.abs(num - got[name]).max() < 1e-7, name
    assert (got["out"][1] == 0).all() and got["lse"][1] == -np.inf and (got["dq"][1] == 0).all()


def test_causal_spans_are_the_causal_oracle():
    r = np.random.default_rng(1)
    q, do = r.normal(size=(2, 2, 4, 9, 8))
    k, v = r.normal(size=(2, 2, 2, 13, 8))
    end = np.broadcast_to(np.arange(9) + 5, (2, 9))
    got = ops.span_attention(q, k, v, end * 0, end, 0.3, dout=do)
    out, lse = oracle.forward(q, k, v, True, 0.3)
    grads = oracle.backward(q, k, v, do, True, 0.3)
    for a, b in zip((got["out"], got["lse"], got["dq"], got["dk"], got["dv"]), (out, lse, *grads)):
        assert np.abs(a - b).max() < 1e-12


def test_ragged_pages_are_spans_of_gathered_keys():
    r = np.random.default_rng(2)
    lens, Sq, bs, W = [5, 0, 17, 2], 3, 4, 6
    q = r.normal(size=(4, 2, Sq, 8))
    kc, vc = r.normal(size=(2, 30, 1, bs, 8))
    table = np.full((4, 5), -1)
    perm = r.permutation(30)
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // bs)
        table[b, :m], at = perm[at: at + m], at + m
    got = ops.ragged_attention(q, kc, vc, table, lens, 0.5, window=W)
    for b, n in enumerate(lens):
        for s in range(Sq):
            p = n - Sq + s
            keys = range(max(0, p + 1 - W), p + 1)
            if p < 0:
                assert (got["out"][b, :, s] == 0).all() and (got["lse"][b, :, s] == -np.inf).all()
                continue
            K = np.stack([kc[table[b, j // bs], 0, j % bs] for j in keys])
            V = np.stack([vc[table[b, j // bs], 0, j % bs] for j in keys])
            e = np.exp(0.5 * q[b, :, s] @ K.T)
            assert np.abs(got["out"][b, :, s] - e @ V / e.sum(1, keepdims=True)).max() < 1e-12


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope_gradients_match_differences(interleaved, norm):
    r = np.random.default_rng(4)
    x, dy = r.normal(size=(2, 1, 2, 3, 8))
    w = r.normal(size=8) if norm else None
    pos = np.array([[0, 5, -3]])
    kw = dict(inv_freq=[0.7, 0.01], positions=pos, eps=0.1, interleaved=interleaved, rope_scale=1.2)
    f = lambda x, w: (ops.norm_rope(x, w, **kw) * dy).sum()
    dx, dw = ops.norm_rope(x, w, dy=dy, **kw)
    h = 1e-6
    for i in np.ndindex(x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += h
        lo[i] -= h
        assert abs((f(hi, w) - f(lo, w)) / (2 * h) - dx[i]) < 1e-7
    if norm:
        for i in range(8):
            hi, lo = w.copy(), w.copy()
            hi[i] += h
            lo[i] -= h
            assert abs((f(x, hi) - f(x, lo)) / (2 * h) - dw[i]) < 1e-7


def test_rotation_keeps_relative_positions():
    """<R_p q, R_t k> depends on p - t only, however far the positions are."""
    r = np.random.default_rng(5)
    q, k = r.normal(size=(2, 1, 1, 1, 8))
    f = [1.0, 0.1, 0.01]
    dot = lambda p, t: (ops.norm_rope(q, None, f, np.array([[p]])) *
                        ops.norm_rope(k, None, f, np.array([[t]]))).sum()
    assert math.isclose(dot(7, 3), dot(2 ** 30 + 7, 2 ** 30 + 3), abs_tol=1e-8)
