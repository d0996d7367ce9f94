"""Query/key preparation at the edges of its arguments."""
import math

import numpy as np
import pytest
import torch

from bounds import check, f64, half_step, norm_rope_bounds
from oracle import operators as ops
from test_gpu_heads import cache, freqs, make

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (64, "fp32")])
def test_infinite_gradient_past_the_rotated_part_stays_where_it_is(fa, interleaved, d, dtype):
    """There y = x, so dx = dy, element by element."""
    q, k, _, _ = make(1, 2, 1, 5, d, dtype, False, "packed", 8)
    turns = fa.rope_turns(freqs(32), DEV)
    dy = [torch.randn_like(t.contiguous()) for t in (q, k)]
    clean = fa.qk_norm_rope_backward(*dy, q, k, turns, interleaved=interleaved)
    for t in (dy[0], clean[0]):
        t[0, 1, 3, 40] = float("inf")
    for t in (dy[1], clean[1]):
        t[0, 0, 2, 63] = float("-inf")
    got = fa.qk_norm_rope_backward(*dy, q, k, turns, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_phases_between_two_steps(fa, interleaved):
    """A phase is taken to the nearest of 2^32 steps a turn: angles this small come out to half
    such a step (2 pi 2^-33), both ways, on either side of zero."""
    F = 2.0 ** -24
    turns = [int((n + f) * 2 ** 32) for n, f in ((0, 0.99), (0, 0.51), (0, 0.3), (3, 0.999),
                                                 (-1, 0.4), (-1, 0.01), (-5, 0.75), (7, 0.25))]
    t = 2 * math.pi * np.array(turns, dtype=np.float64) * 2.0 ** -64
    i = np.arange(8)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + 8)
    q, k = torch.zeros(1, 1, 2, 64, device=DEV), torch.zeros(1, 1, 2, 64, device=DEV)
    q[..., ia] = 1.0       # sin t appears alone in the pairs' second elements
    k[..., ib] = 1.0       # and -sin t in their first
    table = torch.tensor(turns, dtype=torch.int64, device=DEV)
    yq, yk = fa.qk_norm_rope_forward(q, k, table, interleaved=interleaved)
    dq, dk = fa.qk_norm_rope_backward(q, k, None, None, table, interleaved=interleaved)[:2]
    torch.cuda.synchronize()
    tol = 2 * math.pi * 2.0 ** -33 + 4 * F * np.abs(t)
    for y, at, want in ((yq, ib, np.sin(t)), (yk, ia, -np.sin(t)), (dq, ib, -np.sin(t)),
                        (dk, ia, np.sin(t))):
        off = np.abs(f64(y)[0, 0, 1][at] - want)       # row 1 stands at position 1
        assert (off <= tol).all(), off / tol


def test_append_at_the_least_length(fa):
    """Row s of a sequence of -2^31 tokens stands before the cache, at -2^31 - Sq + s: nothing is
    stored, however long the table, and q is rotated by that position."""
    q, k, v, w = make(2, 2, 1, 2, 64, "bf16", True, "packed", 9)
    kc, vc = cache(2, 1, 1024, 64, "bf16"), cache(2, 1, 1024, 64, "bf16")
    lens = [-2 ** 31, -2 ** 31 + 1]
    table = torch.zeros(2, 1 << 21, dtype=torch.int32, device=DEV)
    f = freqs(64)
    got = fa.qk_norm_rope_append(q, k, v, kc, vc, table,
                                 torch.tensor(lens, dtype=torch.int32, device=DEV),
                                 fa.rope_turns(f, DEV), q_weight=w[0], k_weight=w[1])
    torch.cuda.synchronize()
    assert (kc == 9.0).all() and (vc == 9.0).all()
    a = dict(inv_freq=f, positions=np.array(lens)[:, None] - 2 + np.arange(2), eps=1e-6,
             interleaved=False, rope_scale=1.0)
    check("q", got, ops.norm_rope(f64(q), f64(w[0]), **a),
          norm_rope_bounds(f64(q), f64(w[0]), u=half_step(q.dtype), **a))
