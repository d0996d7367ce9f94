"""Query/key preparation at the sizes of training, where a warp keeps a token to itself (8 tokens
a block, no block barrier) and the backward's blocks take several groups of tokens one after the
other; and the append of as many tokens."""
import numpy as np
import pytest
import torch

from bounds import check, f64, half_step, norm_rope_bounds
from oracle import operators as ops
from test_gpu_heads import cache, freqs, make, run_both

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("B,Hq,Hkv,S,d,dtype,rope_dim,interleaved,norm,layout", [
    # one warp a token from 2432 tokens (forward) and 1216 (backward); 304 blocks of 8 tokens are
    # one pass of the backward; no number here fills the last block
    (1, 4, 2, 2433, 64, "bf16", 64, False, True, "packed"),
    (1, 4, 2, 5001, 128, "bf16", 128, False, True, "packed"),
    (3, 4, 2, 1667, 64, "fp32", 64, True, True, "gap"),
    (1, 4, 2, 5001, 128, "fp32", 48, False, True, "heads_first"),
    (1, 4, 2, 5003, 128, "fp16", 128, True, False, "packed"),
    (7, 3, 1, 715, 64, "bf16", 32, False, False, "packed"),
    (1, 12, 3, 7295, 64, "fp16", 64, False, True, "gap"),
])
def test_forward_and_backward(fa, B, Hq, Hkv, S, d, dtype, rope_dim, interleaved, norm, layout):
    q, k, _, w = make(B, Hq, Hkv, S, d, dtype, norm, layout, S)
    r = np.random.default_rng(S)
    positions = torch.from_numpy(r.integers(0, 20000, (B, S)).astype(np.int32)).to(DEV)
    run_both(fa, q, k, w, freqs(rope_dim), positions, 1e-6, interleaved, 1.0)


@pytest.mark.parametrize("d", [64, 128])
def test_same_weight_gradients_again(fa, d):
    q, k, _, w = make(1, 8, 2, 5001, d, "bf16", True, "packed", 1)
    turns = fa.rope_turns(freqs(d), DEV)
    dy = [torch.randn_like(t.contiguous()) for t in (q, k)]
    first, again = (fa.qk_norm_rope_backward(*dy, q, k, turns, q_weight=w[0], k_weight=w[1])
                    for _ in range(2))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (64, "fp32")])
def test_append_of_many_tokens(fa, d, dtype):
    B, Hq, Hkv, Sq, bs, lens = 3, 4, 2, 1001, 32, [1001, 1500, 700]   # the last: 301 not stored
    q, k, v, w = make(B, Hq, Hkv, Sq, d, dtype, True, "packed", 2)
    f, per = freqs(d), -(-max(lens) // bs)
    table = torch.randperm(B * per, generator=torch.Generator().manual_seed(1))
    table = table.to(torch.int32).view(B, per)
    kc, vc = cache(B * per, Hkv, bs, d, dtype), cache(B * per, Hkv, bs, d, dtype)
    q_out = fa.qk_norm_rope_append(q, k, v, kc, vc, table.to(DEV),
                                   torch.tensor(lens, dtype=torch.int32, device=DEV),
                                   fa.rope_turns(f, DEV), q_weight=w[0], k_weight=w[1])
    torch.cuda.synchronize()
    pos = np.array(lens)[:, None] - Sq + np.arange(Sq)
    a = dict(inv_freq=f, positions=pos, eps=1e-6, interleaved=False, rope_scale=1.0)
    u, ws = half_step(q.dtype), [f64(t) for t in w]
    check("q", q_out, ops.norm_rope(f64(q), ws[0], **a), norm_rope_bounds(f64(q), ws[0], u=u, **a))
    want_k, tol_k = ops.norm_rope(f64(k), ws[1], **a), norm_rope_bounds(f64(k), ws[1], u=u, **a)
    K, T, V = np.full(kc.shape, 9.0), np.zeros(kc.shape), np.full(vc.shape, 9.0)
    for b, s in zip(*np.nonzero(pos >= 0)):
        at = (int(table[b, pos[b, s] // bs]), slice(None), pos[b, s] % bs)
        K[at], T[at], V[at] = want_k[b, :, s], tol_k[b, :, s], f64(v)[b, :, s]
    check("k_cache", kc, K, T + 1e-300)
    assert (f64(vc) == V).all()
