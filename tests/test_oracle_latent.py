"""The 64-bit definitions of latent attention against dense formulas, each other and differences."""
import numpy as np
import pytest

import causal_flash_attention_gb300 as fa
from oracle import operators as ops


def data(B, H, Sq, Skv, d, seed):
    r = np.random.default_rng(seed).standard_normal
    return r((B, H, Sq, d + 64)), r((B, H, Skv, d)), r((B, Skv, 64)), r((B, H, Skv, d)), r((B, H, Sq, d))


def dense(q, k, kr, v, see, scale):
    """out, lse over see [B, Sq, Skv]."""
    keys = np.concatenate((k, np.broadcast_to(kr[:, None], k.shape[:3] + (64,))), -1)
    s = np.where(see[:, None], scale * np.einsum("bhid,bhjd->bhij", q, keys), -np.inf)
    with np.errstate(divide="ignore", invalid="ignore"):
        m = np.where(see.any(-1)[:, None], s.max(-1), 0.0)
        e = np.exp(s - m[..., None])
        lse = m + np.log(e.sum(-1))
        p = np.where(np.isfinite(lse)[..., None], np.exp(s - np.where(np.isfinite(lse), lse, 0.0)[..., None]), 0.0)
    return np.einsum("bhij,bhjd->bhid", p, v), lse


def spans(B, Sq, Skv, seed):
    g = np.random.default_rng(seed)
    begin = g.integers(0, Skv, (B, Sq))
    end = np.minimum(begin + g.integers(0, Skv, (B, Sq)), Skv)
    end[:, 0] = begin[:, 0]      # sees nothing
    return begin, end


@pytest.mark.parametrize("B,H,Sq,Skv,d", [(2, 2, 5, 7, 4), (1, 3, 9, 4, 8), (1, 1, 1, 1, 2)])
def test_expanded_against_the_dense_formula(B, H, Sq, Skv, d):
    q, k, kr, v, _ = data(B, H, Sq, Skv, d, d)
    begin, end = spans(B, Sq, Skv, Sq)
    j = np.arange(Skv)
    see = (j >= begin[..., None]) & (j < end[..., None])
    out, lse = dense(q, k, kr, v, see, 0.3)
    got = ops.latent_attention(q, k, kr, v, begin, end, 0.3)
    assert np.allclose(got["out"], out, 1e-12, 1e-13)
    assert np.allclose(got["lse"][np.isfinite(lse)], lse[np.isfinite(lse)], 1e-12)
    assert (np.isfinite(got["lse"]) == np.isfinite(lse)).all() and (got["out"][:, :, 0] == 0).all()


def test_gradients_against_differences():
    x = data(1, 2, 6, 8, 4, 1)
    begin, end = spans(1, 6, 8, 2)
    got = ops.latent_attention(*x[:4], begin, end, 0.4, x[4])
    loss = lambda y: (ops.latent_attention(*y, begin, end, 0.4)["out"] * x[4]).sum()
    rng, h = np.random.default_rng(3), 1e-5
    for i, n in enumerate(("dq", "dk", "dk_rope", "dv")):
        way = rng.standard_normal(x[i].shape)
        y = [[a + s * h * way if j == i else a for j, a in enumerate(x[:4])] for s in (1, -1)]
        want = (loss(y[0]) - loss(y[1])) / (2 * h)
        assert abs((got[n] * way).sum() - want) < 1e-8 * (1 + abs(want)), n


@pytest.mark.parametrize("window,tree", [(0, False), (3, False), (0, True)])
def test_paged_is_the_expanded_form_with_latents_as_keys_and_values(window, tree):
    """Pages gathered by hand, every head's keys and values the rows themselves."""
    g = np.random.default_rng(5)
    B, H, Sq, rank, bs, lens = 3, 2, 3, 6, 4, [9, 2, 0]
    cache = g.standard_normal((7, bs, rank + 64))
    table = np.array([[5, 0, 2], [6, -1, 9], [1, 3, 4]])
    q = g.standard_normal((B, H, Sq, rank + 64))
    masks = fa.tree_masks([[-1, 0, 0], [-1, -1, 1], [-1, 0, 1]])[0].numpy() if tree else None
    got = ops.latent_paged(q, cache, table, lens, 0.2, window, masks)
    for b, n in enumerate(lens):
        if n == 0:
            assert (got["out"][b] == 0).all() and (got["lse"][b] == -np.inf).all()
            continue
        rows = np.stack([cache[table[b, j // bs], j % bs] for j in range(n)])
        see = np.zeros((Sq, n), bool)
        for s in range(Sq):
            for j in range(n):
                p, t = n - Sq + s, j - (n - Sq)
                see[s, j] = ((t < 0 or masks[b, s] >> t & 1) if tree else
                             j <= p and (not window or j > p - window))
        c = np.broadcast_to(rows[None, None, :, :rank], (1, H, n, rank))
        out, lse = dense(q[b:b + 1], c, rows[None, :, rank:], c, see[None], 0.2)
        assert np.allclose(got["out"][b], out[0], 1e-12, 1e-13)
        fin = np.isfinite(lse[0])
        assert (np.isfinite(got["lse"][b]) == fin).all() and np.allclose(got["lse"][b][fin], lse[0][fin], 1e-12)
