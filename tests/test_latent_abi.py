"""Refusals of the latent attention entry points, without a GPU: the C ABI rejects bad arguments on
the host with the documented codes; workspace formulas; tree_masks."""
import ctypes
import math

import pytest
import torch

SHAPE, DTYPE, NULL, ALIGN, WORKSPACE, SCALE = -1, -2, -3, -4, -5, -7
P = 256   # an aligned address that is never read


def view(fa, data=P, sb=1 << 16, sh=128, ss=512):
    return ctypes.byref(fa._View(data, sb, sh, ss))


def views(fa, names, over):
    return [None if over.get(n, ()) is None else view(fa, **over.get(n, {})) for n in names]


def fwd(fa, begin=None, end=None, lse=P, B=2, H=3, Sq=9, Skv=7, d=64, scale=0.1, dtype=2, **over):
    q, k, kr, v, out = views(fa, ("q", "k", "k_rope", "v", "out"), over)
    return fa.lib().fa_fwd_latent(q, k, kr, v, begin, end, out, lse, B, H, Sq, Skv, d, scale, dtype, None)


def bwd(fa, begin=None, end=None, lse=P, B=2, H=3, Sq=9, Skv=7, d=64, scale=0.1, dtype=2, ws=P,
        ws_bytes=1 << 30, **over):
    q, k, kr, v, out, do = views(fa, ("q", "k", "k_rope", "v", "out", "dout"), over)
    grads = views(fa, ("dq", "dk", "dk_rope", "dv"), over)
    return fa.lib().fa_bwd_latent(q, k, kr, v, begin, end, out, do, lse, *grads, B, H, Sq, Skv, d,
                                  scale, dtype, ws, ws_bytes, None)


BAD = [
    (dict(d=96), SHAPE), (dict(Sq=0), SHAPE), (dict(Skv=0), SHAPE), (dict(H=0), SHAPE), (dict(B=0), SHAPE),
    (dict(B=1 << 20, H=1 << 11), SHAPE), (dict(dtype=0), DTYPE), (dict(dtype=7), DTYPE),
    (dict(scale=0.0), SCALE), (dict(scale=math.nan), SCALE), (dict(scale=-1.0), SCALE),
    (dict(begin=P), NULL), (dict(end=P), NULL), (dict(begin=P + 2, end=P), ALIGN), (dict(q=None), NULL),
    (dict(k_rope=None), NULL), (dict(out=dict(data=None)), NULL), (dict(lse=None), NULL),
    (dict(lse=P + 2), ALIGN), (dict(v=dict(data=P + 8)), ALIGN), (dict(k=dict(ss=12)), ALIGN),
    (dict(q=dict(sh=0)), SHAPE), (dict(v=dict(ss=-512)), SHAPE), (dict(out=dict(sb=0)), SHAPE),
    (dict(k_rope=dict(ss=1 << 40)), SHAPE),
]


@pytest.mark.parametrize("kw,code", BAD)
def test_forward_refuses(fa_lib, kw, code):
    assert fwd(fa_lib, **kw) == code


@pytest.mark.parametrize("kw,code", BAD + [
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE), (dict(ws=P + 16), ALIGN),
    (dict(dk_rope=None), NULL), (dict(dout=dict(sh=0)), SHAPE), (dict(dq=dict(data=P + 4)), ALIGN)])
def test_backward_refuses(fa_lib, kw, code):
    assert bwd(fa_lib, **kw) == code


def test_backward_workspace_formula(fa_lib):
    up = lambda x: -(-x // 256) * 256
    for B, H, Sq, Skv, d in [(1, 1, 1, 1, 64), (2, 16, 2999, 2999, 128), (3, 5, 129, 1000, 64)]:
        rows = -(-Sq // 128) * 128
        want = 2 * up(B * H * rows * 4) + up(B * rows // 64 * 8) + B * H * Skv * 64 * 4
        assert fa_lib.fa_bwd_latent_workspace_bytes(B, H, Sq, Skv, d) == want
    assert fa_lib.fa_bwd_latent_workspace_bytes(1, 1, 1, 1, 80) == 0


def paged(fa, cache=P, table=P, lens=P, tree=None, out=P, lse=P, B=2, H=8, Sq=2, rank=512, bs=16, nb=10,
          mb=4, window=0, scale=0.1, dtype=1, ws=P, ws_bytes=1 << 30, **over):
    q, = views(fa, ("q",), over)
    return fa.lib().fa_fwd_latent_paged(q, cache, table, lens, tree, out, lse, B, H, Sq, rank, bs, nb, mb,
                                        window, scale, dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rank=128), SHAPE), (dict(B=0), SHAPE), (dict(H=0), SHAPE), (dict(Sq=0), SHAPE),
    (dict(H=129, Sq=8), SHAPE), (dict(bs=8), SHAPE), (dict(bs=2048), SHAPE), (dict(bs=48), SHAPE),
    (dict(nb=0), SHAPE), (dict(mb=0), SHAPE), (dict(B=1 << 20, mb=1 << 14), SHAPE), (dict(window=-1), SHAPE),
    (dict(tree=P, window=5), SHAPE), (dict(tree=P, H=2, Sq=65), SHAPE), (dict(dtype=0), DTYPE),
    (dict(dtype=9), DTYPE), (dict(scale=-1.0), SCALE), (dict(scale=math.inf), SCALE), (dict(table=None), NULL),
    (dict(lens=None), NULL), (dict(cache=None), NULL), (dict(q=None), NULL), (dict(out=None), NULL),
    (dict(table=P + 2), ALIGN), (dict(tree=P + 4), ALIGN), (dict(cache=P + 8), ALIGN), (dict(q=dict(ss=4)), ALIGN),
    (dict(q=dict(ss=0)), SHAPE), (dict(ws=None), WORKSPACE), (dict(ws_bytes=64), WORKSPACE),
    (dict(ws=P + 32), ALIGN)])
def test_paged_refuses(fa_lib, kw, code):
    assert paged(fa_lib, **kw) == code


def test_paged_workspace_formula(fa_lib):
    up = lambda x: -(-x // 256) * 256
    for (B, H, Sq, rank, bs, mb), groups in [((1, 1, 1, 256, 16, 1), 1), ((16, 128, 1, 512, 64, 128), 2),
                                             ((2, 128, 8, 512, 16, 20), 16), ((4, 20, 3, 512, 64, 9), 1),
                                             ((4, 22, 3, 512, 64, 9), 2), ((1, 7, 130, 256, 64, 9), 21),
                                             ((1, 31, 33, 256, 64, 90), 31)]:
        shares = min(152 // groups, B * -(-(mb * bs) // 64))
        rows = 2 * shares * H * Sq
        want = up(rows * rank * 4) + up(rows * 4) + up(16 * shares)
        assert fa_lib.fa_fwd_latent_paged_workspace_bytes(B, H, Sq, rank, bs, mb) == want
    assert fa_lib.fa_fwd_latent_paged_workspace_bytes(1, 1, 1, 500, 16, 1) == 0


def append(fa, cache=P, table=P, lens=P, positions=None, weight=None, eps=1e-6, turns=P, rope_scale=1.0, B=2,
           H=3, Sq=2, rank=256, bs=16, nb=10, mb=4, dtype=2, **over):
    vs = views(fa, ("latent", "k_rope", "q_rope", "q_out"), over)
    return fa.lib().fa_latent_append(*vs, cache, table, lens, positions, weight, eps, turns, 0, rope_scale, B, H,
                                     Sq, rank, bs, nb, mb, dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rank=576), SHAPE), (dict(B=0), SHAPE), (dict(H=0), SHAPE), (dict(Sq=0), SHAPE), (dict(bs=20), SHAPE),
    (dict(nb=0), SHAPE), (dict(mb=0), SHAPE), (dict(B=1 << 20, Sq=1 << 12), SHAPE), (dict(dtype=3), DTYPE),
    (dict(rope_scale=math.nan), SCALE), (dict(weight=P, eps=-1.0), SCALE), (dict(weight=P, eps=math.inf), SCALE),
    (dict(latent=None), NULL), (dict(q_out=None), NULL), (dict(turns=None), NULL), (dict(cache=None), NULL),
    (dict(lens=None), NULL), (dict(turns=P + 4), ALIGN), (dict(weight=P + 2), ALIGN), (dict(positions=P + 2), ALIGN),
    (dict(latent=dict(ss=4)), ALIGN), (dict(dtype=0, latent=dict(ss=2)), ALIGN), (dict(q_rope=dict(sb=0)), SHAPE),
    (dict(cache=P + 8), ALIGN)])
def test_append_refuses(fa_lib, kw, code):
    assert append(fa_lib, **kw) == code


def test_tree_masks(fa_lib):
    masks, depths = fa_lib.tree_masks([[-1, 0, 0, 1], [-1, -1, 1, 0]])
    assert masks.tolist() == [[1, 3, 5, 11], [1, 2, 6, 9]]
    assert depths.tolist() == [[0, 1, 1, 2], [0, 0, 1, 1]]
    masks, depths = fa_lib.tree_masks(list(range(-1, 63)))
    assert masks[0, 63] == -1 and masks[0, 62] == 2 ** 63 - 1 and depths[0, 63] == 63
    for bad in ([0], [-1, 1], [-2], [], list(range(-1, 64)), torch.zeros(2, 2, 2)):
        with pytest.raises(ValueError):
            fa_lib.tree_masks(bad)


def test_binding_wants_cuda_tensors(fa_lib):
    z = torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa_lib.attention_latent_forward(z, z[..., :64], z[:, 0, :, :64], z[..., :64])
