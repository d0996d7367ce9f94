"""New tokens into the paged latent cache on the GPU, against the 64-bit definition within
derived bounds."""
import numpy as np
import pytest
import torch

from bounds import DT, check, f64, half_step, norm_rope_bounds
from oracle import operators as ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(lens, H, Sq, rank, dtype, bs, norm=True, seed=0, spare=3):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    per = [-(-max(n, 0) // bs) for n in lens]
    nb = sum(per) + spare
    r = lambda *s: torch.randn(*s, generator=g).to(DT[dtype])
    perm = torch.randperm(nb, generator=g)
    table = torch.full((B, max(max(per), 1)), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(per):
        table[b, :m] = perm[at: at + m]
        at += m
    down = r(B, Sq, rank + 64)
    q = r(B, Sq, H, 128 + 64)[..., 128:].transpose(1, 2)
    return dict(latent=down[..., :rank], k_rope=down[..., rank:], q_rope=q, cache=r(nb, bs, rank + 64),
                block_table=table, seq_lens=torch.tensor(lens, dtype=torch.int32),
                weight=(1 + 0.2 * torch.randn(rank, generator=g)).to(DT[dtype]) if norm else None)


def run(fa, x, turns, **kw):
    d = {n: None if t is None else t.to(DEV) for n, t in x.items()}
    kw = {n: v.to(DEV) if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    q = fa.latent_append(turns=turns.to(DEV), **d, **kw)
    torch.cuda.synchronize()
    return dict(q_out=q, cache=d["cache"])


def compare(got, x, inv_freq, interleaved=False, rope_scale=1.0, positions=None, eps=1e-6):
    u = half_step(x["latent"].dtype)
    B, Sq, rank = x["latent"].shape
    bs = x["cache"].shape[1]
    rows = x["seq_lens"].numpy().astype(np.int64)[:, None] - Sq + np.arange(Sq)
    pos = rows if positions is None else positions.numpy()
    f = f64(inv_freq)
    q = f64(x["q_rope"])
    check("q_out", got["q_out"], ops.norm_rope(q, None, f, pos, 0.0, interleaved, rope_scale),
          norm_rope_bounds(q, None, f, pos, u, 0.0, interleaved, rope_scale))
    kr, lat = f64(x["k_rope"])[:, None], f64(x["latent"])[:, None]
    w = None if x["weight"] is None else f64(x["weight"])
    none = np.zeros(0)
    kr_t = norm_rope_bounds(kr, None, f, pos, u, 0.0, interleaved, rope_scale)
    kr = ops.norm_rope(kr, None, f, pos, 0.0, interleaved, rope_scale)
    lat_t = norm_rope_bounds(lat, w, none, pos, u, eps, False, 1.0)
    lat = ops.norm_rope(lat, w, none, pos, eps, False, 1.0)
    want = f64(x["cache"])
    tol = np.zeros_like(want)
    for b in range(B):
        for s in range(Sq):
            p = rows[b, s]
            if p < 0 or p // bs >= x["block_table"].shape[1]:
                continue
            page = int(x["block_table"][b, p // bs])
            if 0 <= page < want.shape[0]:
                want[page, p % bs] = np.concatenate((lat[b, 0, s], kr[b, 0, s]))
                tol[page, p % bs] = np.concatenate((lat_t[b, 0, s], kr_t[b, 0, s]))
    check("cache", got["cache"], want, tol)     # the rest stays as it was, bit by bit


CASES = [
    # lens, H, Sq, rank, dtype, block, norm, interleaved
    ([1], 1, 1, 256, "bf16", 16, True, False),
    ([1, 40, 33], 16, 1, 512, "bf16", 16, True, True),
    ([5, 17, 64], 5, 3, 512, "fp16", 32, True, False),
    ([2, 0, 300], 128, 4, 512, "bf16", 64, False, True),      # tokens before the first row
    ([300, 201], 3, 200, 256, "fp32", 16, True, False),
    ([70, 64], 7, 64, 512, "fp32", 1024, False, True),
    ([500] * 3, 20, 100, 256, "fp16", 64, True, True),
]


@pytest.mark.parametrize("lens,H,Sq,rank,dtype,bs,norm,interleaved", CASES)
def test_append(fa, lens, H, Sq, rank, dtype, bs, norm, interleaved):
    x = make(lens, H, Sq, rank, dtype, bs, norm, len(lens) + H)
    f, scale = fa.rope_inv_freq(64, scaling="parts", factor=4.0)
    got = run(fa, x, fa.rope_turns(f), interleaved=interleaved, rope_scale=scale)
    compare(got, x, f, interleaved, scale)


MANY = [
    # from 608 tokens on a block takes four of them: here 1, 2, 3 or none over, of two sequences or with one
    # token of each, heads in one unit, in several, and past a multiple of eight
    (3, 205, 7, 512, "fp16", 16, True, True),        # 615: 3 over
    (2, 305, 16, 256, "bf16", 64, False, False),     # 610: 2 over
    (7, 87, 1, 512, "fp32", 32, True, False),        # 609: 1 over
    (4, 152, 8, 256, "fp32", 16, False, True),       # 608, none
    (611, 1, 9, 256, "fp16", 16, True, False),       # sequences of one token
    (1, 1025, 40, 512, "bf16", 256, True, True),
]


@pytest.mark.parametrize("B,Sq,H,rank,dtype,bs,norm,interleaved", MANY)
def test_append_of_many_tokens(fa, B, Sq, H, rank, dtype, bs, norm, interleaved):
    """Some of them not stored: before their sequence's start, past the table, in pages outside."""
    lens = [Sq + (37 * b) % 23 for b in range(B)]
    lens[B // 2] = Sq - min(Sq, 3)
    x = make(lens, H, Sq, rank, dtype, bs, norm, B + Sq)
    x["seq_lens"][-1] += bs
    x["block_table"][0, 0] = x["cache"].shape[0]
    f, scale = fa.rope_inv_freq(64, scaling="parts", factor=4.0)
    compare(run(fa, x, fa.rope_turns(f), interleaved=interleaved, rope_scale=scale), x, f, interleaved, scale)
    g = torch.Generator().manual_seed(B)
    pos = torch.randint(-2 ** 31, 2 ** 31, (B, Sq), generator=g).to(torch.int32)
    compare(run(fa, x, fa.rope_turns(f), interleaved=interleaved, positions=pos), x, f, interleaved, positions=pos)


@pytest.mark.parametrize("dtype,rank", [("fp32", 256), ("fp16", 512), ("bf16", 512)])
def test_many_tokens_at_once_or_a_few_at_a_time(fa, dtype, rank):
    """The same bits, whichever form a call takes."""
    B, Sq, H = 3, 250, 11
    x = make([Sq + 5, Sq, Sq + 40], H, Sq, rank, dtype, 16, True, 5)
    f, _ = fa.rope_inv_freq(64)
    want = run(fa, x, fa.rope_turns(f))
    d = {n: t.to(DEV) for n, t in x.items()}
    turns, parts = fa.rope_turns(f).to(DEV), []
    for a, b in ((0, 1), (1, 100), (100, 249), (249, 250)):
        part = {n: d[n][:, a:b] for n in ("latent", "k_rope")}
        parts.append(fa.latent_append(**part, q_rope=d["q_rope"][:, :, a:b], cache=d["cache"], turns=turns,
                                      block_table=d["block_table"], seq_lens=d["seq_lens"] - (Sq - b), weight=d["weight"]))
    assert torch.equal(torch.cat(parts, 2), want["q_out"]) and torch.equal(d["cache"], want["cache"])


def test_positions(fa):
    """Drafted tokens stand at their depth, wherever their rows are; far and negative positions."""
    x = make([20, 1000], 4, 8, 512, "bf16", 16)
    _, depth = fa.tree_masks([[-1, 0, 0, 1, 1, 2, 5, 6]] * 2)
    pos = x["seq_lens"][:, None] - 8 + depth
    pos[0, 3], pos[1, 7] = 2 ** 31 - 1, -5
    f, _ = fa.rope_inv_freq(64)
    compare(run(fa, x, fa.rope_turns(f), positions=pos), x, f, positions=pos)


def test_tokens_that_are_not_stored(fa):
    """Lengths past the table, pages outside the cache: q_out is written, nothing else."""
    x = make([40, 40, 40], 4, 2, 256, "bf16", 16)
    x["seq_lens"] = torch.tensor([-(2 ** 31) + 1, 49, 40], dtype=torch.int32)
    x["block_table"][2, 2] = x["cache"].shape[0]
    f, _ = fa.rope_inv_freq(64)
    compare(run(fa, x, fa.rope_turns(f)), x, f)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_queries_in_place_and_as_part_of_the_absorbed(fa, dtype):
    x = make([30, 77], 6, 3, 512, dtype, 16)
    f, _ = fa.rope_inv_freq(64)
    turns = fa.rope_turns(f)
    want = run(fa, x, turns)["q_out"]
    absorbed = torch.full((2, 6, 3, 512 + 64), 3.0, dtype=DT[dtype], device=DEV)
    got = run(fa, x, turns, q_out=absorbed[..., 512:])["q_out"]
    assert torch.equal(got, want) and (absorbed[..., :512] == 3.0).all()
    d = {n: t.to(DEV) for n, t in x.items()}
    assert torch.equal(fa.latent_append(turns=turns.to(DEV), q_out=d["q_rope"], **d), want)


def test_zeros_keep_to_themselves(fa):
    """A latent of zeros gives zeros with eps = 0, an infinite query its own pair only."""
    x = make([16], 1, 1, 256, "bf16", 16)
    x["latent"] = torch.zeros_like(x["latent"])
    x["q_rope"] = torch.zeros_like(x["q_rope"])
    x["q_rope"][..., 3] = float("inf")
    f, _ = fa.rope_inv_freq(64)
    got = run(fa, x, fa.rope_turns(f), eps=0.0)
    page = int(x["block_table"][0, 0])
    assert (got["cache"][page, 15, :256] == 0).all()
    bad = ~got["q_out"].isfinite().flatten()
    assert set(bad.nonzero().flatten().tolist()) == {3, 35}
