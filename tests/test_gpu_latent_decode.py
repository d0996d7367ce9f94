"""Absorbed latent attention over a paged cache on the GPU, against the 64-bit definition within
derived bounds."""
import pytest
import torch

from bounds import DT, check, f64, half_step
from oracle import operators as ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SCALE = (128 + 64) ** -0.5


def make(lens, H, Sq, rank, dtype, bs, seed=0, scale_q=0.5, max_blocks=None, spare=4, fill=None):
    """q, cache, table, lengths; rows of the cache that no sequence holds are `fill`."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    per = [-(-max(n, 0) // bs) for n in lens]
    nb = sum(per) + spare
    cache = torch.randn(nb, bs, rank + 64, generator=g)
    perm = torch.randperm(nb, generator=g)
    table = torch.full((B, max_blocks or max(max(per), 1)), -1, dtype=torch.int32)
    used, at = torch.zeros(nb, bs, dtype=torch.bool), 0
    for b, m in enumerate(per):
        table[b, :m] = perm[at: at + m]
        at += m
        for j in range(max(lens[b], 0)):
            used[table[b, j // bs], j % bs] = True
    if fill is not None:
        cache[~used] = fill
    q = torch.randn(B, H, Sq, rank + 64, generator=g) * scale_q
    return [q.to(DT[dtype]), cache.to(DT[dtype]), table, torch.tensor(lens, dtype=torch.int32)]


def run(fa, x, **kw):
    kw = {n: v.to(DEV) if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    out, lse = fa.decode_latent_paged(*(t.to(DEV) for t in x), SCALE, **kw)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == 0
    return dict(out=out, lse=lse)


def compare(got, x, window=0, tree_masks=None):
    q, cache, table, lens = x
    want = ops.latent_paged(f64(q), f64(cache), table.numpy(), lens.tolist(), SCALE, window,
                            None if tree_masks is None else tree_masks.numpy(), half_step(q.dtype))
    for name in got:
        check(name, got[name], want[name], want[name + "_tol"])


CASES = [
    # lens, H, Sq, rank, dtype, block, window
    ([1], 1, 1, 256, "bf16", 16, 0),
    ([1], 1, 1, 512, "fp16", 16, 0),
    ([0], 4, 1, 512, "bf16", 16, 0),
    ([64], 16, 1, 512, "bf16", 64, 0),
    ([0, 5, 0, 0, 300, 1, 0], 5, 1, 256, "fp16", 16, 0),
    ([127, 128, 129, 255, 257], 16, 1, 512, "bf16", 64, 0),
    ([63, 65, 200], 17, 1, 512, "bf16", 32, 0),
    ([3, 1, 0, 200], 6, 4, 512, "fp16", 32, 0),           # fewer keys than new tokens
    ([1000, 17], 16, 4, 512, "bf16", 256, 0),             # 64 rows
    ([700, 30, 1500], 128, 1, 512, "bf16", 1024, 0),      # two groups
    ([700, 30], 40, 2, 256, "fp16", 128, 0),
    ([700, 129, 640], 20, 3, 512, "bf16", 128, 1),        # a window of one key
    ([900, 899], 16, 5, 256, "bf16", 16, 333),
    ([4000], 16, 1, 512, "bf16", 64, 0),                  # one sequence cut into many shares
    ([3000], 128, 8, 256, "bf16", 64, 0),                 # the most rows
    ([500, 333], 7, 130, 256, "bf16", 64, 0),             # heads cut into groups of tokens
    ([90, 700], 11, 33, 512, "bf16", 64, 100),            # one head a group
    ([90, 700], 10, 20, 512, "fp16", 64, 0),              # three heads a group, the last of one
    ([3, 1, 0, 200], 4, 4, 256, "bf16", 16, 2 ** 31 - 1),
    ([40] * 160, 2, 1, 256, "fp16", 16, 0),               # as many tiles as CTAs, and more
    ([5] * 200 + [2000] + [0] * 200, 2, 1, 256, "bf16", 64, 0),
]


@pytest.mark.parametrize("lens,H,Sq,rank,dtype,bs,window", CASES)
def test_decode(fa, lens, H, Sq, rank, dtype, bs, window):
    x = make(lens, H, Sq, rank, dtype, bs, len(lens) + rank + H)
    compare(run(fa, x, window=window), x, window=window)


@pytest.mark.parametrize("rank,H,Sq", [(256, 8, 1), (512, 16, 1), (512, 20, 3), (256, 128, 8)])
def test_segments_of_one_tile(fa, rank, H, Sq):
    """Short sequences, and a longer one whose tiles go to shares of their own: a row's two halves of
    the keys exchange maxima and then sums of weights with nothing in between but the tile's product.
    Maxima that differ by tens between the halves, and the same bits in every call."""
    lens = [33, 64, 40, 500, 1, 63, 50] + [60] * 20
    x = make(lens, H, Sq, rank, "bf16", 16, 13, scale_q=6.0)
    first = run(fa, x)
    compare(first, x)
    d = [t.to(DEV) for t in x]
    got = [fa.decode_latent_paged(*d, SCALE) for _ in range(200)]
    for out, lse in got:
        assert torch.equal(out, first["out"]) and torch.equal(lse, first["lse"])


@pytest.mark.parametrize("rank,H,scale_q", [(512, 16, 8.0), (256, 64, 8.0), (512, 64, 8.0)])
def test_large_scores(fa, rank, H, scale_q):
    """Scores of tens: the reference maximum moves from tile to tile."""
    x = make([700, 333], H, 1, rank, "bf16", 64, 3, scale_q=scale_q)
    compare(run(fa, x), x)


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("H", [16, 40])
def test_rows_outside_the_sequences_may_hold_anything(fa, fill, window, H):
    lens = [1, 90, 200, 513]
    x = make(lens, H, 2, 512, "bf16", 64, 3, fill=fill)
    if window:
        q, cache, table, n = x
        for b, L in enumerate(lens):
            for j in range(max(0, L - 2 + 1 - window)):
                cache[table[b, j // 64], j % 64] = fill
    got = run(fa, x, window=window)
    x[1] = torch.where(x[1].isfinite(), x[1], torch.zeros_like(x[1]))
    compare(got, x, window=window)


TREES = [[-1, 0, 0, 1, 1, 2, 5, 6], [-1, -1, 0, 1, 2, 3, 4, 5], [-1, 0, 1, 2, 3, 4, 5, 6]]


@pytest.mark.parametrize("lens", [[9, 8, 300], [64, 130, 68], [3, 71, 1000]])
@pytest.mark.parametrize("H,rank,dtype", [(16, 512, "bf16"), (3, 256, "fp16")])
def test_tree(fa, lens, H, rank, dtype):
    masks, depths = fa.tree_masks(TREES)
    x = make(lens, H, 8, rank, dtype, 16, 7)
    compare(run(fa, x, tree_masks=masks), x, tree_masks=masks)


def test_tree_of_64(fa):
    g = torch.Generator().manual_seed(2)
    parents = [-1] + [int(torch.randint(0, t, (1,), generator=g)) for t in range(1, 64)]
    masks, _ = fa.tree_masks([parents, list(range(-1, 63))])
    x = make([100, 500], 4, 64, 256, "bf16", 32, 8)
    got = run(fa, x, tree_masks=masks)
    compare(got, x, tree_masks=masks)
    # the second sequence's tree is a chain: the same as without one
    plain = run(fa, x)
    assert torch.equal(got["out"][1], plain["out"][1]) and torch.equal(got["lse"][1], plain["lse"][1])


def test_tree_rows_that_see_nothing(fa):
    """A mask without the row's own bit, over a cache that holds new tokens only."""
    masks = torch.tensor([[0, 2], [1, 0]])
    x = make([2, 2], 4, 2, 512, "bf16", 16, 9)
    got = run(fa, x, tree_masks=masks)
    compare(got, x, tree_masks=masks)
    assert (got["out"][0, :, 0] == 0).all() and (got["lse"][1, :, 1] == float("-inf")).all()


def test_entries_outside_the_cache_read_zeros(fa):
    x = make([300, 260], 16, 1, 512, "fp16", 64, 5)
    x[2][0, 1], x[2][1, 3] = x[1].shape[0] + 7, -5
    compare(run(fa, x), x)


def test_lengths_outside_the_table(fa):
    x = make([64, 128], 4, 1, 256, "bf16", 16, 6, max_blocks=8)
    x[3] = torch.tensor([-3, 5000], dtype=torch.int32)
    compare(run(fa, x), x)


def test_strided_queries(fa):
    """Queries as a product per head leaves them: heads outermost."""
    x = make([300, 70], 16, 2, 512, "bf16", 64, 11)
    want = run(fa, x)
    q = x[0].to(DEV).permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3)
    out, lse = fa.decode_latent_paged(q, *(t.to(DEV) for t in x[1:]), SCALE)
    assert torch.equal(out, want["out"]) and torch.equal(lse, want["lse"])


@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
@pytest.mark.parametrize("H,rank,Sq", [(16, 512, 8), (40, 256, 8), (3, 512, 64)])
def test_drafted_tokens_that_nobody_sees(fa, fill, H, rank, Sq):
    """A batch's trees padded to the same number of tokens, and a token that no mask has: their cache
    rows may hold anything, as what lies past a sequence may."""
    lens = [Sq, 70, 300, 64 + Sq - 3]
    real = [Sq, Sq - 3, 5, 1]                # tokens of each tree; the rest see the prefix only
    masks = fa.tree_masks([[-1 if s == 0 else (s - 1) // 2 for s in range(Sq)]] * 4)[0]
    x = make(lens, H, Sq, rank, "bf16", 16, 21)
    for b, n in enumerate(real):
        masks[b, n:] = 0
        masks[b] &= ~4 if b == 1 else -1     # token 2 of a tree: not even its own row sees it
        for t in [*range(n, Sq)] + [2] * (b == 1):
            j = lens[b] - Sq + t
            x[1][x[2][b, j // 16], j % 16] = fill
    got = run(fa, x, tree_masks=masks)
    compare(got, x, tree_masks=masks)
