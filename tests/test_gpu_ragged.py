"""New tokens over a paged cache of unequal sequences, on the GPU, against the 64-bit definition
within derived bounds."""
import numpy as np
import pytest
import torch

from bounds import DT, check, f64, half_step
from oracle import operators as ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(lens, Hq, Hkv, Sq, d, dtype, bs, seed=0, scale_q=1.0, max_blocks=None, spare=4, fill=None):
    """q, caches and table; rows of the cache that no sequence holds are `fill`."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    per = [-(-max(n, 0) // bs) for n in lens]
    nb = sum(per) + spare
    kc, vc = torch.randn(2, nb, Hkv, bs, d, generator=g)
    perm = torch.randperm(nb, generator=g)
    table = torch.full((B, max_blocks or max(max(per), 1)), -1, dtype=torch.int32)
    used, at = torch.zeros(nb, bs, dtype=torch.bool), 0
    for b, m in enumerate(per):
        table[b, :m] = perm[at: at + m]
        for j in range(max(lens[b], 0)):
            used[table[b, j // bs], j % bs] = True
        at += m
    if fill is not None:
        kc.transpose(1, 2)[~used] = fill
        vc.transpose(1, 2)[~used] = fill
    q = torch.randn(B, Hq, Sq, d, generator=g) * scale_q
    return [t.to(DT[dtype]) for t in (q, kc, vc)] + [table, torch.tensor(lens, dtype=torch.int32)]


def run(fa, q, kc, vc, table, lens, **kw):
    kw = {n: v.to(DEV) if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    out, lse = fa.decode_forward_ragged(*(t.to(DEV) for t in (q, kc, vc, table, lens)), **kw)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == 0
    return dict(out=out, lse=lse)


def compare(got, q, kc, vc, table, lens, window=0, softcap=0.0, slopes=None, scale=None):
    want = ops.ragged_attention(f64(q), f64(kc), f64(vc), table.numpy(), lens.tolist(),
                                q.shape[-1] ** -0.5 if scale is None else scale, window, softcap,
                                None if slopes is None else slopes.numpy(), half_step(q.dtype))
    for name in got:
        check(name, got[name], want[name], want[name + "_tol"])


def slopes_of(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)])


CASES = [
    # lens, Hq, Hkv, Sq, d, dtype, block, window, softcap, alibi
    ([1], 1, 1, 1, 64, "bf16", 16, 0, 0.0, False),
    ([0], 4, 2, 1, 128, "bf16", 16, 0, 0.0, False),
    ([0, 5, 0, 0, 300, 1, 0], 4, 2, 1, 64, "fp16", 16, 0, 0.0, False),
    ([127, 128, 129, 255, 257], 8, 2, 1, 128, "bf16", 64, 0, 0.0, True),
    ([3, 1, 0, 200], 6, 3, 4, 128, "fp16", 32, 0, 0.0, False),      # fewer keys than new tokens
    ([1000, 17], 16, 1, 8, 64, "bf16", 256, 0, 20.0, False),        # G * Sq = 128
    ([700, 30, 2500], 4, 4, 1, 128, "bf16", 1024, 100, 0.0, False),
    ([700, 129, 640], 4, 2, 3, 64, "fp16", 128, 1, 0.0, False),     # a window of one key
    ([2000, 1999], 2, 1, 5, 128, "fp16", 16, 333, 15.0, True),
    ([4000], 2, 2, 1, 64, "bf16", 64, 0, 0.0, True),
    ([3, 1, 0, 200], 4, 2, 4, 64, "bf16", 16, 2 ** 31 - 1, 0.0, False),   # the largest window
    ([2, 200], 16, 1, 5, 64, "bf16", 16, 208, 0.0, False),          # as many keys as the table
    ([40] * 160, 2, 1, 1, 64, "fp16", 16, 0, 0.0, False),           # as many tiles as CTAs, and more
    ([130] * 77, 3, 3, 1, 128, "bf16", 32, 0, 0.0, False),
    ([5] * 200 + [3000] + [0] * 200, 2, 1, 1, 64, "bf16", 64, 0, 0.0, False),
]


@pytest.mark.parametrize("lens,Hq,Hkv,Sq,d,dtype,bs,window,softcap,alibi", CASES)
def test_ragged(fa, lens, Hq, Hkv, Sq, d, dtype, bs, window, softcap, alibi):
    x = make(lens, Hq, Hkv, Sq, d, dtype, bs, len(lens) + d, 4.0 if softcap else 1.0)
    kw = dict(window=window, softcap=softcap, slopes=slopes_of(Hq) if alibi else None)
    compare(run(fa, *x, **kw), *x, **kw)


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("window", [0, 70])
def test_rows_outside_the_sequences_may_hold_anything(fa, fill, window):
    """The tail of every last page, unused pages and, under a window, keys before it."""
    lens = [1, 90, 200, 513]
    x = make(lens, 4, 2, 2, 128, "bf16", 64, 3, fill=fill)
    if window:
        q, kc, vc, table, n = x
        for b, L in enumerate(lens):
            for j in range(max(0, L - 2 + 1 - window)):
                kc[table[b, j // 64], :, j % 64] = fill
                vc[table[b, j // 64], :, j % 64] = fill
    got = run(fa, *x, window=window)
    x[1], x[2] = (torch.where(t.isfinite(), t, torch.zeros_like(t)) for t in x[1:3])
    compare(got, *x, window=window)


def test_pages_before_the_window_need_no_entry(fa):
    """Freed pages: entries of pages wholly before every row's window are not read as pages."""
    x = make([1000], 2, 1, 1, 64, "bf16", 16, 4)
    want = run(fa, *x, window=100)
    y = [t.clone() for t in x]
    y[3][0, : (1000 - 100) // 16] = -1
    got = run(fa, *y, window=100)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


def test_entries_outside_the_cache_read_zeros(fa):
    q, kc, vc, table, lens = make([300, 260], 4, 2, 1, 128, "fp16", 64, 5)
    table[0, 1], table[1, 3] = kc.shape[0] + 7, -5
    compare(run(fa, q, kc, vc, table, lens), q, kc, vc, table, lens)


def test_lengths_outside_the_table(fa):
    """Negative lengths count as 0, lengths above the table's capacity as that."""
    x = make([64, 128], 4, 2, 1, 64, "bf16", 16, 6, max_blocks=8)
    x[4] = torch.tensor([-3, 5000], dtype=torch.int32)
    compare(run(fa, *x), *x)


def test_same_bits_and_replay_with_other_lengths(fa):
    """A captured call follows the lengths that stand in its buffer; results repeat bit for bit."""
    lens = [1500, 3, 800, 0, 129]
    x = make(lens, 4, 2, 2, 128, "bf16", 32, 7)
    dev = [t.to(DEV) for t in x]
    with torch.cuda.stream(torch.cuda.Stream()):
        first = [t.clone() for t in fa.decode_forward_ragged(*dev)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = fa.decode_forward_ragged(*dev)
    for now in (lens, [1, 1, 1, 0, 1], [1400, 3, 799, 0, 2], lens):
        dev[4].copy_(torch.tensor(now, dtype=torch.int32))
        for t in held:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        y = x[:4] + [torch.tensor(now, dtype=torch.int32)]
        compare(dict(out=held[0], lse=held[1]), *y)
    assert torch.equal(held[0], first[0]) and torch.equal(held[1], first[1])


def test_two_streams_with_a_workspace_each(fa):
    xs = [make([900, 70, 333], 8, 2, 1, 64, "fp16", 64, s) for s in (1, 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    devs = [[t.to(DEV) for t in x] for x in xs]
    torch.cuda.synchronize()
    held = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            held[i].append(fa.decode_forward_ragged(*devs[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in held[i]:
            compare(dict(out=out, lse=lse), *xs[i])


def test_workspace_of_garbage_and_its_size(fa):
    x = make([3000, 40], 8, 2, 1, 128, "bf16", 64, 8)
    dev = [t.to(DEV) for t in x]
    out, lse = torch.empty_like(dev[0]), torch.empty(2, 8, 1, device=DEV)
    n = fa.fa_fwd_ragged_paged_workspace_bytes(2, 8, 2, 1, 128, 64, x[3].shape[1])
    buf = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    fa.fa_fwd_ragged_paged(*dev, out, lse, buf[:n])
    torch.cuda.synchronize()
    compare(dict(out=out, lse=lse), *x)
    assert (buf[n:] == 0xFF).all()
    with pytest.raises(fa.FAError) as e:
        fa.fa_fwd_ragged_paged(*dev, out, lse, buf[: n - 1])
    assert e.value.code == -5


def test_random_shapes(fa):
    r = np.random.default_rng(12)
    for i in range(25):
        Hkv, G, Sq = int(r.integers(1, 5)), int(r.choice([1, 2, 4, 8])), int(r.choice([1, 1, 2, 7]))
        B, top = int(r.integers(1, 40)), int(r.choice([20, 200, 1500]))
        lens = [int(n) for n in r.integers(0, top, B)]
        bs, d = int(r.choice([16, 32, 64, 128, 256])), int(r.choice([64, 128]))
        x = make(lens, Hkv * G, Hkv, Sq, d, ["bf16", "fp16"][i % 2], bs, i)
        kw = dict(window=int(r.choice([0, 0, 37, 300])))
        compare(run(fa, *x, **kw), *x, **kw)
