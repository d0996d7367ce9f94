"""Span attention on the GPU against the 64-bit definition, within derived bounds."""
import numpy as np
import pytest
import torch

from bounds import DT, check, f64, half_step
from oracle import operators as ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def inputs(B, Hq, Hkv, Sq, Skv, d, dtype, seed=0, scale_q=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    q, do = r(B, Hq, Sq, d) * scale_q, r(B, Hq, Sq, d)
    k, v = r(B, Hkv, Skv, d), r(B, Hkv, Skv, d)
    return [t.to(DT[dtype]) for t in (q, k, v, do)]


def slopes_of(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)])


def run(fa, q, k, v, do, begin, end, softcap=0.0, slopes=None, scale=None, **kw):
    dev = [t.to(DEV) for t in (q, k, v, do)]
    lo, hi = begin.to(DEV), end.to(DEV)
    sl = None if slopes is None else slopes.to(DEV)
    out, lse = fa.attention_span_forward(*dev[:3], lo, hi, softcap, sl, scale, **kw)
    dq, dk, dv = fa.attention_span_backward(*dev[:3], out, dev[3], lse, lo, hi, softcap, sl, scale,
                                            **kw)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == 0
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv)


def compare(got, q, k, v, do, begin, end, softcap=0.0, slopes=None, scale=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    want = ops.span_attention(*map(f64, (q, k, v)), begin.numpy(), end.numpy(), scale, softcap,
                              None if slopes is None else slopes.numpy(), f64(do),
                              half_step(q.dtype))
    for name, t in got.items():
        check(name, t, want[name], want[name + "_tol"])


def random_spans(B, Sq, Skv, seed):
    """Any spans at all: unordered, empty, reversed, outside the keys."""
    r = np.random.default_rng(seed)
    lo, hi = r.integers(-20, Skv + 5, (B, Sq)), r.integers(-5, Skv + 40, (B, Sq))
    return (torch.from_numpy(x.astype(np.int32)) for x in (lo, hi))


SHAPES = [
    # B, Hq, Hkv, Sq, Skv, d, dtype, softcap, alibi
    (1, 1, 1, 1, 1, 64, "bf16", 0.0, False),
    (1, 2, 1, 1, 300, 128, "fp16", 0.0, True),
    (1, 2, 2, 300, 1, 64, "bf16", 5.0, True),
    (2, 4, 2, 127, 129, 64, "fp16", 0.0, False),
    (1, 3, 1, 129, 127, 128, "bf16", 20.0, False),
    (2, 2, 1, 128, 128, 128, "fp16", 20.0, True),
    (1, 4, 4, 257, 513, 64, "bf16", 10.0, True),
    (3, 2, 1, 385, 200, 128, "bf16", 0.0, False),
    (1, 8, 1, 260, 260, 64, "fp16", 0.0, False),
]


@pytest.mark.parametrize("B,Hq,Hkv,Sq,Skv,d,dtype,softcap,alibi", SHAPES)
def test_any_spans(fa, B, Hq, Hkv, Sq, Skv, d, dtype, softcap, alibi):
    x = inputs(B, Hq, Hkv, Sq, Skv, d, dtype, Sq + Skv, 3.0 if softcap else 1.0)
    begin, end = random_spans(B, Sq, Skv, Sq)
    sl = slopes_of(Hq) if alibi else None
    compare(run(fa, *x, begin, end, softcap, sl), *x, begin, end, softcap, sl)


MASKS = {
    "documents": dict(doc_lens=[[1, 1, 130, 37, 128, 1], [200, 0, 3]]),
    "window_1": dict(window=1),
    "window_77": dict(window=77),
    "prefix": dict(prefix_lens=[150, 1]),
    "padding": dict(kv_lens=[131, 1]),
    "documents_prefix": dict(doc_lens=[64, 100, 90], prefix_lens=40),
    "bidirectional_documents": dict(doc_lens=[100, 28, 128, 42], causal=False),
    "nothing": dict(doc_lens=[]),
    "everything": dict(causal=False),
}


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_masks(fa, mask, d, dtype):
    S = 298
    x = inputs(2, 4, 2, S, S, d, dtype, 11)
    begin, end = fa.key_spans(2, S, **MASKS[mask])
    compare(run(fa, *x, begin, end), *x, begin, end)


@pytest.mark.parametrize("d", [64, 128])
def test_chunk_behind_a_longer_context(fa, d):
    """Sq < Skv, with the distance bias counted from positions i + Skv - Sq."""
    x = inputs(2, 2, 1, 70, 333, d, "bf16", 5)
    begin, end = fa.key_spans(2, 70, 333, window=100)
    sl = slopes_of(2)
    compare(run(fa, *x, begin, end, 0.0, sl), *x, begin, end, 0.0, sl)


def test_scores_far_beyond_the_cap(fa):
    """Scores of +-1000 against a cap of 2: tanh saturates, gradients of q and k vanish."""
    x = inputs(1, 2, 1, 150, 150, 64, "fp16", 6, 60.0)
    begin, end = fa.key_spans(1, 150)
    compare(run(fa, *x, begin, end, 2.0, None, 1.0), *x, begin, end, 2.0, None, 1.0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("most", [0.02, 0.29, 0.31, 0.74, 0.76, 4.0])
def test_scores_on_both_sides_of_the_cap_forms(fa, d, most):
    """The greatest |score| just inside and outside 0.3 and 0.75 of the cap, where the capping
    changes form; whole tiles and, at the last keys, partly masked ones."""
    x = inputs(1, 2, 1, 130, 390, d, "bf16", 8)
    s = torch.einsum("bhid,bhjd->bhij", x[0].float(), x[1].float().repeat_interleave(2, 1))
    scale = most * 10.0 / s.abs().max().item()
    begin, end = fa.key_spans(1, 130, 390, kv_lens=389, causal=False)
    compare(run(fa, *x, begin, end, 10.0, None, scale), *x, begin, end, 10.0, None, scale)


def test_steep_distance_bias_far_from_the_row(fa):
    """A bias of -40 a key over 3000 keys: far tiles underflow, the nearest keys decide."""
    x = inputs(1, 1, 1, 40, 3001, 64, "bf16", 7)
    begin, end = fa.key_spans(1, 40, 3001)
    sl = torch.tensor([40.0])
    compare(run(fa, *x, begin, end, 0.0, sl), *x, begin, end, 0.0, sl)


def test_causal_spans_agree_with_the_causal_call(fa):
    """Forward bit for bit; the gradients of few key tiles are summed in slices, so they are held
    to their bounds, and of many (no slices) dk and dv agree bit for bit too."""
    for Hkv, S in ((2, 700), (12, 3300)):
        x = inputs(1, 2 * Hkv, Hkv, S, S, 128, "bf16", 8)
        dev = [t.to(DEV) for t in x]
        begin, end = fa.key_spans(1, S)
        lo, hi = begin.to(DEV), end.to(DEV)
        out, lse = fa.attention_span_forward(*dev[:3], lo, hi)
        out2, lse2 = fa.attention_forward(*dev[:3])
        g = fa.attention_span_backward(*dev[:3], out, dev[3], lse, lo, hi)
        g2 = fa.attention_backward(*dev[:3], out2, dev[3], lse2)
        torch.cuda.synchronize()
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
        if Hkv == 2:
            compare(dict(zip(("dq", "dk", "dv"), g)), *x, begin, end)
        else:
            assert torch.equal(g[1], g2[1]) and torch.equal(g[2], g2[2])


@pytest.mark.parametrize("B,Hq,Hkv,Sq,Skv,mask", [
    (1, 8, 1, 1000, 1000, dict()),                       # 8 tiles of 8 to 64 steps: many slices
    (3, 4, 2, 900, 900, dict(kv_lens=[900, 130, 517])),  # uneven sequences
    (2, 6, 2, 300, 700, dict(window=90)),                # key tiles that nothing sees
    (1, 16, 2, 130, 2000, dict(causal=False)),
])
@pytest.mark.parametrize("d", [64, 128])
def test_items_cut_into_slices(fa, B, Hq, Hkv, Sq, Skv, mask, d):
    """Few key tiles with many steps each: their dk and dv are joined from slices, and repeat."""
    x = inputs(B, Hq, Hkv, Sq, Skv, d, "fp16", Sq)
    begin, end = fa.key_spans(B, Sq, Skv, **mask)
    got = run(fa, *x, begin, end)
    compare(got, *x, begin, end)
    again = run(fa, *x, begin, end)
    assert torch.equal(got["dk"], again["dk"]) and torch.equal(got["dv"], again["dv"])


def test_more_key_tiles_than_the_work_list_holds(fa):
    """Above 128 key tiles over the batch items go in index order, uncut: a few rows over many
    keys, and a batch of many short sequences."""
    x = inputs(1, 1, 1, 3, 131300, 64, "bf16", 3)
    begin, end = fa.key_spans(1, 3, 131300, window=200)
    compare(run(fa, *x, begin, end), *x, begin, end)
    x = inputs(1100, 1, 1, 20, 20, 64, "fp16", 4)
    begin, end = random_spans(1100, 20, 20, 5)
    compare(run(fa, *x, begin, end), *x, begin, end)


def test_same_bits_again_and_captured_with_changed_spans(fa):
    """dk, dv, out and lse repeat; a captured graph takes the spans that stand in its buffers."""
    x = inputs(2, 2, 1, 300, 300, 128, "fp16", 9)
    dev = [t.to(DEV) for t in x]
    a = [t.to(DEV) for t in fa.key_spans(2, 300, window=50)]
    b = [t.to(DEV) for t in fa.key_spans(2, 300, doc_lens=[10, 200, 60])]
    lo, hi = a[0].clone(), a[1].clone()

    def step():
        out, lse = fa.attention_span_forward(*dev[:3], lo, hi, 4.0)
        return (out, lse, *fa.attention_span_backward(*dev[:3], out, dev[3], lse, lo, hi, 4.0))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        first = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for spans in (a, b, a):
        lo.copy_(spans[0])
        hi.copy_(spans[1])
        for t in held:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        compare(dict(zip(("out", "lse", "dq", "dk", "dv"), held)), *x,
                *(s.cpu() for s in spans), 4.0)
    for i in (0, 1, 3, 4):
        assert torch.equal(held[i], first[i])
    assert fa.fa_last_device_status() == 0


def test_workspace_of_garbage_and_its_size(fa):
    x = inputs(1, 2, 1, 200, 333, 64, "bf16", 10)
    dev = [t.to(DEV) for t in x]
    begin, end = random_spans(1, 200, 333, 3)
    lo, hi = begin.to(DEV), end.to(DEV)
    out, lse = fa.attention_span_forward(*dev[:3], lo, hi)
    n = fa.fa_bwd_span_workspace_bytes(1, 2, 1, 200, 333, 64)
    buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    g = fa.attention_span_backward(*dev[:3], out, dev[3], lse, lo, hi, workspace=buf[:n])
    torch.cuda.synchronize()
    compare(dict(zip(("dq", "dk", "dv"), g)), *x, begin, end)
    assert (buf[n:] == 0xA5).all()
    with pytest.raises(fa.FAError) as e:
        fa.attention_span_backward(*dev[:3], out, dev[3], lse, lo, hi, workspace=buf[: n - 1])
    assert e.value.code == -5


def test_two_streams_at_once(fa):
    x = inputs(1, 4, 2, 500, 500, 64, "bf16", 12)
    begin, end = fa.key_spans(1, 500, window=200)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [run_on(fa, s, x, begin, end) for s in (s1, s2)]
    torch.cuda.synchronize()
    for g in got:
        compare(g, *x, begin, end)


def run_on(fa, stream, x, begin, end):
    """On a stream that is not the current one, given as argument."""
    with torch.cuda.stream(stream):
        dev = [t.to(DEV) for t in x]
        lo, hi = begin.to(DEV), end.to(DEV)
    out, lse = fa.attention_span_forward(*dev[:3], lo, hi, stream=stream)
    g = fa.attention_span_backward(*dev[:3], out, dev[3], lse, lo, hi, stream=stream)
    stream.synchronize()
    return dict(out=out, lse=lse, dq=g[0], dk=g[1], dv=g[2])
