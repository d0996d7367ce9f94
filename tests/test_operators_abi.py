"""Refusals of the span, ragged and query/key-preparation entry points, without a GPU: the C ABI
rejects bad arguments on the host with the documented codes, the binding rejects tensors that do
not fit together, and key_spans builds the masks it documents."""
import ctypes
import math

import numpy as np
import pytest
import torch

SHAPE, DTYPE, NULL, ALIGN, WORKSPACE, SCALE = -1, -2, -3, -4, -5, -7
P = 256   # an aligned address that is never read


def span_fwd(L, q=P, k=P, v=P, begin=P, end=P, out=P, lse=P, B=1, Hq=2, Hkv=1, Sq=9, Skv=7, d=64,
             scale=0.1, softcap=0.0, slopes=None, dtype=2):
    return L.fa_fwd_span(q, k, v, begin, end, out, lse, B, Hq, Hkv, Sq, Skv, d, scale, softcap,
                         slopes, dtype, None)


def span_bwd(L, B=1, Hq=2, Hkv=1, Sq=9, Skv=7, d=64, scale=0.1, softcap=0.0, slopes=None, dtype=2,
             ws=P, ws_bytes=1 << 30, **over):
    names = ("q", "k", "v", "begin", "end", "out", "dout", "lse", "dq", "dk", "dv")
    return L.fa_bwd_span(*(over.get(n, P) for n in names), B, Hq, Hkv, Sq, Skv, d, scale, softcap,
                         slopes, dtype, ws, ws_bytes, None)


SPAN_BAD = [
    (dict(d=96), SHAPE), (dict(Sq=0), SHAPE), (dict(Skv=0), SHAPE), (dict(Hq=3, Hkv=2), SHAPE),
    (dict(B=1 << 30, Hq=4, Hkv=4), SHAPE), (dict(dtype=0), DTYPE), (dict(dtype=5), DTYPE),
    (dict(scale=0.0), SCALE), (dict(scale=math.nan), SCALE), (dict(softcap=-1.0), SCALE),
    (dict(softcap=math.inf), SCALE), (dict(softcap=math.nan), SCALE),
    (dict(softcap=1e-20), SCALE), (dict(softcap=1e20), SCALE), (dict(softcap=50.0, scale=1e-20), SCALE),
    (dict(softcap=1e-10, scale=1e10), SCALE), (dict(begin=None), NULL),
    (dict(end=None), NULL), (dict(q=None), NULL), (dict(lse=None), NULL), (dict(begin=P + 2), ALIGN),
    (dict(end=P + 1), ALIGN), (dict(slopes=P + 2), ALIGN), (dict(v=P + 8), ALIGN),
    (dict(out=P + 4), ALIGN),
]


@pytest.mark.parametrize("kw,code", SPAN_BAD)
def test_span_forward_refuses(fa_lib, kw, code):
    assert span_fwd(fa_lib.lib(), **kw) == code


@pytest.mark.parametrize("kw,code", SPAN_BAD + [
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE), (dict(ws=P + 16), ALIGN),
    (dict(dk=None), NULL), (dict(dout=P + 8), ALIGN)])
def test_span_backward_refuses(fa_lib, kw, code):
    assert span_bwd(fa_lib.lib(), **kw) == code


def test_span_workspace_formula(fa_lib):
    up = lambda x: -(-x // 256) * 256
    for B, Hq, Hkv, Sq, Skv, d in [(1, 2, 1, 1, 1, 64), (3, 8, 2, 1537, 200, 128),
                                   (1, 32, 8, 8192, 8192, 128), (2, 2, 1, 64, 100000, 64),
                                   (3, 2, 1, 8000, 8000, 64)]:
        tiles, rows = B * -(-Skv // 128), B * -(-Sq // 128) * 128
        want = fa_lib.fa_bwd_kv_workspace_bytes(B, Hq, Hkv, Sq, Skv, d) + up(rows * 8) + up(tiles * 8)
        if tiles <= 128 and tiles * Hkv < 304:     # cut tiles and partial results
            parts = min(304, tiles * Hkv * (Hq // Hkv) * (rows // B // 128))
            want += up(16 + parts * 16) + parts * 2 * 128 * d * 4
        assert fa_lib.fa_bwd_span_workspace_bytes(B, Hq, Hkv, Sq, Skv, d) == want
    assert fa_lib.fa_bwd_span_workspace_bytes(1, 3, 2, 9, 9, 64) == 0


def ragged(L, q=P, k=P, v=P, table=P, lens=P, out=P, lse=P, B=2, Hq=8, Hkv=2, Sq=1, d=64, bs=16,
           nb=10, mb=4, window=0, scale=0.1, softcap=0.0, slopes=None, dtype=1, ws=P,
           ws_bytes=1 << 30):
    return L.fa_fwd_ragged_paged(q, k, v, table, lens, out, lse, B, Hq, Hkv, Sq, d, bs, nb, mb,
                                 window, scale, softcap, slopes, dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=80), SHAPE), (dict(B=0), SHAPE), (dict(Sq=33), SHAPE), (dict(bs=8), SHAPE),
    (dict(bs=2048), SHAPE), (dict(bs=48), SHAPE), (dict(nb=0), SHAPE), (dict(mb=0), SHAPE),
    (dict(nb=1 << 30), SHAPE), (dict(B=1 << 20, mb=1 << 14), SHAPE), (dict(window=-1), SHAPE), (dict(Hq=256, Hkv=1), SHAPE),
    (dict(dtype=0), DTYPE), (dict(dtype=9), DTYPE), (dict(scale=-1.0), SCALE),
    (dict(softcap=math.nan), SCALE), (dict(softcap=-0.5), SCALE), (dict(softcap=1e-30), SCALE), (dict(softcap=1e30), SCALE), (dict(table=None), NULL),
    (dict(lens=None), NULL), (dict(k=None), NULL), (dict(table=P + 2), ALIGN),
    (dict(lens=P + 1), ALIGN), (dict(slopes=P + 3), ALIGN), (dict(q=P + 8), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=64), WORKSPACE), (dict(ws=P + 32), ALIGN)])
def test_ragged_refuses(fa_lib, kw, code):
    assert ragged(fa_lib.lib(), **kw) == code


def test_ragged_workspace_formula(fa_lib):
    up = lambda x: -(-x // 256) * 256
    for B, Hq, Hkv, Sq, d, bs, mb in [(1, 1, 1, 1, 64, 16, 1), (16, 32, 8, 1, 128, 64, 128),
                                      (2, 12, 12, 3, 64, 16, 20)]:
        ctas = min(152, B * Hkv * -(-(mb * bs) // 128))
        rows = 2 * ctas * (Hq // Hkv) * Sq
        want = up(rows * d * 4) + up(rows * 4) + up(16 * ctas)
        assert fa_lib.fa_fwd_ragged_paged_workspace_bytes(B, Hq, Hkv, Sq, d, bs, mb) == want
    assert fa_lib.fa_fwd_ragged_paged_workspace_bytes(1, 8, 1, 17, 64, 16, 4) == 0
    assert fa_lib.fa_fwd_ragged_paged_workspace_bytes(1, 8, 1, 1, 64, 24, 4) == 0


def view(fa, data=P, sb=64, sh=64, ss=64):
    return ctypes.byref(fa._View(data, sb, sh, ss))


def heads(fa, q=(), k=(), q_out=(), k_out=(), wq=None, wk=None, eps=1e-6, pos=None, turns=P,
          rope_dim=64, rope_scale=1.0, B=1, Hq=2, Hkv=1, S=3, d=64, dtype=2):
    views = [None if v is None else view(fa, *v) for v in (q, k, q_out, k_out)]
    return fa.lib().fa_qk_norm_rope(*views, wq, wk, eps, pos, turns, rope_dim, 0, rope_scale, B, Hq,
                                    Hkv, S, d, dtype, None)


def heads_bwd(fa, q=(), dq=(), wq=P, wk=P, dwq=P, dwk=P, ws=P, ws_bytes=1 << 30, S=3, **kw):
    a = dict(eps=1e-6, pos=None, turns=P, rope_dim=64, rope_scale=1.0, B=1, Hq=2, Hkv=1, d=64,
             dtype=2)
    a.update(kw)
    q, dq = (None if v is None else view(fa, *v) for v in (q, dq))
    return fa.lib().fa_qk_norm_rope_bwd(view(fa), view(fa), q, view(fa), dq, view(fa), dwq, dwk, wq,
                                        wk, a["eps"], a["pos"], a["turns"], a["rope_dim"], 0,
                                        a["rope_scale"], a["B"], a["Hq"], a["Hkv"], S, a["d"],
                                        a["dtype"], ws, ws_bytes, None)


HEADS_BAD = [
    (dict(d=32), SHAPE), (dict(S=0), SHAPE), (dict(rope_dim=8), SHAPE), (dict(rope_dim=-16), SHAPE),
    (dict(rope_dim=80), SHAPE), (dict(Hq=3, Hkv=2), SHAPE), (dict(dtype=3), DTYPE),
    (dict(rope_scale=math.inf), SCALE), (dict(turns=None), NULL), (dict(turns=P + 4), ALIGN),
    (dict(pos=P + 2), ALIGN), (dict(wq=P, wk=None), NULL), (dict(wq=None, wk=P), NULL),
    (dict(wq=P, wk=P + 4), ALIGN), (dict(wq=P, wk=P, eps=-1.0), SCALE),
    (dict(wq=P, wk=P, eps=math.nan), SCALE), (dict(q=None), NULL), (dict(q=(None,)), NULL),
    (dict(q=(P + 8,)), ALIGN), (dict(q=(P, 4)), ALIGN), (dict(q=(P, 64, 12)), ALIGN),
    (dict(q=(P, 64, 64, 2), dtype=0), ALIGN),
]


@pytest.mark.parametrize("kw,code", HEADS_BAD + [
    (dict(k_out=None), NULL), (dict(q_out=(P, 64, 64, 1)), ALIGN)])
def test_norm_rope_refuses(fa_lib, kw, code):
    assert heads(fa_lib, **kw) == code


@pytest.mark.parametrize("kw,code", HEADS_BAD + [
    (dict(dq=None), NULL), (dict(dwq=None), NULL), (dict(dwk=P + 2), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=16), WORKSPACE), (dict(ws=P + 16), ALIGN)])
def test_norm_rope_backward_refuses(fa_lib, kw, code):
    assert heads_bwd(fa_lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(bs=12), SHAPE), (dict(nb=0), SHAPE), (dict(mb=0), SHAPE), (dict(kc=None), NULL),
    (dict(table=None), NULL), (dict(lens=None), NULL), (dict(vc=P + 8), ALIGN),
    (dict(table=P + 2), ALIGN), (dict(lens=P + 2), ALIGN), (dict(v=None), NULL),
    (dict(v=(P, 64, 4)), ALIGN), (dict(dtype=7), DTYPE)])
def test_append_refuses(fa_lib, kw, code):
    a = dict(v=(), kc=P, vc=P, table=P, lens=P, bs=16, nb=4, mb=2, dtype=2)
    a.update(kw)
    v = None if a["v"] is None else view(fa_lib, *a["v"])
    assert fa_lib.lib().fa_qk_norm_rope_append(
        view(fa_lib), view(fa_lib), v, view(fa_lib), a["kc"], a["vc"], a["table"], a["lens"], None,
        None, 0.0, P, 64, 0, 1.0, 1, 2, 1, 1, 64, a["bs"], a["nb"], a["mb"], a["dtype"],
        None) == code


def test_norm_rope_workspace(fa_lib):
    f = fa_lib.fa_qk_norm_rope_bwd_workspace_bytes
    assert f(1, 2, 1, 1, 64) == 2 * 64 * 4                       # one block of partial sums
    assert f(64, 32, 8, 8192, 128) == 304 * 2 * 128 * 4          # the most
    assert f(4, 2, 1, 100, 64, norm=False) == 0
    assert f(0, 2, 1, 100, 64) == 0 and f(1, 3, 2, 100, 64) == 0 and f(1, 2, 1, 100, 80) == 0


# --------------------------------------------------------------- the binding --
def test_binding_refuses_host_tensors(fa_lib):
    q, k = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 4, 64).bfloat16()
    i = torch.zeros(1, 4, dtype=torch.int32)
    t = torch.zeros(32, dtype=torch.int64)
    for call in (lambda: fa_lib.attention_span_forward(q, k, k, i, i),
                 lambda: fa_lib.attention_span_backward(q, k, k, q, q, q[..., 0], i, i),
                 lambda: fa_lib.decode_forward_ragged(q, k, k, i, i[:, 0]),
                 lambda: fa_lib.qk_norm_rope_forward(q, k, t),
                 lambda: fa_lib.qk_norm_rope_backward(q, k, q, k, t),
                 lambda: fa_lib.qk_norm_rope_append(q, k, k, k, k, i, i[:, 0], t)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_turns_table(fa_lib):
    t = fa_lib.rope_turns([2 * math.pi * 0.25, -2 * math.pi * 0.25, 2 * math.pi * 3.5, 0.0])
    assert t.dtype == torch.int64
    assert t.tolist() == [1 << 62, -(1 << 62), -(1 << 63), 0]
    with pytest.raises(ValueError):
        fa_lib.rope_turns([math.inf])
    for bad in (dict(rope_dim=3), dict(rope_dim=8, factor=0.5), dict(rope_dim=8, scaling="other"),
                dict(rope_dim=8, scaling="parts", low_turns=4.0, high_turns=4.0)):
        with pytest.raises(ValueError):
            fa_lib.rope_inv_freq(**bad)


def brute(B, Sq, Skv, causal=True, window=0, docs=None, prefix=None, kv_lens=None):
    ok = np.zeros((B, Sq, Skv), bool)
    for b in range(B):
        doc = np.full(Skv, -1)
        lens = docs[b] if docs is not None else [Skv]
        start, first = 0, {}
        for n, m in enumerate(lens):
            doc[start: start + m], first[n] = n, start
            start += m
        L = Skv if kv_lens is None else kv_lens[b]
        for i in range(Sq):
            p = i + Skv - Sq
            for j in range(Skv):
                if p < 0 or p >= L or j >= L or doc[p] < 0 or doc[j] != doc[p]:
                    continue
                see = (j <= p or not causal) and (not window or j > p - window)
                if prefix is not None and j < first[doc[p]] + prefix[b]:
                    see = True
                ok[b, i, j] = see
    return ok


@pytest.mark.parametrize("kw,ref", [
    (dict(), dict()), (dict(causal=False), dict(causal=False)), (dict(window=3), dict(window=3)),
    (dict(doc_lens=[3, 0, 5, 2]), dict(docs=[[3, 0, 5, 2]] * 2)),
    (dict(doc_lens=[[4, 4], [1, 9]], window=2), dict(docs=[[4, 4], [1, 9]], window=2)),
    (dict(doc_lens=[[4, 4], []], causal=False), dict(docs=[[4, 4], []], causal=False)),
    (dict(prefix_lens=[2, 6]), dict(prefix=[2, 6])),
    (dict(doc_lens=[5, 5], prefix_lens=3), dict(docs=[[5, 5]] * 2, prefix=[3, 3])),
    (dict(kv_lens=[4, 12], window=2), dict(kv_lens=[4, 12], window=2)),
    (dict(kv_lens=7, prefix_lens=6), dict(kv_lens=[7, 7], prefix=[6, 6])),
])
@pytest.mark.parametrize("Sq,Skv", [(12, 12), (5, 12)])
def test_key_spans(fa_lib, kw, ref, Sq, Skv):
    begin, end = fa_lib.key_spans(2, Sq, Skv, **kw)
    assert begin.dtype == end.dtype == torch.int32 and begin.shape == end.shape == (2, Sq)
    j = torch.arange(Skv)
    got = (j >= begin[..., None]) & (j < end[..., None])
    assert (got.numpy() == brute(2, Sq, Skv, **ref)).all()


def test_key_spans_of_rows_before_the_keys(fa_lib):
    """Fewer keys than rows: documents hold no row before the first key; without documents and
    without the causal mask every row sees every key."""
    begin, end = fa_lib.key_spans(1, 8, 5, doc_lens=[3, 2], causal=False)
    assert (end - begin).tolist() == [[0, 0, 0, 3, 3, 3, 2, 2]]
    begin, end = fa_lib.key_spans(1, 8, 5, causal=False)
    assert (end - begin).tolist() == [[5] * 8]
    begin, end = fa_lib.key_spans(1, 8, 5)
    assert (end - begin).tolist() == [[0, 0, 0, 1, 2, 3, 4, 5]]


@pytest.mark.parametrize("kw", [dict(doc_lens=[20]), dict(doc_lens=[-1, 2]), dict(kv_lens=[1, 2, 3]),
                                dict(doc_lens=[[1]]), dict(window=2, prefix_lens=1)])
def test_key_spans_refuses(fa_lib, kw):
    with pytest.raises(ValueError):
        fa_lib.key_spans(2, 8, **kw)
