"""The latent calls as they are used: a prompt and its decoding agree with the expanded forward,
from several threads and in graphs they give the bits of a call by itself, and what a workspace,
a mask or a long cache can do to them."""
import threading

import numpy as np
import pytest
import torch

from bounds import DT, check, f64, half_step
from causal_flash_attention_gb300 import build as fa_build
from oracle import operators as ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, H, S, D, RANK, BS = 2, 4, 200, 64, 256, 16


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


class Model:
    """One set of inputs, and calls whose results repeat bit for bit."""

    def __init__(self, fa, seed, d=D, rank=RANK, heads=H):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)
        self.fa, self.scale = fa, (d + 64) ** -0.5
        self.q, kv = r(B, S, heads, d + 64).transpose(1, 2), r(B, S, heads, 2 * d).transpose(1, 2)
        self.k, self.v, self.kr = kv[..., :d], kv[..., d:], r(B, S, 96 + 64)[..., 96:]
        self.do = r(B, S, heads, d).transpose(1, 2)
        self.spans = fa.key_spans(B, S, doc_lens=[90, 110], window=70, device=DEV)
        self.turns = fa.rope_turns(fa.rope_inv_freq(64)[0], DEV)
        self.cache = r(B * 16, BS, rank + 64)
        self.table = torch.randperm(B * 16, generator=g).to(torch.int32).view(B, 16).to(DEV)
        self.lens = torch.tensor([150, 77], dtype=torch.int32, device=DEV)
        down = r(B, 2, rank + 64)
        self.latent, self.new_kr, self.w = down[..., :rank], down[..., rank:], r(rank)
        self.absorbed = r(B, heads, 2, rank + 64)

    def train(self):
        fa, x = self.fa, (self.q, self.k, self.kr, self.v)
        out, lse = fa.attention_latent_forward(*x, *self.spans)
        return [out, lse, *fa.attention_latent_backward(*x, out, self.do, lse, *self.spans)]

    def serve(self, **kw):
        fa = self.fa
        q = self.absorbed.clone()
        fa.latent_append(self.latent, self.new_kr, q[..., -64:], self.cache, self.table, self.lens,
                         self.turns, self.w, q_out=q[..., -64:])
        return [q, *fa.decode_latent_paged(q, self.cache, self.table, self.lens, self.scale, **kw)]


def test_threads_with_a_stream_each(fa):
    models = [Model(fa, s, d=(64, 128)[s % 2], rank=(256, 512)[s % 2]) for s in range(4)]
    want = [(m.train(), m.serve()) for m in models]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = models[i].train(), models[i].serve()
                    torch.cuda.current_stream().synchronize()
                    if not (same(got[0], want[i][0]) and same(got[1], want[i][1])):
                        wrong.append(i)
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and fa.fa_last_device_status() == 0


def test_graph_with_copies_fills_and_a_forked_stream(fa):
    """Each call after a node that is no kernel (copy, fill), or after a join of two streams."""
    m, side = Model(fa, 7, d=128), torch.cuda.Stream()
    want = m.train(), m.serve()
    torch.cuda.synchronize()
    src, src_new = m.q.clone(), m.absorbed.clone()
    pad = torch.empty(1 << 20, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        m.q.copy_(src)
        with torch.cuda.stream(side):
            m.absorbed.copy_(src_new)
            served = m.serve()
            pad.zero_()
        trained = m.train()
        torch.cuda.current_stream().wait_stream(side)
        pad.zero_()
        again = m.serve()
        pad.zero_()
        last = m.train()
    for _ in range(3):
        m.q.fill_(float("nan"))
        m.absorbed.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert same(trained, want[0]) and same(last, want[0])
        assert same(served, want[1]) and same(again, want[1])
    assert fa.fa_last_device_status() == 0


@pytest.mark.parametrize("rank,heads,tree", [(256, 4, False), (512, 16, False), (512, 40, True)])
def test_captured_step_with_lengths_that_grow(fa, rank, heads, tree):
    """One captured step serves every length: new tokens, lengths and tree are read at replay."""
    m = Model(fa, 3, rank=rank, heads=heads)
    kw = dict(tree_masks=fa.tree_masks([-1, -1], device=DEV)[0].expand(B, 2).contiguous()) if tree else {}
    start = m.cache.clone()
    m.serve(**kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.serve(**kw)
    for lens in ([2, 256], [3, 16], [0, 1], [64, 65], [255, 130], [300, 2]):   # 300: more than the table holds
        m.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        m.latent.mul_(-0.5)
        m.cache.copy_(start)
        want = [t.clone() for t in m.serve(**kw)] + [m.cache.clone()]
        m.cache.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got + [m.cache], want), lens
    assert fa.fa_last_device_status() == 0


@pytest.mark.parametrize("fill", [0xff, 0x7f, 0x00])
@pytest.mark.parametrize("d,rank,heads", [(64, 256, 4), (128, 512, 16), (128, 512, 40)])
def test_workspace_contents_have_no_meaning(fa, d, rank, heads, fill):
    m = Model(fa, 5, d=d, rank=rank, heads=heads)
    x = (m.q, m.k, m.kr, m.v)
    out, lse = fa.attention_latent_forward(*x, *m.spans)
    want = fa.attention_latent_backward(*x, out, m.do, lse, *m.spans)
    ws = torch.full((fa.fa_bwd_latent_workspace_bytes(B, heads, S, S, d),), fill, dtype=torch.uint8, device=DEV)
    assert same(fa.attention_latent_backward(*x, out, m.do, lse, *m.spans, workspace=ws), want)
    q, *want = m.serve()
    got = [torch.full_like(t, float("nan")) for t in want]
    ws = torch.full((fa.fa_fwd_latent_paged_workspace_bytes(B, heads, 2, rank, BS, 16),), fill,
                    dtype=torch.uint8, device=DEV)
    fa.fa_fwd_latent_paged(q, m.cache, m.table, m.lens, *got, ws, m.scale)
    assert same(got, want)


@pytest.mark.parametrize("d,rank,dtype", [(128, 512, "bf16"), (64, 256, "fp16")])
def test_a_prompt_and_its_decoding(fa, d, rank, dtype):
    """One sequence through both forms. The cache is filled by a prompt and five single tokens;
    keys and values expanded from its rows give the expanded forward, queries absorbed by the same
    weights give the paged one, and both are within their roundings of the 64-bit result:
    scores off by t change weights by at most e^(2t) - 1, and P, V (or the cache's rows as values)
    and the output are rounded once each, u of their size."""
    heads, n, u, F = 4, 150, half_step(DT[dtype]), 2.0 ** -20
    g = torch.Generator().manual_seed(d)
    r = lambda *s: torch.randn(*s, generator=g).to(DT[dtype]).to(DEV)
    wk, wv = r(heads, d, rank) * rank ** -0.5, r(heads, d, rank) * rank ** -0.5
    down, q = r(1, n, rank + 64), r(1, n, heads, d + 64).transpose(1, 2)
    weight, scale = r(rank), (d + 64) ** -0.5
    turns = fa.rope_turns(fa.rope_inv_freq(64)[0], DEV)
    cache = torch.full((14, BS, rank + 64), float("nan"), dtype=DT[dtype], device=DEV)
    table = torch.randperm(14, generator=g).to(torch.int32)[None, :10].contiguous().to(DEV)
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    absorbed = torch.empty(1, heads, n, rank + 64, dtype=DT[dtype], device=DEV)
    torch.matmul(q[0, :, :, :d], wk, out=(qk := torch.empty(heads, n, rank, dtype=DT[dtype], device=DEV)))
    absorbed[0, :, :, :rank] = qk
    steps = [(0, n - 5)] + [(i, i + 1) for i in range(n - 5, n)]
    outs = []
    for a, b in steps:
        lens.fill_(b)
        fa.latent_append(down[:, a:b, :rank], down[:, a:b, rank:], q[:, :, a:b, d:], cache, table, lens, turns,
                         weight, q_out=absorbed[:, :, a:b, rank:])
        outs.append(fa.decode_latent_paged(absorbed[:, :, a:b], cache, table, lens, scale)[0])
    rows = cache[table[0].long()].flatten(0, 1)[:n]
    c, kr = rows[:, :rank], rows[:, rank:]
    k, v = torch.matmul(c, wk.mT)[None], torch.matmul(c, wv.mT)[None]
    qe = torch.cat((q[..., :d], absorbed[..., rank:]), -1)
    out, _ = fa.attention_latent_forward(qe, k, kr[None].contiguous(), v, scale=scale)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == 0

    C, KR, WK, WV, Q = (f64(t) for t in (c, kr, wk, wv, qe[0]))
    paged = f64(torch.cat(outs, 2))[0]
    see = np.tril(np.ones((n, n), bool))
    for h in range(heads):
        K, V, qn = C @ WK[h].T, C @ WV[h].T, Q[h, :, :d]
        s = np.where(see, scale * (qn @ K.T + Q[h, :, d:] @ KR.T), -np.inf)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        want = p @ V
        both = np.abs(Q[h, :, d:]) @ np.abs(KR).T * F
        # expanded: K and V are products in fp32 (F per unit of their terms), rounded
        dK, dV = u * np.abs(K) + F * (np.abs(C) @ np.abs(WK[h]).T), u * np.abs(V) + F * (np.abs(C) @ np.abs(WV[h]).T)
        t = np.where(see, scale * (np.abs(qn) @ (dK + F * np.abs(K)).T + both), 0).max(1, keepdims=True)
        tol = (np.expm1(2 * t) + 2 * u) * (p @ np.abs(V)) + 1.1 * (p @ dV) + 1.1 * u * np.abs(want) + 1e-6
        check("expanded", f64(out[0, h]), want, tol)
        # absorbed: the query's product rounded, then the rows' mean, rounded, times the values' weights
        qa = qn @ WK[h]
        dq = u * np.abs(qa) + F * (np.abs(qn) @ np.abs(WK[h]))
        t = np.where(see, scale * ((dq + F * np.abs(qa)) @ np.abs(C).T + both), 0).max(1, keepdims=True)
        mean = (np.expm1(2 * t) + 2 * u) * (p @ np.abs(C)) + 1.1 * u * np.abs(p @ C) + 1e-6
        check("absorbed", paged[h] @ WV[h].T, want, mean @ np.abs(WV[h]).T)


def test_a_cache_past_32_bits_of_elements(fa):
    """Pages at the end of a cache of more than 2^31 elements: the same bits as in a small one."""
    rank, bs, nb = 256, 64, 105000
    assert nb * bs * (rank + 64) > 2 ** 31
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)
    at = torch.tensor([nb - 1, 0, nb - 2, 52001, 104857, 104858])
    small = r(6, bs, rank + 64)
    big = torch.empty(nb, bs, rank + 64, dtype=torch.bfloat16, device=DEV)
    for i, p in enumerate(at.tolist()):
        big[p] = small[i]
    lens = torch.tensor([190, 65], dtype=torch.int32, device=DEV)
    table = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32)
    q, lat, kr = r(2, 16, 1, rank + 64), r(2, 1, rank), r(2, 1, 64)
    turns = fa.rope_turns(fa.rope_inv_freq(64)[0], DEV)
    got = []
    for cache, t in ((small, table), (big, at[table.long()].to(torch.int32))):
        t = t.to(DEV)
        qr = fa.latent_append(lat, kr, q[..., rank:], cache, t, lens, turns)
        got.append([qr, *fa.decode_latent_paged(q, cache, t, lens, 0.1)])
    assert same(*got) and torch.equal(big[at.to(DEV)], small) and fa.fa_last_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_views_past_32_bits_of_elements(fa, d):
    """A batch further than 2^31 elements from the first, in what is read and what is written."""
    m = Model(fa, 8, d=d)
    x = [m.q, m.k, m.kr, m.v]
    out, lse = fa.attention_latent_forward(*x, *m.spans)
    want = fa.attention_latent_backward(*x, out, m.do, lse, *m.spans)
    far = (1 << 31) + 64
    bases = [torch.empty(far + S * H * (d + 64), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    view = lambda base, w: base.as_strided((B, H, S, w), (far, w, H * w, 1))
    q, dq = view(bases[0], d + 64), view(bases[1], d + 64)
    q.copy_(m.q)
    o2 = view(bases[1], d)
    l2 = torch.empty_like(lse)
    fa.fa_fwd_latent(q, *x[1:], *m.spans, o2, l2)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    got = fa.attention_latent_backward(q, *x[1:], out, m.do, lse, *m.spans, dq=dq)
    assert same(got, want) and got[0].data_ptr() == dq.data_ptr()


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_nan_where_a_row_sees_it(fa, d, dtype):
    m = Model(fa, 13, d=d)
    x = [t.to(DT[dtype]) for t in (m.q, m.k, m.kr, m.v)]
    out, lse = fa.attention_latent_forward(*x, *m.spans)
    y = [t.clone() for t in x]
    y[0][1, 2, 140, 7] = float("nan")                # a query's own row
    y[1][0, 1, 95, 3] = float("nan")                 # a key of one head
    y[2][1, 33, 5] = float("nan")                    # a shared part: every head
    bad = torch.zeros(B, H, S, dtype=torch.bool, device=DEV)
    bad[1, 2, 140] = True
    bad[0, 1, 95:165] = True                         # its document and window
    bad[1, :, 33:90] = True
    out2, lse2 = fa.attention_latent_forward(*y, *m.spans)
    assert torch.equal(lse2.isnan(), bad) and torch.equal(out2.isnan().all(-1), bad)
    assert torch.equal(out2[~bad], out[~bad]) and torch.equal(lse2[~bad], lse[~bad])


@pytest.mark.parametrize("rank,heads", [(256, 4), (512, 16), (512, 40)])
def test_paged_scores_that_are_not_finite(fa, rank, heads):
    m = Model(fa, 17, rank=rank, heads=heads)
    q = m.absorbed
    out, lse = fa.decode_latent_paged(q, m.cache, m.table, m.lens, m.scale)
    q2 = q.clone()
    q2[0, 1, 1, 9] = float("nan")                    # a row of its own
    got = fa.decode_latent_paged(q2, m.cache, m.table, m.lens, m.scale)
    bad = torch.zeros(B, heads, 2, dtype=torch.bool, device=DEV)
    bad[0, 1, 1] = True
    assert torch.equal(got[1].isnan(), bad) and torch.equal(got[0].isnan().all(-1), bad)
    assert torch.equal(got[0][~bad], out[~bad]) and torch.equal(got[1][~bad], lse[~bad])
    m.cache[..., -1] = -3e38                         # in the rotated part, which is no value
    q2 = q.clone()
    q2[..., -1] = 0
    q2[1, 2, 0, -1] = 3e38                           # all its scores are -infinity
    q2[1, 3, 1, -1] = -3e38                          # all +infinity
    out, lse = fa.decode_latent_paged(q2, m.cache, m.table, m.lens, m.scale)
    assert (out[1, 2, 0] == 0).all() and lse[1, 2, 0] == float("-inf")
    assert out[1, 3, 1].isnan().all() and lse[1, 3, 1].isnan()
    rest = torch.ones(B, heads, 2, dtype=torch.bool, device=DEV)
    rest[1, 2, 0] = rest[1, 3, 1] = False
    assert out[rest].isfinite().all() and lse[rest].isfinite().all()


@pytest.mark.parametrize("d,rank,heads", [(64, 256, 4), (128, 512, 16), (128, 512, 40)])
def test_wait_that_runs_out(fa, monkeypatch, d, rank, heads):
    m = Model(fa, 19, d=d, rank=rank, heads=heads)
    x = (m.q, m.k, m.kr, m.v)
    out, lse = fa.attention_latent_forward(*x, *m.spans)
    calls = dict(forward=lambda: fa.attention_latent_forward(*x, *m.spans),
                 backward=lambda: fa.attention_latent_backward(*x, out, m.do, lse, *m.spans),
                 paged=lambda: fa.decode_latent_paged(m.absorbed, m.cache, m.table, m.lens, m.scale))
    want = {n: [t.clone() for t in c()] for n, c in calls.items()}
    torch.cuda.synchronize()
    with monkeypatch.context() as mp:
        mp.setattr(fa, "LIB_PATH", fa_build.build(variant="waittest"))
        mp.setattr(fa, "_lib", None)
        for name, call in calls.items():
            call()
            torch.cuda.synchronize()
            assert fa.fa_last_device_status() == 1, name
            assert fa.fa_last_device_status() == 0, name
    for name, call in calls.items():
        assert same(call(), want[name]), name
    assert fa.fa_last_device_status() == 0


@pytest.mark.parametrize("role,heads", [("producer", 3), ("issuer", 4), ("softmax", 5), ("softmax", 20)])
@pytest.mark.parametrize("n,d,rank", [(60, 64, 512), (60, 128, 256), (1000, 64, 256), (1000, 128, 512)])
def test_wait_that_runs_out_in_any_role(fa, monkeypatch, role, heads, n, d, rank):
    """The role that gives up goes by the heads in that build. With few tiles the others have issued
    all their copies and products by then, and are done before it is known."""
    g = torch.Generator().manual_seed(n + heads)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)
    x = (r(2, heads, n, d + 64), r(2, heads, n, d), r(2, n, 64), r(2, heads, n, d))
    do, q, cache = r(2, heads, n, d), r(3, heads, 2, rank + 64), r(3 * 64, BS, rank + 64)
    table = torch.randperm(3 * 64, generator=g).to(torch.int32).view(3, 64).to(DEV)
    lens = torch.tensor([n, 40, n // 2], dtype=torch.int32, device=DEV)
    out, lse = fa.attention_latent_forward(*x)
    calls = dict(forward=lambda: fa.attention_latent_forward(*x),
                 backward=lambda: fa.attention_latent_backward(*x, out, do, lse),
                 paged=lambda: fa.decode_latent_paged(q, cache, table, lens, 0.1))
    want = {name: [t.clone() for t in c()] for name, c in calls.items()}
    torch.cuda.synchronize()
    with monkeypatch.context() as mp:
        mp.setattr(fa, "LIB_PATH", fa_build.build(variant="waittest"))
        mp.setattr(fa, "_lib", None)
        for name, call in calls.items():
            for _ in range(3):
                call()
            torch.cuda.synchronize()
            assert fa.fa_last_device_status() == 1, name
            assert fa.fa_last_device_status() == 0, name
    for name, call in calls.items():
        assert same(call(), want[name]), name
    assert fa.fa_last_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_fp16_training_in_graphs_and_threads(fa, d):
    """fp16's backward has a kernel more in front, and scratch where results come later."""
    g = torch.Generator().manual_seed(d)
    r = lambda *s: torch.randn(*s, generator=g).half().to(DEV)
    sets = [(r(2, 5, 333, d + 64), r(2, 5, 400, d), r(2, 400, 64), r(2, 5, 400, d), r(2, 5, 333, d) * 2.0 ** -9)
            for _ in range(2)]

    def step(x):
        out, lse = fa.attention_latent_forward(*x[:4])
        return [out, lse, *fa.attention_latent_backward(*x[:4], out, x[4], lse)]

    want = [step(x) for x in sets]
    torch.cuda.synchronize()
    graph, pad = torch.cuda.CUDAGraph(), torch.empty(1 << 20, device=DEV)
    with torch.cuda.graph(graph):
        first = step(sets[0])
        pad.zero_()
        second = step(sets[1])
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = step(sets[i])
                torch.cuda.current_stream().synchronize()
                if not same(got, want[i]):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for _ in range(10):
        graph.replay()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong and same(first, want[0]) and same(second, want[1])
    assert fa.fa_last_device_status() == 0


@pytest.mark.parametrize("heads", [3, 4, 5])
@pytest.mark.parametrize("n,d", [(60, 128), (1000, 64)])
def test_wait_that_runs_out_in_fp16(fa, monkeypatch, heads, n, d):
    g = torch.Generator().manual_seed(n + heads)
    r = lambda *s: torch.randn(*s, generator=g).half().to(DEV)
    x, do = (r(2, heads, n, d + 64), r(2, heads, n, d), r(2, n, 64), r(2, heads, n, d)), r(2, heads, n, d)
    out, lse = fa.attention_latent_forward(*x)
    call = lambda: fa.attention_latent_backward(*x, out, do, lse)
    want = call()
    torch.cuda.synchronize()
    with monkeypatch.context() as mp:
        mp.setattr(fa, "LIB_PATH", fa_build.build(variant="waittest"))
        mp.setattr(fa, "_lib", None)
        call()
        torch.cuda.synchronize()
        assert fa.fa_last_device_status() == 1
    assert same(call(), want) and fa.fa_last_device_status() == 0


def test_tensors_that_do_not_fit(fa):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=DEV)
    i32 = z(2, 8, dt=torch.int32)
    ok = dict(q=z(2, 4, 8, 128), k=z(2, 4, 9, 64), k_rope=z(2, 9, 64), v=z(2, 4, 9, 64),
              key_begin=i32, key_end=i32)
    for bad in (dict(key_begin=i32.long()), dict(key_end=i32[:1]), dict(key_begin=None), dict(v=z(2, 4, 8, 64)),
                dict(k_rope=z(2, 9, 32)), dict(k_rope=z(2, 8, 64)), dict(k_rope=z(2, 1, 9, 64)),
                dict(v=z(2, 4, 9, 64).half()), dict(k=z(2, 2, 9, 64)), dict(q=z(2, 4, 8, 64)),
                dict(key_begin=i32.cpu()), dict(q=z(2, 4, 8, 128).cpu()), dict(q=z(4, 8, 128))):
        with pytest.raises(ValueError):
            fa.attention_latent_forward(**{**ok, **bad})
    with pytest.raises(fa.FAError) as e:
        fa.attention_latent_forward(*(z(1, 2, 8, w).float() for w in (128, 64)), z(1, 8, 64).float(),
                                    z(1, 2, 8, 64).float())
    assert e.value.code == -2
    o, l = z(2, 4, 8, 64), z(2, 4, 8, dt=torch.float32)
    ok.update(out=o, dout=o, lse=l)
    for bad in (dict(out=z(2, 4, 8, 128)), dict(dout=o.half()), dict(lse=l.half()), dict(lse=l[:1]), dict(dq=o),
                dict(dk_rope=z(2, 1, 9, 64)), dict(dv=z(2, 4, 8, 64)),
                dict(dk=z(2, 1, 9, 64).expand(2, 4, 9, 64))):
        with pytest.raises(ValueError):
            fa.attention_latent_backward(**{**ok, **bad})
    with pytest.raises(fa.FAError) as e:
        fa.attention_latent_backward(**ok, workspace=z(16, dt=torch.uint8))
    assert e.value.code == -5
    c, tab, n = z(5, 16, 320), z(2, 3, dt=torch.int32), z(2, dt=torch.int32)
    ok = dict(q=z(2, 4, 8, 320), cache=c, block_table=tab, seq_lens=n, scale=0.1)
    for bad in (dict(seq_lens=n[:1]), dict(seq_lens=n.long()), dict(block_table=tab.long()), dict(cache=c.half()),
                dict(cache=c[..., :256]), dict(cache=c.transpose(0, 1)), dict(block_table=tab.cpu()),
                dict(tree_masks=z(2, 8, dt=torch.int32)), dict(tree_masks=z(2, 7, dt=torch.int64)),
                dict(tree_masks=z(2, 8, dt=torch.int64).cpu())):
        with pytest.raises(ValueError):
            fa.decode_latent_paged(**{**ok, **bad})
    t = z(32, dt=torch.int64)
    ok = dict(latent=z(2, 8, 256), k_rope=z(2, 8, 64), q_rope=z(2, 4, 8, 64), cache=c, block_table=tab,
              seq_lens=n, turns=t)
    for bad in (dict(turns=t.int()), dict(turns=t.cpu()), dict(turns=z(16, dt=torch.int64)),
                dict(latent=z(2, 8, 128)), dict(k_rope=z(2, 7, 64)), dict(q_rope=z(2, 4, 8, 32)),
                dict(weight=z(128)), dict(weight=z(256).half()), dict(positions=i32.long()),
                dict(positions=i32[:1]), dict(cache=c.half()),
                dict(q_out=z(2, 1, 8, 64).expand(2, 4, 8, 64))):
        with pytest.raises(ValueError):
            fa.latent_append(**{**ok, **bad})


@pytest.mark.parametrize("d", [64, 128])
def test_gradients_against_differences(fa, d):
    """<gradient, direction> against a central difference of the 64-bit loss along it. The
    difference's own error: its step squared times the loss's third derivative (here 1e-9 of the
    terms' size), and rounding of the loss over the step."""
    m = Model(fa, 23, d=d)
    x = [m.q[:1, :2, :60], m.k[:1, :2, :60], m.kr[:1, :60], m.v[:1, :2, :60]]
    do = m.do[:1, :2, :60]
    spans = fa.key_spans(1, 60, doc_lens=[13, 1, 46], window=20, device=DEV)
    out, lse = fa.attention_latent_forward(*x, *spans)
    grads = fa.attention_latent_backward(*x, out, do, lse, *spans)
    X, DO, sp = [f64(t) for t in x], f64(do), [t.cpu().numpy() for t in spans]
    tol = ops.latent_attention(*X, *sp, m.scale, DO, half_step(torch.bfloat16))
    loss = lambda y: (ops.latent_attention(*y, *sp, m.scale)["out"] * DO).sum()
    rng, h = np.random.default_rng(d), 1e-4
    for i, name in ((0, "dq"), (1, "dk"), (2, "dk_rope"), (3, "dv")):
        way = rng.standard_normal(X[i].shape)
        y = [[a + s * h * way if j == i else a for j, a in enumerate(X)] for s in (1, -1)]
        want = (loss(y[0]) - loss(y[1])) / (2 * h)
        g = f64(grads[i])
        assert abs((g * way).sum() - want) <= (tol[name + "_tol"] * np.abs(way)).sum() + 1e-5 * np.abs(g * way).sum() + 1e-8


@pytest.mark.parametrize("d,interleaved", [(64, False), (128, True)])
def test_training_step_of_a_layer(fa, d, interleaved):
    """Queries' and keys' rotated parts turned in place, attention, and both backward calls. The
    whole gradient along a direction w of the unrotated parts is the attention's along R w, which a
    difference of the 64-bit loss at the rotated values gives; it is off by the attention's bounds on
    R w and by one rounding where the gradient is turned back."""
    heads, n, u = 3, 90, half_step(torch.bfloat16)
    g = torch.Generator().manual_seed(d)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)
    q, kv = r(1, n, heads, d + 64).transpose(1, 2), r(1, n, heads, 2 * d).transpose(1, 2)
    kr, do, scale = r(1, n, 96)[..., 32:], r(1, n, heads, d).transpose(1, 2), (d + 64) ** -0.5
    freq, rope_scale = fa.rope_inv_freq(64)
    turns, spans = fa.rope_turns(freq, DEV), fa.key_spans(1, n, doc_lens=[50, 40], device=DEV)
    rot = dict(interleaved=interleaved, rope_scale=rope_scale)
    fa.fa_qk_norm_rope(q[..., d:], kr[:, None], q[..., d:], kr[:, None], turns, **rot)
    k, v = kv[..., :d], kv[..., d:]
    out, lse = fa.attention_latent_forward(q, k, kr, v, *spans)
    dkv = torch.empty(1, n, heads, 2 * d, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    dq, _, dkr, _ = fa.attention_latent_backward(q, k, kr, v, out, do, lse, *spans, dk=dkv[..., :d], dv=dkv[..., d:])
    fa.qk_norm_rope_backward(dq[..., d:], dkr[:, None], None, None, turns, **rot, dq=dq[..., d:], dk=dkr[:, None])
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == 0

    X, DO, sp = [f64(t) for t in (q, k, kr, v)], f64(do), [t.cpu().numpy() for t in spans]
    tol = ops.latent_attention(*X, *sp, scale, DO, u)
    loss = lambda y: (ops.latent_attention(*y, *sp, scale)["out"] * DO).sum()
    pos, f = np.arange(n)[None], f64(torch.as_tensor(freq))
    turn = lambda z: ops.norm_rope(z, None, f, pos, 0.0, interleaved, rope_scale)
    rng, h = np.random.default_rng(d), 1e-4
    ways = [rng.standard_normal(x.shape) for x in X]
    moved = [w.copy() for w in ways]
    moved[0][..., d:] = turn(ways[0][..., d:])
    moved[2] = turn(ways[2][:, None])[:, 0]
    grads = [f64(t) for t in (dq, dkv[..., :d], dkr, dkv[..., d:])]
    for i, name in enumerate(("dq", "dk", "dk_rope", "dv")):
        y = [[a + s * h * moved[i] if j == i else a for j, a in enumerate(X)] for s in (1, -1)]
        want = (loss(y[0]) - loss(y[1])) / (2 * h)
        got = (grads[i] * ways[i]).sum()
        bound = (tol[name + "_tol"] * np.abs(moved[i])).sum() + 1e-5 * abs(got) + 1e-8
        if i in (0, 2):
            bound += 1.1 * u * np.abs(grads[i] * ways[i]).sum() + 1e-6
        assert abs(got - want) <= bound, name
