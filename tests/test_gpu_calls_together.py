"""The span, ragged and preparation calls among other work: from several threads at once, in graphs
beside copies, fills and forked streams, and mixed back to back on two streams."""
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, Hq, Hkv, S, D, BS = 2, 4, 2, 200, 64, 16


class Model:
    """One set of inputs, and calls whose results repeat bit for bit (dq aside)."""

    def __init__(self, fa, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)
        self.fa = fa
        self.x = r(B, S, Hq + 2 * Hkv, D).transpose(1, 2)
        self.w = [r(D), r(D)]
        self.do = r(B, Hq, S, D)
        self.turns = fa.rope_turns(fa.rope_inv_freq(D)[0], DEV)
        self.spans = fa.key_spans(B, S, doc_lens=[90, 110], window=70, device=DEV)
        self.cache = [r(B * 16, Hkv, BS, D) for _ in range(2)]
        self.table = torch.randperm(B * 16, generator=g).to(torch.int32).view(B, 16).to(DEV)
        self.lens = torch.tensor([150, 77], dtype=torch.int32, device=DEV)
        self.new = [r(B, h, 1, D) for h in (Hq, Hkv, Hkv)]

    def train(self):
        fa, (q, k, v) = self.fa, self.x.split([Hq, Hkv, Hkv], dim=1)
        qr, kr = fa.qk_norm_rope_forward(q, k, self.turns, None, *self.w)
        v = v.contiguous()
        out, lse = fa.attention_span_forward(qr, kr, v, *self.spans, 20.0)
        _, dk, dv = fa.attention_span_backward(qr, kr, v, out, self.do, lse, *self.spans, 20.0)
        g = fa.qk_norm_rope_backward(self.do, dk, q, k, self.turns, None, *self.w)
        return [out, lse, dk, dv, *g]

    def serve(self):
        return list(self.fa.decode_step_ragged(*self.new, *self.cache, self.table, self.lens,
                                               self.turns, *self.w, window=60))


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_threads_with_a_stream_each(fa):
    models = [Model(fa, s) for s in range(4)]
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
    m, side = Model(fa, 7), torch.cuda.Stream()
    want = m.train(), m.serve()
    torch.cuda.synchronize()
    x, new = m.x.clone(), m.new[0].clone()
    src, src_new = m.x.clone(), m.new[0].clone()
    m.x, m.new[0] = x, new
    pad = torch.empty(1 << 20, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        x.copy_(src)
        with torch.cuda.stream(side):
            new.copy_(src_new)
            served = m.serve()
            pad.zero_()
        trained = m.train()
        torch.cuda.current_stream().wait_stream(side)
        pad.zero_()
        again = m.serve()
        pad.zero_()
        last = m.train()
    for _ in range(3):
        x.fill_(float("nan"))
        new.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert same(trained, want[0]) and same(last, want[0])
        assert same(served, want[1]) and same(again, want[1])
    assert fa.fa_last_device_status() == 0


def test_mixed_calls_back_to_back_on_two_streams(fa):
    models = [Model(fa, s) for s in (11, 12)]
    want = [(m.train(), m.serve()) for m in models]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    order, got = np.random.default_rng(1).integers(0, 2, (60, 2)), []
    for i, kind in order:
        with torch.cuda.stream(streams[i]):
            got.append((i, kind, (models[i].train, models[i].serve)[kind]()))
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == 0
    assert all(same(r, want[i][kind]) for i, kind, r in got)
