"""Caps far above the scores: a capped score is then known relative to itself, not to the cap, in
every kernel that caps."""
import numpy as np
import pytest
import torch

from bounds import DT, check, f64, half_step
from oracle import operators as ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CAPS = [300.0, 900.0, 1e4, 1e6, 1e9, 2.0 ** 56]


@pytest.fixture
def relative(monkeypatch):
    """The oracle with the cap's error relative to the score: the fit is off by 4.0e-6 of tanh u at
    most for |u| <= 0.3 (at u = 0), a few fp32 steps beside it: 2^-17.8."""
    plain = ops.score_parts

    def parts(q, k, scale, softcap=0.0, slope=0.0, offset=None):
        assert not slope
        s, _, err = plain(q, k, scale)
        t = np.tanh(s / softcap)
        assert np.abs(s).max() <= 0.3 * softcap
        return softcap * t, 1.0 - t * t, err + 2.0 ** -17.8 * np.abs(s)

    monkeypatch.setattr(ops, "score_parts", parts)


def randn(g, dtype, *s):
    return torch.randn(*s, generator=g).to(DT[dtype])


@pytest.mark.parametrize("softcap", CAPS)
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_span(fa, relative, softcap, d, dtype):
    g = torch.Generator().manual_seed(d)
    q, do = 3 * randn(g, dtype, 1, 2, 200, d), randn(g, dtype, 1, 2, 200, d)
    k, v = randn(g, dtype, 1, 1, 260, d), randn(g, dtype, 1, 1, 260, d)
    begin, end = fa.key_spans(1, 200, 260)
    dev = [t.to(DEV) for t in (q, k, v)]
    lo, hi = begin.to(DEV), end.to(DEV)
    out, lse = fa.attention_span_forward(*dev, lo, hi, softcap)
    grads = fa.attention_span_backward(*dev, out, do.to(DEV), lse, lo, hi, softcap)
    torch.cuda.synchronize()
    want = ops.span_attention(f64(q), f64(k), f64(v), begin.numpy(), end.numpy(), d ** -0.5, softcap,
                              None, f64(do), half_step(q.dtype))
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        check(name, t, want[name], want[name + "_tol"])


@pytest.mark.parametrize("softcap", CAPS)
@pytest.mark.parametrize("Hq,Hkv,Sq", [(4, 2, 1), (24, 1, 1), (40, 1, 1), (8, 1, 16)])
@pytest.mark.parametrize("garbage", [False, True])
def test_ragged(fa, relative, softcap, Hq, Hkv, Sq, garbage):
    """Also with infinities in rows of the last pages that no row sees, which do not decide how
    the scores beside them are capped."""
    d, bs, lens = 128, 64, [900, 300, 70]
    g = torch.Generator().manual_seed(Hq)
    q, (kc, vc) = 3 * randn(g, "bf16", 3, Hq, Sq, d), randn(g, "bf16", 2, 45, Hkv, bs, d)
    table = torch.randperm(45, generator=g).to(torch.int32).view(3, 15)
    if garbage:
        for b, n in enumerate(lens):
            kc[table[b, n // bs], :, n % bs:] = float("inf")
            kc[table[b, n // bs], :, n % bs:, ::2] = -3e38
    x = [q, kc, vc, table, torch.tensor(lens, dtype=torch.int32)]
    out, lse = fa.decode_forward_ragged(*(t.to(DEV) for t in x), softcap=softcap)
    torch.cuda.synchronize()
    kc = torch.where(kc.abs() < 1e30, kc, torch.zeros_like(kc))
    want = ops.ragged_attention(f64(q), f64(kc), f64(vc), table.numpy(), lens, d ** -0.5, 0, softcap,
                                u=half_step(q.dtype))
    check("out", out, want["out"], want["out_tol"])
    check("lse", lse, want["lse"], want["lse_tol"])
