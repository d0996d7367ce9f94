"""Latent attention with expanded keys and values on the GPU, forward and backward, against the
64-bit definition within derived bounds (differences: test_gpu_latent_together.py)."""
import math

import numpy as np
import pytest
import torch

from bounds import DT, check, f64, half_step
from oracle import operators as ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(B, H, Sq, Skv, d, dtype, seed=0, packed=True, scale_q=1.0):
    """q, k, k_rope, v, dout on the CPU; packed: as views of two projections' rows."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    q = (r(B, Sq, H, d + 64) * scale_q).to(DT[dtype]).transpose(1, 2)
    kv = r(B, Skv, H, 2 * d).to(DT[dtype]).transpose(1, 2)
    k, v = kv[..., :d], kv[..., d:]
    down = r(B, Skv, 96 + 64).to(DT[dtype])[..., 96:]
    dout = r(B, Sq, H, d).to(DT[dtype]).transpose(1, 2)
    x = [q, k, down, v, dout]
    return x if packed else [t.contiguous() for t in x]


def to_dev(x):
    """On the device with the strides it has."""
    if x is None or x.is_contiguous():
        return None if x is None else x.to(DEV)
    base = torch.empty(x.untyped_storage().nbytes() // x.element_size(), dtype=x.dtype, device=DEV)
    y = base.as_strided(x.shape, x.stride(), x.storage_offset())
    y.copy_(x)
    return y


def run(fa, x, spans=None, scale=None, backward=True):
    q, k, kr, v, do = (to_dev(t) for t in x)
    b, e = (None, None) if spans is None else (t.to(DEV) for t in spans)
    out, lse = fa.attention_latent_forward(q, k, kr, v, b, e, scale=scale)
    res = dict(out=out, lse=lse)
    if backward:
        g = fa.attention_latent_backward(q, k, kr, v, out, do, lse, b, e, scale=scale)
        res.update(zip(("dq", "dk", "dk_rope", "dv"), g))
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == 0
    return res


def compare(got, x, spans=None, scale=None):
    q, k, kr, v, do = (f64(t) for t in x)
    B, H, Sq, w = q.shape
    Skv = k.shape[2]
    if spans is None:
        end = np.tile(np.clip(np.arange(Sq) + Skv - Sq + 1, 0, Skv), (B, 1))
        begin = np.zeros_like(end)
    else:
        begin, end = (t.numpy() for t in spans)
    want = ops.latent_attention(q, k, kr, v, begin, end, w ** -0.5 if scale is None else scale,
                                do if "dq" in got else None, half_step(x[0].dtype))
    for n in got:
        check(n, got[n], want[n], want[n + "_tol"])


CASES = [
    # B, H, Sq, Skv, d, dtype, mask
    (1, 1, 1, 1, 64, "bf16", None),
    (1, 1, 1, 1, 128, "fp16", None),
    (1, 2, 1, 300, 128, "bf16", None),            # one query at the end of a longer context
    (2, 3, 127, 127, 128, "bf16", None),
    (1, 2, 129, 129, 64, "fp16", None),
    (1, 2, 257, 257, 128, "fp16", None),
    (2, 2, 300, 200, 128, "bf16", None),          # fewer keys than queries: rows that see nothing
    (1, 2, 200, 450, 64, "bf16", None),
    (3, 1, 65, 1000, 128, "bf16", None),
    (1, 3, 640, 640, 128, "bf16", "documents"),
    (2, 2, 500, 500, 64, "fp16", "documents"),
    (1, 2, 700, 700, 128, "fp16", "window"),
    (2, 2, 333, 333, 128, "bf16", "padded"),
    (1, 2, 333, 600, 64, "bf16", "prefix"),
    (1, 1, 400, 900, 128, "bf16", "gaps"),
    (1, 2, 384, 384, 64, "fp16", "gaps"),
    (2, 1, 260, 260, 128, "bf16", "nothing"),
    (1, 2, 130, 70, 64, "bf16", "all"),
    (1, 40, 64, 64, 64, "bf16", None),
]


def spans_of(fa, mask, B, Sq, Skv, seed):
    if mask is None:
        return None
    g = torch.Generator().manual_seed(seed)
    if mask == "documents":
        return fa.key_spans(B, Sq, Skv, doc_lens=[[100, 28, 1, 200, 60 + b] for b in range(B)])
    if mask == "window":
        return fa.key_spans(B, Sq, Skv, window=150)
    if mask == "padded":
        return fa.key_spans(B, Sq, Skv, kv_lens=[Skv - 70 - 130 * b for b in range(B)])
    if mask == "prefix":
        return fa.key_spans(B, Sq, Skv, prefix_lens=Skv - Sq + 200)
    if mask == "all":
        return fa.key_spans(B, Sq, Skv, causal=False)
    if mask == "nothing":
        return torch.full((B, Sq), 7, dtype=torch.int32), torch.full((B, Sq), 7, dtype=torch.int32)
    # any ranges, in no order, some empty, some reaching outside the keys
    begin = torch.randint(-20, Skv, (B, Sq), generator=g, dtype=torch.int32)
    end = begin + torch.randint(-30, Skv // 3, (B, Sq), generator=g, dtype=torch.int32)
    begin[:, 128:200] = Skv + 5      # rows of a tile that see nothing
    return begin, end


@pytest.mark.parametrize("B,H,Sq,Skv,d,dtype,mask", CASES)
def test_expanded(fa, B, H, Sq, Skv, d, dtype, mask):
    x = make(B, H, Sq, Skv, d, dtype, seed=Sq + Skv + d)
    spans = spans_of(fa, mask, B, Sq, Skv, Sq)
    compare(run(fa, x, spans), x, spans)


@pytest.mark.parametrize("B,H,Sq,Skv,d,dtype,mask", [
    (2, 40, 600, 600, 128, "bf16", None),         # 400 CTAs of the backward kernels
    (2, 40, 600, 600, 128, "fp16", "gaps"),
    (4, 24, 500, 500, 64, "bf16", "padded"),
    (3, 30, 500, 500, 64, "fp16", "documents"),
    (9, 20, 130, 400, 64, "bf16", None),
    (200, 2, 70, 70, 128, "bf16", "all"),
])
def test_several_waves_of_ctas(fa, B, H, Sq, Skv, d, dtype, mask):
    """An SM takes one CTA after another: barriers, tensor memory and shared memory are set up anew."""
    x = make(B, H, Sq, Skv, d, dtype, seed=B + H)
    spans = spans_of(fa, mask, B, Sq, Skv, B)
    compare(run(fa, x, spans), x, spans)


@pytest.mark.parametrize("d", [64, 128])
def test_large_scores(fa, d):
    """Scores of tens: the reference maximum moves from tile to tile."""
    x = make(1, 2, 400, 400, d, "bf16", seed=9, scale_q=30.0)
    compare(run(fa, x), x)
    x = make(1, 2, 400, 400, d, "fp16", seed=10)
    compare(run(fa, x, scale=1.0), x, scale=1.0)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_few_keys(fa, d):
    """Short documents, whose rows take D from their scores: the errors of dQ and dK stay within 1.5
    times an output's own rounding (dS and the output rounded: 1.41, measured 1.44)."""
    lens = [75, 3, 130, 50, 128, 1, 200, 53]
    x = make(1, 4, 640, 640, d, "fp16", seed=4)
    spans = fa.key_spans(1, 640, doc_lens=lens)
    got = run(fa, x, spans)
    compare(got, x, spans)
    q, k, kr, v, do = (f64(t) for t in x)
    want = ops.latent_attention(q, k, kr, v, *(t.numpy() for t in spans), (d + 64) ** -0.5, do)
    for n in ("dq", "dk", "dk_rope"):
        step = np.linalg.norm(torch.from_numpy(want[n]).half().double().numpy() - want[n])
        assert np.linalg.norm(f64(got[n]) - want[n]) < 1.5 * step, n


def rms(x):
    return np.sqrt((x * x).mean())


@pytest.mark.parametrize("d,n,size,large", [(64, 2048, 2.0 ** -13, 1.0), (128, 2048, 2.0 ** -13, 1.0),
                                            (128, 1024, 2.0 ** -18, 1.0), (64, 300, 2.0 ** 11, 16.0),
                                            (128, 300, 2.0 ** 11, 16.0)])
def test_fp16_gradients_of_any_size(fa, d, n, size, large):
    """Gradients are linear in dout, and so are the bounds for a dout of size one, but for the
    outputs' own rounding, half of fp16's least step 2^-24 where they are small. At 1e-4 over 2048
    keys dS is a few such steps itself; with large values and dout short rows' dS are past fp16's
    largest value, while no gradient is."""
    x = make(1, 2, n, n, d, "fp16", seed=d + n)
    x[3] = x[3] * large
    if large > 1:
        x[:3] = [t * 0.25 for t in x[:3]]
    x[4] = (x[4].float().clamp(-2, 2) * size).half()
    got = run(fa, x)
    q, k, kr, v, do = (f64(t) for t in x)
    end = np.arange(1, n + 1)[None]
    want = ops.latent_attention(q, k, kr, v, np.zeros_like(end), end, (d + 64) ** -0.5, do / size, half_step(torch.float16))
    for name in ("dq", "dk", "dk_rope", "dv"):
        ref = want[name] * size
        assert np.abs(ref).max() < 65504
        check(name, got[name], ref, want[name + "_tol"] * size + 1.01 * 2.0 ** -25)
        if large == 1:
            own = rms(torch.from_numpy(ref).half().double().numpy() - ref)
            assert rms(f64(got[name]) - ref) < 1.5 * own, name


@pytest.mark.parametrize("d", [64, 128])
def test_fp16_gradients_of_rows_that_weigh_differently(fa, d):
    """Rows whose dout is 2^-20 of the others': dq is each row's own, and so is its bound."""
    x = make(2, 2, 700, 700, d, "fp16", seed=d)
    x[1:3] = [t * 8 for t in x[1:3]]         # gradients well above fp16's least steps
    x[0] = x[0] * 0.125
    size = torch.where(torch.arange(700) % 3 == 0, 1.0, 2.0 ** -20)[:, None]
    x[4] = (x[4].float() * size).half()
    spans = fa.key_spans(2, 700, doc_lens=[[300, 1, 399], [64, 600, 36]], window=500)
    got = run(fa, x, spans)
    compare({n: got[n] for n in ("dk", "dk_rope", "dv", "dq")}, x, spans)
    q, k, kr, v, do = (f64(t) for t in x)
    size = size.double().numpy()
    want = ops.latent_attention(q, k, kr, v, *(t.numpy() for t in spans), (d + 64) ** -0.5, do / size,
                                half_step(torch.float16))
    check("dq", got["dq"], want["dq"] * size, want["dq_tol"] * size + 1.01 * 2.0 ** -25)


@pytest.mark.parametrize("fill", [0xff, 0x7f, 0x00])
def test_fp16_workspace_contents_have_no_meaning(fa, fill):
    x = [to_dev(t) for t in make(2, 3, 300, 410, 64, "fp16", seed=3)]
    out, lse = fa.attention_latent_forward(*x[:4])
    want = fa.attention_latent_backward(*x[:4], out, x[4], lse)
    ws = torch.full((fa.fa_bwd_latent_workspace_bytes(2, 3, 300, 410, 64),), fill, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        got = fa.attention_latent_backward(*x[:4], out, x[4], lse, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
