"""Per-head norm and rotary positions on the GPU (forward, backward, append) against the 64-bit
definition within derived bounds, and the operators run together as a model uses them."""
import numpy as np
import pytest
import torch

from bounds import DT, check, f64, half_step, norm_rope_bounds
from oracle import operators as ops

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def freqs(rope_dim):
    return (10000.0 ** (-np.arange(0, rope_dim, 2) / max(rope_dim, 1))).tolist()


def make(B, Hq, Hkv, S, d, dtype, norm, layout, seed=0):
    """q [B,Hq,S,d], k, v [B,Hkv,S,d] views of a layout; weights."""
    g = torch.Generator().manual_seed(seed)
    H = Hq + 2 * Hkv
    if layout == "packed":            # one projection's rows [q | k | v]
        x = torch.randn(B, S, H, d, generator=g).to(DT[dtype]).to(DEV).transpose(1, 2)
    elif layout == "heads_first":
        x = torch.randn(H, B, S, d, generator=g).to(DT[dtype]).to(DEV).transpose(0, 1)
    else:                             # rows with a gap between heads
        x = torch.randn(B, S, H, d + 16, generator=g).to(DT[dtype]).to(DEV)[..., :d].transpose(1, 2)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(DT[dtype]).to(DEV) if norm else None
         for _ in range(2)]
    return q, k, v, w


def run_both(fa, q, k, w, inv_freq, positions, eps, interleaved, rope_scale, seed=1):
    turns = fa.rope_turns(inv_freq, DEV) if inv_freq else None
    g = torch.Generator().manual_seed(seed)
    kw = dict(turns=turns, positions=positions, q_weight=w[0], k_weight=w[1], eps=eps,
              interleaved=interleaved, rope_scale=rope_scale)
    outs = fa.qk_norm_rope_forward(q, k, **kw)
    dys = [torch.randn(t.shape, generator=g).to(q.dtype).to(DEV) for t in outs]
    grads = fa.qk_norm_rope_backward(*dys, q, k, **kw)
    torch.cuda.synchronize()
    B, S = q.shape[0], q.shape[2]
    pos = np.broadcast_to(np.arange(S), (B, S)) if positions is None else positions.cpu().numpy()
    u = half_step(q.dtype)
    for i, (x, y, dy) in enumerate(zip((q, k), outs, dys)):
        wi = None if w[i] is None else f64(w[i])
        a = dict(inv_freq=inv_freq, positions=pos, eps=eps, interleaved=interleaved,
                 rope_scale=rope_scale)
        check("y%d" % i, y, ops.norm_rope(f64(x), wi, **a), norm_rope_bounds(f64(x), wi, u=u, **a))
        dx, dw = ops.norm_rope(f64(x), wi, dy=f64(dy), **a)
        tol, dw_tol = norm_rope_bounds(f64(x), wi, u=u, dy=f64(dy), **a)
        check("dx%d" % i, grads[i], dx, tol)
        assert (grads[2 + i] is None) == (wi is None)
        if wi is not None:
            assert grads[2 + i].dtype == torch.float32
            check("dw%d" % i, grads[2 + i], dw, dw_tol)
    return outs, grads


CASES = [
    # B, Hq, Hkv, S, d, dtype, rope_dim, interleaved, norm, layout
    (1, 1, 1, 1, 64, "bf16", 64, False, True, "packed"),
    (2, 3, 1, 5, 128, "fp16", 128, False, True, "gap"),
    (1, 5, 5, 33, 64, "fp32", 16, True, True, "heads_first"),
    (3, 2, 2, 17, 128, "bf16", 48, False, False, "packed"),
    (1, 12, 4, 129, 64, "fp16", 48, True, True, "packed"),
    (2, 8, 2, 64, 128, "fp32", 128, True, False, "gap"),
    (1, 4, 2, 301, 128, "bf16", 0, False, True, "packed"),      # the norm alone
    (1, 6, 3, 700, 64, "fp32", 64, False, True, "packed"),
    (1, 32, 8, 1200, 128, "bf16", 128, False, True, "packed"),  # every warp takes all heads
    (1, 40, 1, 9, 64, "bf16", 32, False, True, "heads_first"),
]


@pytest.mark.parametrize("B,Hq,Hkv,S,d,dtype,rope_dim,interleaved,norm,layout", CASES)
def test_forward_and_backward(fa, B, Hq, Hkv, S, d, dtype, rope_dim, interleaved, norm, layout):
    q, k, _, w = make(B, Hq, Hkv, S, d, dtype, norm, layout, S)
    r = np.random.default_rng(S)
    positions = torch.from_numpy(r.integers(0, 20000, (B, S)).astype(np.int32)).to(DEV)
    run_both(fa, q, k, w, freqs(rope_dim), positions, 1e-6, interleaved, 1.0)


def test_positions_default_scale_and_zero_rows(fa):
    q, k, _, w = make(2, 4, 2, 50, 64, "bf16", True, "packed", 3)
    q[0, 1, 7] = 0          # the norm of a zero row is zero
    outs, grads = run_both(fa, q, k, w, freqs(64), None, 1e-5, False, 1.25)
    assert (outs[0][0, 1, 7] == 0).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_at_the_ends_of_int32(fa, interleaved):
    q, k, _, w = make(1, 2, 1, 6, 64, "fp32", False, "packed", 4)
    pos = torch.tensor([[0, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 1 << 24]], dtype=torch.int32)
    run_both(fa, q, k, w, freqs(64), pos.to(DEV), 1e-6, interleaved, 1.0)


def test_frequency_scalings(fa):
    plain, one = fa.rope_inv_freq(64)
    assert one == 1.0 and plain[0] == 1.0
    linear, _ = fa.rope_inv_freq(64, scaling="linear", factor=4.0)
    assert torch.equal(linear, plain / 4)
    base, _ = fa.rope_inv_freq(64, scaling="base", factor=4.0)
    assert base[0] == 1.0 and abs(base[-1] / plain[-1] - 0.25) < 1e-12
    parts, scale = fa.rope_inv_freq(64, scaling="parts", factor=4.0, trained_len=4096)
    assert parts[0] == plain[0] and abs(parts[-1] / plain[-1] - 0.25) < 1e-12 and scale > 1
    q, k, _, w = make(1, 2, 1, 40, 64, "fp16", True, "packed", 5)
    pos = (torch.arange(40, dtype=torch.int32) * 700)[None].to(DEV)
    for f in (linear, base, parts):
        run_both(fa, q, k, w, f.tolist(), pos, 1e-6, False, scale)


def test_in_place_and_into_views(fa):
    """Outputs over their inputs; gradients into views of one packed buffer."""
    q, k, v, w = make(2, 4, 2, 37, 128, "bf16", True, "packed", 6)
    turns = fa.rope_turns(freqs(128), DEV)
    kw = dict(q_weight=w[0], k_weight=w[1])
    want = fa.qk_norm_rope_forward(q, k, turns, **kw)
    dy = [torch.randn_like(t) for t in want]
    want_g = fa.qk_norm_rope_backward(*dy, q, k, turns, **kw)
    packed = torch.full((2, 37, 8, 128), 5.0, dtype=q.dtype, device=DEV).transpose(1, 2)
    got_g = fa.qk_norm_rope_backward(*dy, q, k, turns, dq=packed[:, :4], dk=packed[:, 4:6], **kw)
    q2, k2 = q.clone(), k.clone()
    fa.fa_qk_norm_rope(q2, k2, q2, k2, turns, **kw)
    torch.cuda.synchronize()
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    assert torch.equal(packed[:, :4], want_g[0]) and torch.equal(packed[:, 4:6], want_g[1])
    assert (packed[:, 6:] == 5.0).all()          # what is not named stays as it was
    assert torch.equal(got_g[2], want_g[2]) and torch.equal(got_g[3], want_g[3])


@pytest.mark.parametrize("d", [64, 128])
def test_eps_zero(fa, d):
    """With eps = 0 only a head of zeros has no norm: it gives zeros, and neither it nor the
    lanes past the last head (one key head here) reach the weight gradients."""
    q, k, _, w = make(1, 3, 1, 21, d, "bf16", True, "packed", 8)
    outs, grads = run_both(fa, q, k, w, freqs(d), None, 0.0, False, 1.0)
    turns = fa.rope_turns(freqs(d), DEV)
    kw = dict(q_weight=w[0], k_weight=w[1], eps=0.0)
    q, dy = q.clone(), [torch.randn_like(t) for t in outs]
    dy[0][0, 1, 4] = 0
    want = fa.qk_norm_rope_backward(*dy, q, k, turns, **kw)   # this head's dy is 0: no share of dw
    q[0, 1, 4] = 0
    assert (fa.qk_norm_rope_forward(q, k, turns, **kw)[0][0, 1, 4] == 0).all()
    got = fa.qk_norm_rope_backward(*dy, q, k, turns, **kw)
    assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])
    assert (got[0][0, 1, 4] == 0).all()
    q[0, 2, 9, 3] = float("nan")
    assert fa.qk_norm_rope_forward(q, k, turns, **kw)[0][0, 2, 9].isnan().all()


def test_a_bad_row_stays_its_own(fa):
    """NaN and infinity in one head of one token reach no other head or token."""
    q, k, _, w = make(1, 4, 2, 20, 64, "bf16", True, "packed", 7)
    turns = fa.rope_turns(freqs(64), DEV)
    clean = fa.qk_norm_rope_forward(q, k, turns, q_weight=w[0], k_weight=w[1])
    q[0, 1, 3, 5], q[0, 2, 4, 0] = float("nan"), float("inf")
    got = fa.qk_norm_rope_forward(q, k, turns, q_weight=w[0], k_weight=w[1])
    same = torch.ones(1, 4, 20, dtype=torch.bool, device=DEV)
    same[0, 1, 3] = same[0, 2, 4] = False
    assert torch.equal(got[0][same], clean[0][same]) and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_infinity_past_the_rotated_part_stays_where_it_is(fa, interleaved):
    q, k, _, w = make(1, 2, 1, 5, 64, "fp16", False, "packed", 8)
    turns = fa.rope_turns(freqs(32), DEV)
    clean = fa.qk_norm_rope_forward(q, k, turns, interleaved=interleaved)
    q, k = q.clone(), k.clone()
    q[0, 1, 3, 40], k[0, 0, 2, 63] = float("inf"), float("-inf")
    got = fa.qk_norm_rope_forward(q, k, turns, interleaved=interleaved)
    clean[0][0, 1, 3, 40], clean[1][0, 0, 2, 63] = float("inf"), float("-inf")
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])


# ------------------------------------------------------------------ append --
def cache(nb, Hkv, bs, d, dtype):
    return torch.full((nb, Hkv, bs, d), 9.0, dtype=DT[dtype], device=DEV)


@pytest.mark.parametrize("lens,Sq,Hq,Hkv,d,dtype,bs,rope_dim,interleaved,norm", [
    ([1], 1, 1, 1, 64, "bf16", 16, 64, False, True),
    ([5, 200, 64, 65], 1, 8, 2, 128, "bf16", 64, 128, False, True),
    ([3, 0, 40], 4, 4, 4, 64, "fp32", 16, 32, True, True),      # fewer positions than tokens
    ([130, 77], 77, 6, 2, 128, "fp16", 32, 128, False, False),
    ([1500, 900], 900, 4, 1, 64, "fp32", 256, 64, False, True),
])
def test_append(fa, lens, Sq, Hq, Hkv, d, dtype, bs, rope_dim, interleaved, norm):
    B = len(lens)
    q, k, v, w = make(B, Hq, Hkv, Sq, d, dtype, norm, "packed", Sq)
    f = freqs(rope_dim)
    per = max(-(-n // bs) for n in lens)
    nb = B * per + 2
    table = torch.randperm(nb, generator=torch.Generator().manual_seed(1))[: B * per]
    table = table.to(torch.int32).view(B, per)
    kc, vc = cache(nb, Hkv, bs, d, dtype), cache(nb, Hkv, bs, d, dtype)
    q_out = fa.qk_norm_rope_append(q, k, v, kc, vc, table.to(DEV),
                                   torch.tensor(lens, dtype=torch.int32, device=DEV),
                                   fa.rope_turns(f, DEV), q_weight=w[0], k_weight=w[1],
                                   interleaved=interleaved)
    torch.cuda.synchronize()
    pos = np.array([[n - Sq + s for s in range(Sq)] for n in lens])
    a = dict(inv_freq=f, positions=pos, eps=1e-6, interleaved=interleaved, rope_scale=1.0)
    u = half_step(q.dtype)
    ws = [None if t is None else f64(t) for t in w]
    check("q", q_out, ops.norm_rope(f64(q), ws[0], **a), norm_rope_bounds(f64(q), ws[0], u=u, **a))
    want_k = ops.norm_rope(f64(k), ws[1], **a)
    tol_k = norm_rope_bounds(f64(k), ws[1], u=u, **a)
    K, T, V = np.full(kc.shape, 9.0), np.zeros(kc.shape), np.full(vc.shape, 9.0)
    for b in range(B):
        for s in range(Sq):
            if pos[b, s] >= 0:
                page, row = int(table[b, pos[b, s] // bs]), pos[b, s] % bs
                K[page, :, row], T[page, :, row] = want_k[b, :, s], tol_k[b, :, s]
                V[page, :, row] = f64(v)[b, :, s]
    check("k_cache", kc, K, T + 1e-300)
    assert (f64(vc) == V).all()


def test_append_outside_the_cache_stores_nothing(fa):
    """Entries outside the pool and positions past the table: not stored, nothing else touched."""
    q, k, v, w = make(3, 2, 1, 2, 64, "bf16", True, "packed", 9)
    kc, vc = cache(4, 1, 16, 64, "bf16"), cache(4, 1, 16, 64, "bf16")
    table = torch.tensor([[4, 0], [-1, 1], [2, 3]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([2, 16, 40], dtype=torch.int32, device=DEV)
    fa.qk_norm_rope_append(q, k, v, kc, vc, table, lens, fa.rope_turns(freqs(64), DEV),
                           q_weight=w[0], k_weight=w[1])
    torch.cuda.synchronize()
    assert (kc == 9.0).all() and (vc == 9.0).all()


def test_pages_past_two_to_the_31_elements(fa):
    """The same step on a cache whose pages lie past 2^31 elements, and on a small one."""
    Hkv, d, bs, lens = 8, 128, 64, [130, 64]
    q, k, v, w = make(2, 16, Hkv, 1, d, "bf16", True, "packed", 11)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    turns = fa.rope_turns(freqs(d), DEV)
    small = [torch.randn(4, Hkv, bs, d, generator=torch.Generator().manual_seed(i)).to(q) for i in (1, 2)]
    nb = (1 << 31) // (Hkv * bs * d) + 50
    big = [torch.empty(nb, Hkv, bs, d, dtype=q.dtype, device=DEV) for _ in range(2)]
    for s, t in zip(small, big):
        t[nb - 4:] = s
    table = torch.tensor([[2, 0, 3], [1, -1, -1]], dtype=torch.int32, device=DEV)
    got = [fa.decode_step_ragged(q, k, v, *c, t, n, turns, w[0], w[1])
           for c, t in ((small, table), (big, torch.where(table < 0, table, table + nb - 4)))]
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert all(torch.equal(t[nb - 4:], s) for s, t in zip(small, big))


# ---------------------------------------------------------------- together --
def test_training_step_of_an_attention_layer(fa):
    """Packed projection -> norm and rotation -> span attention -> backward through both, each
    stage against the 64-bit definition on what the stage before gave."""
    B, Hq, Hkv, S, d = 2, 4, 2, 260, 64
    q, k, v, w = make(B, Hq, Hkv, S, d, "bf16", True, "packed", 10)
    f = freqs(d)
    begin, end = fa.key_spans(B, S, doc_lens=[100, 33, 127], device=DEV)
    pos = (torch.arange(S, device=DEV, dtype=torch.int32)[None] - begin).contiguous()
    kw = dict(turns=fa.rope_turns(f, DEV), positions=pos, q_weight=w[0], k_weight=w[1])
    qr, kr = fa.qk_norm_rope_forward(q, k, **kw)
    vc = v.contiguous()
    out, lse = fa.attention_span_forward(qr, kr, vc, begin, end, 30.0)
    do = torch.randn(out.shape, generator=torch.Generator().manual_seed(2)).to(out).contiguous()
    dqr, dkr, dv = fa.attention_span_backward(qr, kr, vc, out, do, lse, begin, end, 30.0)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(dqr, dkr, q, k, **kw)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == 0
    u = half_step(q.dtype)
    want = ops.span_attention(f64(qr), f64(kr), f64(vc), begin.cpu().numpy(), end.cpu().numpy(),
                              d ** -0.5, 30.0, None, f64(do), u)
    for name, t in (("out", out), ("lse", lse), ("dq", dqr), ("dk", dkr), ("dv", dv)):
        check(name, t, want[name], want[name + "_tol"])
    a = dict(inv_freq=f, positions=pos.cpu().numpy(), eps=1e-6, interleaved=False, rope_scale=1.0)
    for x, wi, y, dy, g, gw in ((q, w[0], qr, dqr, dq, dwq), (k, w[1], kr, dkr, dk, dwk)):
        check("y", y, ops.norm_rope(f64(x), f64(wi), **a),
              norm_rope_bounds(f64(x), f64(wi), u=u, **a))
        dx, dw = ops.norm_rope(f64(x), f64(wi), dy=f64(dy), **a)
        tol, dw_tol = norm_rope_bounds(f64(x), f64(wi), u=u, dy=f64(dy), **a)
        check("dx", g, dx, tol)
        check("dw", gw, dw, dw_tol)


@pytest.mark.parametrize("captured", [False, True])
def test_steps_back_to_back_over_the_same_buffers(fa, captured):
    """Training steps one after the other without a wait, every step over the same intermediate
    buffers and workspaces, each kernel set up beside the one before: the same results as step
    by step (dq is summed in any order, all that does not depend on it has the same bits)."""
    B, Hq, Hkv, S, d, steps = 1, 4, 2, 260, 128, 12
    turns = fa.rope_turns(freqs(d), DEV)
    begin, end = fa.key_spans(B, S, window=100, device=DEV)
    xs = [make(B, Hq, Hkv, S, d, "bf16", True, "packed", 20 + i) for i in range(steps)]
    e = lambda H, *s: torch.empty(B, H, *s, dtype=torch.bfloat16, device=DEV)
    qr, kr, out, dq, dk, dv = e(Hq, S, d), e(Hkv, S, d), e(Hq, S, d), e(Hq, S, d), e(Hkv, S, d), e(Hkv, S, d)
    lse = torch.empty(B, Hq, S, device=DEV)
    ws = torch.empty(fa.fa_bwd_span_workspace_bytes(B, Hq, Hkv, S, S, d), dtype=torch.uint8, device=DEV)
    ws2 = torch.empty(fa.fa_qk_norm_rope_bwd_workspace_bytes(B, Hq, Hkv, S, d), dtype=torch.uint8, device=DEV)
    do = torch.randn(B, Hq, S, d, generator=torch.Generator().manual_seed(1)).to(out)

    def step(x, r):
        q, k, v, w = x
        fa.fa_qk_norm_rope(q, k, qr, kr, turns, None, *w)
        fa.fa_fwd_span(qr, kr, r["v"], begin, end, out, lse, 20.0)
        fa.fa_bwd_span(qr, kr, r["v"], begin, end, out, do, lse, dq, dk, dv, ws, 20.0)
        fa.fa_qk_norm_rope_bwd(dq, dk, q, k, r["dq"], r["dk"], r["dwq"], r["dwk"], ws2, turns, None, *w)

    def results():
        return [dict(v=x[2].contiguous(), dq=e(Hq, S, d), dk=e(Hkv, S, d),
                     dwq=torch.empty(d, device=DEV), dwk=torch.empty(d, device=DEV)) for x in xs]

    want, got = results(), results()
    for x, r in zip(xs, want):
        step(x, r)
        torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for x, r in zip(xs, got):
                step(x, r)
        for _ in range(3):
            graph.replay()
    else:
        for _ in range(3):
            for x, r in zip(xs, got):
                step(x, r)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == 0
    for a, b in zip(got, want):
        assert torch.equal(a["dk"], b["dk"]) and torch.equal(a["dwk"], b["dwk"])
        # one rounding of bf16 each way where the sums of dq differ in their last bits
        most = b["dq"].float().abs().max().item()
        assert (a["dq"].float() - b["dq"].float()).abs().max().item() <= 2 * 2.0 ** -8 * most


def test_serving_loop(fa):
    """Prompts of unequal length into the cache, then steps of new tokens, captured once and
    replayed: every step against the 64-bit definition on the cache as it stands."""
    Hq, Hkv, d, bs, prompts = 4, 2, 128, 16, [30, 7, 64]
    B, f = len(prompts), freqs(128)
    turns = fa.rope_turns(f, DEV)
    nb = 24
    table = torch.randperm(nb, generator=torch.Generator().manual_seed(3)).to(torch.int32)
    table = table.view(B, 8).to(DEV).contiguous()
    kc, vc = cache(nb, Hkv, bs, d, "bf16"), cache(nb, Hkv, bs, d, "bf16")
    Sp = max(prompts)       # left-padded prompts: rows at negative positions are not stored
    q, k, v, w = make(B, Hq, Hkv, Sp, d, "bf16", True, "packed", 11)
    lens = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    kw = dict(q_weight=w[0], k_weight=w[1])
    fa.qk_norm_rope_append(q, k, v, kc, vc, table, lens, turns, **kw)
    q1, k1, v1, _ = make(B, Hq, Hkv, 1, d, "bf16", True, "packed", 12)
    lens.add_(1)
    with torch.cuda.stream(torch.cuda.Stream()):
        fa.decode_step_ragged(q1, k1, v1, kc, vc, table, lens, turns, window=40, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = fa.decode_step_ragged(q1, k1, v1, kc, vc, table, lens, turns, window=40, **kw)
    for step in range(4):
        g = torch.Generator().manual_seed(20 + step)
        for t in (q1, k1, v1):
            t.copy_(torch.randn(t.shape, generator=g).to(t))
        if step:
            lens.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        n = lens.cpu().numpy()
        a = dict(inv_freq=f, positions=(n - 1)[:, None], eps=1e-6, interleaved=False, rope_scale=1.0)
        qn = ops.norm_rope(f64(q1), f64(w[0]), **a)
        # the stored key is the definition's within its bound
        kn, tol = ops.norm_rope(f64(k1), f64(w[1]), **a), norm_rope_bounds(
            f64(k1), f64(w[1]), u=half_step(q1.dtype), **a)
        for b in range(B):
            at = (int(table[b, (n[b] - 1) // bs]), slice(None), (n[b] - 1) % bs)
            check("k", f64(kc)[at], kn[b, :, 0], tol[b, :, 0])
            assert (f64(vc)[at] == f64(v1)[b, :, 0]).all()
        # q is rounded to bf16 on the way: its own kernel gives the rounded one
        qr = fa.qk_norm_rope_append(q1, k1, v1, kc, vc, table, lens, turns, **kw)
        check("q", qr, qn, norm_rope_bounds(f64(q1), f64(w[0]), u=half_step(q1.dtype), **a))
        want = ops.ragged_attention(f64(qr), f64(kc), f64(vc), table.cpu().numpy(), n.tolist(),
                                    d ** -0.5, 40, u=half_step(q1.dtype))
        check("out", out, want["out"], want["out_tol"])
        check("lse", lse, want["lse"], want["lse_tol"])
    assert fa.fa_last_device_status() == 0
