"""A bounded wait that runs out in the span and ragged kernels (see test_gpu_wait_limit.py): with
the wait-limit test library each call returns, reports the timeout once, and the product library
then works in the same context. Also: tensors that do not fit together are refused before a
launch."""
import pytest
import torch

from causal_flash_attention_gb300 import build as fa_build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("d", [64, 128])
def test_wait_that_runs_out(fa, monkeypatch, d):
    g = torch.Generator().manual_seed(d)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().to(DEV)
    q, k, v, do = r(1, 2, 400, d), r(1, 1, 400, d), r(1, 1, 400, d), r(1, 2, 400, d)
    begin, end = fa.key_spans(1, 400, window=150, device=DEV)
    qd, kc, vc = r(2, 4, 1, d), r(40, 2, 16, d), r(40, 2, 16, d)
    table = torch.arange(40, dtype=torch.int32, device=DEV).view(2, 20)
    lens = torch.tensor([300, 17], dtype=torch.int32, device=DEV)
    calls = dict(
        forward=lambda: fa.attention_span_forward(q, k, v, begin, end),
        backward=lambda: fa.attention_span_backward(q, k, v, out, do, lse, begin, end),
        ragged=lambda: fa.decode_forward_ragged(qd, kc, vc, table, lens))
    out, lse = calls["forward"]()
    want = {n: [t.clone() for t in c()] for n, c in calls.items()}
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(fa, "LIB_PATH", fa_build.build(variant="waittest"))
        m.setattr(fa, "_lib", None)
        for name, call in calls.items():
            call()
            torch.cuda.synchronize()
            assert fa.fa_last_device_status() == 1, name
            assert fa.fa_last_device_status() == 0, name
    for name, call in calls.items():
        got = call()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want[name])):
            if (name, i) != ("backward", 0):       # dq: the order of additions may differ
                assert torch.equal(a, b), (name, i)
    assert fa.fa_last_device_status() == 0


def test_tensors_that_do_not_fit(fa):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=DEV)
    q, k = z(2, 4, 8, 64), z(2, 2, 8, 64)
    i32 = z(2, 8, dt=torch.int32)
    ok = dict(q=q, k=k, v=k, key_begin=i32, key_end=i32)
    for bad in (dict(key_begin=i32.long()), dict(key_end=i32[:1]), dict(v=z(2, 2, 9, 64)),
                dict(v=k.half()), dict(k=z(2, 2, 8, 128)), dict(q=q.transpose(1, 2)),
                dict(key_begin=i32.cpu()), dict(slopes=z(3, dt=torch.float32)),
                dict(slopes=z(4))):
        with pytest.raises(ValueError):
            fa.attention_span_forward(**{**ok, **bad})
    with pytest.raises(fa.FAError) as e:
        fa.attention_span_forward(q.float(), k.float(), k.float(), i32, i32)
    assert e.value.code == -2
    kc, tab, n = z(5, 2, 16, 64), z(2, 3, dt=torch.int32), z(2, dt=torch.int32)
    ok = dict(q=q, k_cache=kc, v_cache=kc, block_table=tab, seq_lens=n)
    for bad in (dict(seq_lens=n[:1]), dict(seq_lens=n.long()), dict(block_table=tab.long()),
                dict(v_cache=kc[:4]), dict(k_cache=kc.half()), dict(block_table=tab.cpu()),
                dict(k_cache=kc.transpose(1, 2)), dict(slopes=z(2, dt=torch.float32))):
        with pytest.raises(ValueError):
            fa.decode_forward_ragged(**{**ok, **bad})
    t = z(32, dt=torch.int64)
    ok = dict(q=q, k=k, turns=t)
    for bad in (dict(turns=t.int()), dict(turns=t.cpu()), dict(k=z(2, 2, 7, 64)), dict(k=k.half()),
                dict(positions=i32.long()), dict(positions=i32[:1]),
                dict(q_weight=z(32), k_weight=z(32)), dict(q=q.transpose(2, 3))):
        with pytest.raises((ValueError, fa.FAError)):
            fa.qk_norm_rope_forward(**{**ok, **bad})
    with pytest.raises(ValueError, match="overlap"):
        fa.fa_qk_norm_rope(q, k, q[:, :1].expand(2, 4, 8, 64), k, t)
    with pytest.raises(fa.FAError):
        fa.qk_norm_rope_forward(z(2, 4, 8, 68)[..., 2:66], k, t)     # not 16-byte aligned
