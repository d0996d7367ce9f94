"""NaN and overflowing scores where a row of span attention sees them: out and lse say so, as the
causal calls' do, and the gradients take no such row for one that sees nothing."""
import pytest
import torch

from bounds import DT

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def inputs(d, dtype, S=300, Hq=4, Hkv=2):
    g = torch.Generator().manual_seed(d)
    r = lambda H: torch.randn(1, H, S, d, generator=g).to(DT[dtype]).to(DEV)
    return r(Hq), r(Hkv), r(Hkv), r(Hq)


def plant(where, q, k):
    if where == "query":
        q[0, 1, 140, 7] = float("nan")
    elif where == "key":
        k[0, 1, 133, 5] = float("nan")
    elif where == "infinite key":
        k[0, 0, 20] = float("inf")
    else:   # the row's only score is -infinity: its weights have no sum
        q[0, 2, 0], k[0, 1, 0] = 200.0, 0.0
        q[0, 2, 0, 0], k[0, 1, 0, 0] = 3e38 if q.dtype == torch.bfloat16 else 6e4, float("-inf")


def same(a, b):
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


@pytest.mark.parametrize("where", ["query", "key", "infinite key", "only score"])
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16")])
def test_as_the_causal_call(fa, where, d, dtype):
    q, k, v, _ = inputs(d, dtype)
    plant(where, q, k)
    begin, end = fa.key_spans(1, 300, device=DEV)
    out, lse = fa.attention_span_forward(q, k, v, begin, end)
    out2, lse2 = fa.attention_forward(q, k, v)
    torch.cuda.synchronize()
    assert out2.isnan().any() and (where == "only score" or lse2.isnan().any())
    assert same(out, out2) and same(lse, lse2)


@pytest.mark.parametrize("softcap,alibi", [(0.0, False), (20.0, False), (0.0, True), (20.0, True)])
@pytest.mark.parametrize("d", [64, 128])
def test_lse_says_nan_where_out_does(fa, softcap, alibi, d):
    """Rows that see the NaN: NaN in out and lse. Rows that do not: finite. Rows that see nothing:
    zeros and -infinity, beside them."""
    q, k, v, _ = inputs(d, "bf16")
    k[0, 1, 133, 5] = float("nan")
    begin, end = fa.key_spans(1, 300, doc_lens=[100, 60, 70], device=DEV)
    sl = torch.tensor([0.5, 0.25, 0.1, 0.05], device=DEV) if alibi else None
    out, lse = fa.attention_span_forward(q, k, v, begin, end, softcap, sl)
    torch.cuda.synchronize()
    bad = torch.zeros(1, 4, 300, dtype=torch.bool, device=DEV)
    bad[0, 2:, 133:160] = True
    assert torch.equal(lse.isnan(), bad) and torch.equal(out.isnan().all(-1), bad)
    assert torch.equal(out.isnan().any(-1), bad)
    none = (end <= begin)[:, None].expand_as(lse)
    assert none.any() and torch.equal(lse == float("-inf"), none) and (out[none] == 0).all()


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16")])
def test_gradients_of_a_nan_row(fa, d, dtype):
    q, k, v, do = inputs(d, dtype)
    q[0, 1, 140, 7] = float("nan")
    begin, end = fa.key_spans(1, 300, device=DEV)
    out, lse = fa.attention_span_forward(q, k, v, begin, end)
    got = fa.attention_span_backward(q, k, v, out, do, lse, begin, end)
    out2, lse2 = fa.attention_forward(q, k, v)
    want = fa.attention_backward(q, k, v, out2, do, lse2)
    torch.cuda.synchronize()
    assert fa.fa_last_device_status() == 0
    assert got[2][0, 0, :141].isnan().all()      # dv of every key the row sees
    for a, b in zip(got, want):
        assert torch.equal(a.isnan(), b.isnan())
