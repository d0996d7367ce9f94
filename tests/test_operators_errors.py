"""Errors of the span, ragged and query/key-preparation calls, without a GPU: their texts name
the kind of argument that is wrong."""
import pytest

from test_operators_abi import P, heads, heads_bwd, ragged, span_bwd, span_fwd


@pytest.mark.parametrize("call,kw,names", [
    (span_fwd, dict(softcap=-1.0), "softcap"), (ragged, dict(softcap=1e30), "softcap"),
    (heads, dict(rope_scale=float("inf")), "rope_scale"), (heads, dict(wq=P, wk=P, eps=-1.0), "eps"),
    (span_fwd, dict(dtype=0), "this call"), (ragged, dict(dtype=0), "this call"),
    (ragged, dict(bs=24), "block_size"), (ragged, dict(window=-1), "window"),
    (ragged, dict(Sq=33), "Hq / Hkv * Sq"), (heads, dict(rope_dim=8), "rope_dim"),
    (span_fwd, dict(begin=P + 2), "4"), (heads, dict(turns=P + 4), "8"),
    (heads, dict(q=(P, 4)), "stride"), (span_bwd, dict(ws=P + 16), "256"),
    (heads_bwd, dict(ws=P + 16), "256"),
    (heads_bwd, dict(ws_bytes=16), "_workspace_bytes"), (ragged, dict(ws=None), "_workspace_bytes"),
])
def test_text_names_the_argument(fa_lib, call, kw, names):
    code = call(fa_lib if call in (heads, heads_bwd) else fa_lib.lib(), **kw)
    text = fa_lib.fa_strerror(code)
    assert code < 0 and names in text, text
    assert "fa_bwd_workspace_bytes" not in text
