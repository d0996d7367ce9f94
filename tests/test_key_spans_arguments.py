"""key_spans: negative windows and lengths are refused instead of hiding every key, and document
lengths may come as a tensor like the other lengths."""
import pytest
import torch


@pytest.mark.parametrize("kw", [dict(window=-1), dict(kv_lens=-1), dict(kv_lens=[3, -2]),
                                dict(prefix_lens=-4), dict(prefix_lens=[0, -1])])
def test_negative_lengths_are_refused(fa_lib, kw):
    with pytest.raises(ValueError):
        fa_lib.key_spans(2, 8, **kw)


@pytest.mark.parametrize("docs", [[3, 5], [[3, 5], [1, 6]]])
def test_document_lengths_as_a_tensor(fa_lib, docs):
    want = fa_lib.key_spans(2, 8, doc_lens=docs)
    for form in (torch.tensor(docs), torch.tensor(docs, dtype=torch.int32),
                 [torch.tensor(d) for d in docs] if isinstance(docs[0], list) else tuple(docs)):
        got = fa_lib.key_spans(2, 8, doc_lens=form)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
