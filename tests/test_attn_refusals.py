"""Refusals of the attention calls that name what is wrong: heads of no columns, messages."""
import pytest

torch = pytest.importorskip("torch")
DEV = "cuda:0"


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_token_amd as g
    g.load_library()
    return g


@pytest.mark.gpu
def test_heads_of_no_columns(gdn):
    q, k = torch.empty(2, 5, 4, 0, device=DEV), torch.empty(2, 5, 2, 0, device=DEV)
    lse = torch.empty(2, 5, 4, device=DEV)
    cu = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    table, lengths = (torch.zeros(s, dtype=torch.int32, device=DEV) for s in ((2, 1), (2,)))
    cache = torch.empty(1, 16, 2, 0, device=DEV)
    for call in (lambda: gdn.gdn_attn_prefill(q, k, k),
                 lambda: gdn.gdn_attn_varlen_prefill(q[0], k[0], k[0], cu),
                 lambda: gdn.gdn_attn_backward(q, q, k, k, q, lse),
                 lambda: gdn.gdn_attn_varlen_backward(q[0], q[0], k[0], k[0], q[0], lse[0], cu),
                 lambda: gdn.gdn_attn_decode(q, cache, cache, table, lengths)):
        with pytest.raises(gdn.GDNError, match="size is out of range"):
            call()


def test_message_of_an_unsupported_call(gdn):
    """Whoever passes heads of 96 columns, or pages of 24 tokens, reads what there is."""
    text = gdn.load_library().gdn_status_string(3).decode()
    assert "attention: 64, 128 or 256" in text and "page size" in text
    assert str(gdn.GDNError(3, text)).endswith(text)
