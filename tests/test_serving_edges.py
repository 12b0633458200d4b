"""Host checks of the serving calls at their edges: what is allowed is not refused (CPU only)."""
import pytest

from bit_weight_only_tq_amd import _lib
from test_serving_checks import ATTN, call


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_attention_of_no_tokens(lib):
    """A step in which every request rests has no new tokens, and none as the most of a request."""
    assert call(lib, "tq_paged_attention", ATTN, T=0, max_q=0) == "TQ_OK"
    assert call(lib, "tq_paged_attention", ATTN, T=0, max_q=0, max_kv=0, q=None) == "TQ_OK"
    assert call(lib, "tq_paged_attention", ATTN, T=0, max_q=-1) == "TQ_ERR_SHAPE"
    assert call(lib, "tq_paged_attention", ATTN, T=1, max_q=0) == "TQ_ERR_SHAPE"
