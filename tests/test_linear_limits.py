"""pa_linear_attention's refusals at the end of its range (no GPU: the calls return before they
look for one)."""
import pytest

import paged_kv_cache_284_gb300 as pk
from test_hybrid_host import linear


@pytest.mark.parametrize("tokens", [(1 << 30) + 1, 2**31 - 1])
def test_more_than_2_30_tokens_are_refused(tokens):
    assert linear(T=tokens) == pk.PA_ERR_UNSUPPORTED
    assert b"2^30 tokens" in pk.lib().pa_last_error_message()


def test_the_most_tokens_meet_the_other_checks():
    assert linear(T=1 << 30, ws=None) == pk.PA_ERR_WORKSPACE
