"""Calls of the operators that drop tokens from a paged cache that are refused before any CUDA call."""

import pytest

P = 1 << 20


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_382_b200 import build

    build.build()
    from paged_kv_cache_382_b200 import pa as binding

    return binding


@pytest.mark.parametrize("lens,ctx,budgets,S", [(P, P, 2 * P, 1), (P, 2 * P, P, 4), (P + 12, P, 2 * P, 4), (P, 2 * P, P + 12, 4)])
def test_select_refuses_lengths_over_its_inputs(pa, lens, ctx, budgets, S):
    """keep_lens is written by one CTA of a sequence while others read the lengths and budgets."""
    assert pa.lib.pa_select_tokens(8 * P, lens, 4 * P, ctx, budgets, S, 2, 64, 64, 3, None, None) == pa.PA_ERR_INVALID_ARG
