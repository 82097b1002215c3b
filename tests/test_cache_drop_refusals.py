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


@pytest.mark.parametrize("stride,width", [(2 ** 31 - 1, 64), (2 ** 31 - 2 ** 15, 64), (64, 2 ** 31 - 1)])
def test_rows_near_the_end_of_32_bits(pa, stride, width):
    """A kernel's segments and pages end past the row's own end, which still has to fit 32 bits."""
    assert pa.lib.pa_select_tokens(8 * P, P, 4 * P, 2 * P, 3 * P, 2, 2, stride, width, 3, None, None) == pa.PA_ERR_UNSUPPORTED
    if width > 64:
        assert pa.lib.pa_compact(P, P, None, None, 0, P, P, 4, 4, P, 2, width, None, P, 1, 2, 64, 16, 8, 1, None,
                                 None) == pa.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("blocks,bound,ok", [(2 ** 27 - 1, 0, False), (2 ** 27 - 1, 2 ** 31 - 100, False), (2 ** 27 - 1, 4096, True)])
def test_tree_contexts_near_the_end_of_32_bits(pa, blocks, bound, ok):
    rc = pa.lib.pa_tree_decode(P, 0, P, P, P, P, P, P, P, 1, 1, 0 if ok else 6, 4, 2, 64, 16, 8, blocks, bound, 0.1, P, 1 << 30, 1, None,
                               None)
    assert rc == (pa.PA_OK if ok else pa.PA_ERR_UNSUPPORTED)


def test_weights_of_contexts_near_the_end_of_32_bits(pa):
    n = 2 ** 27 - 1
    assert pa.lib.pa_decode_weights(P, 0, P, None, None, 2 ** 31 - 1, P, P, P, P, P, 1, 4, 2, 64, 16, 8, n, 0, 0.1, 8192, P, 1 << 40, 0,
                                    None, None) == pa.PA_ERR_UNSUPPORTED


def test_python_manager_refuses_what_the_native_one_does():
    """A sequence named twice, lengths that are not one per sequence or do not fit it: nothing changes."""
    from paged_kv_cache_382_b200.blocks import BlockManager, BlockPool

    pool = BlockPool(8)
    bm = BlockManager(pool, 4)
    a = bm.new_sequence()
    bm.append_tokens(a, 10)
    b = bm.fork(a)
    before = (list(a.block_table), list(b.block_table), a.num_tokens, pool.num_free, pool.ref_cnt.tolist())
    for seqs, u, n in [([a, a], [0, 0], [4, 4]), ([a, b], [0], [4]), ([a], [0], [4, 4]), ([a, b], [0, 5], [4, 4]), ([a, b], [0, 0], [4, 11])]:
        with pytest.raises(ValueError):
            bm.compact(seqs, u, n)
        assert before == (list(a.block_table), list(b.block_table), a.num_tokens, pool.num_free, pool.ref_cnt.tolist())
    assert bm.compact([a, b], [4, 0], [4, 4]) == []
