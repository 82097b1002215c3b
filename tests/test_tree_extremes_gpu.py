"""pa_tree_decode and pa_decode_weights at the ends of their ranges: as many nodes as a mask row holds, many query heads
to a kv head, one of each, several sequences over the same blocks.  Bounds as in the tests beside it."""

import numpy as np
import pytest
import torch

import oracle
from test_cache_drop_gpu import ready
from test_tree_gpu import close, f64, inputs, reference, run
from paged_kv_cache_382_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from paged_kv_cache_382_b200 import build

    build.build()
    from paged_kv_cache_382_b200 import pa as binding

    return binding


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ctx,nodes,Hq,Hkv,d,B,words,kind", [
    ([600], [512], 2, 1, 64, 16, 8, "any"),           # every bit of the widest mask row
    ([513, 512], [511, 512], 1, 1, 128, 32, 8, "tree"),
    ([200, 190], [150, 190], 2, 2, 64, 4, 3, "any"),  # an odd number of words, no prefix
    ([70, 300], [3, 2], 256, 1, 64, 16, 1, "tree"),   # 256 query heads to a kv head
    ([40, 9], [5, 1], 130, 2, 128, 8, 2, "tree"),     # a group that no row tile holds a multiple of
])
def test_tree_at_the_ends_of_its_range(pa, ctx, nodes, Hq, Hkv, d, B, words, kind, dtype):
    step, q, mask, start = inputs(ctx, nodes, Hq, Hkv, d, B, dtype, kind=kind, words=words)
    out, err = run(pa, step, q, mask, start)
    assert err == 0
    close(out, reference(step, q, mask, start), dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sequences_that_share_blocks(pa, dtype):
    """Samples of one prompt: each verifies and keeps totals by itself, as with blocks of its own."""
    step = W.shared_prefix(prompt_len=96, suffix_max=50, prompts=2, samples=4, num_heads=8, num_kv_heads=2, head_dim=64, block_size=16,
                           device="cuda")
    kc, vc, tables, lens = ready(pa, step)
    kc, vc, q = kc.to(dtype), vc.to(dtype), step.q.to(dtype)
    S, ctx = len(step.context_lens), [int(c) for c in step.context_lens]
    out = torch.empty(S, 8, 64, dtype=torch.float32, device="cuda")
    w = torch.zeros(S, 2, tables.shape[1] * 16, device="cuda")
    pa.decode_weights(out, w, q, kc, vc, tables, lens, step.scale)
    ref = oracle.decode_attention(f64(q), f64(kc), f64(vc), step.block_tables, step.context_lens, step.scale)
    tol = 1e-5 if dtype == torch.float32 else 2e-3
    assert np.abs(f64(out) - ref).max() <= tol
    exact = oracle.attention_weights(f64(q), f64(kc), step.block_tables, step.context_lens, step.scale)
    for s, c in enumerate(ctx):
        assert np.all(np.abs(f64(w[s, :, :c]) - exact[s]) <= 6e-4 * exact[s] + 2.0 ** -22)
    # the last token of each as a draft of one node
    start, mask = np.arange(S + 1, dtype=np.int32), np.ones((S, 1), dtype=np.int64)
    t_out = torch.empty_like(out)
    pa.tree_decode(t_out, q, kc, vc, tables, lens, torch.from_numpy(start).cuda(), torch.from_numpy(mask).cuda(), step.scale)
    assert np.abs(f64(t_out) - ref).max() <= tol
