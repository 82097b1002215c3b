"""pa_tree_decode over long runs: the output's accuracy does not fall with the length of the context.

The tensor cores add a product to an accumulator in tensor memory by cutting off what does not fit 24 bits, so an
accumulator that takes N products in a row comes out too small by up to N * 2^-23, half of that on average.  The kernel
folds it into a 32-bit sum every 64 steps of 8 products: N <= 512.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from paged_kv_cache_382_b200 import build

    build.build()
    from paged_kv_cache_382_b200 import pa as binding

    return binding


# (sequences over one context, its length, nodes, query heads, head_dim, block, out rows of one unit).  More units than
# SMs, so that a CTA works through whole contexts; one row tile (streams take half a tile each) and two
@pytest.mark.parametrize("S,ctx,n,Hq,d,B", [(300, 131072, 1, 8, 64, 32), (160, 70001, 3, 5, 128, 16), (150, 40000, 17, 8, 128, 8),
                                            (2, 131072, 2, 3, 64, 4)])
def test_error_does_not_grow_with_the_run(pa, S, ctx, n, Hq, d, B):
    dev, gen = "cuda", torch.Generator(device="cuda").manual_seed(ctx + n)
    blocks = -(-ctx // B)
    perm = torch.randperm(blocks, generator=torch.Generator().manual_seed(1))
    k = torch.empty(blocks, 1, B, d, device=dev, dtype=torch.bfloat16).normal_(generator=gen)
    v = (torch.empty(blocks, 1, B, d, device=dev).normal_(generator=gen) + 1).to(torch.bfloat16)   # sums that grow all along
    q = torch.empty(S * n, Hq, d, device=dev, dtype=torch.bfloat16).normal_(generator=gen)
    tables = perm.to(torch.int32).cuda().expand(S, blocks).contiguous()
    lens = torch.full((S,), ctx, dtype=torch.int32, device=dev)
    start = (torch.arange(S + 1, dtype=torch.int32) * n).cuda()
    mask = torch.tensor([(1 << (i + 1)) - 1 for i in range(n)] * S, dtype=torch.int64).reshape(-1, 1).cuda()
    out = torch.empty(q.shape, dtype=torch.float32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    scale = d ** -0.5
    pa.tree_decode(out, q, k, v, tables, lens, start, mask, scale, dev_err=err)
    assert int(err.item()) == 0
    at = torch.arange(ctx, device=dev)
    keys, values = (x[tables[0].long()[at // B], 0, at % B].double() for x in (k, v))
    scale64 = float(np.float32(scale))
    worst = shrink = 0.0
    some = list(range(0, S * n, max(1, S * n // 64)))      # 64 rows in 64 bits, from all over the batch
    for t in some:
        x = q[t].double() @ keys.T * scale64
        x[:, ctx - n + t % n + 1:] = -torch.inf
        ref = torch.softmax(x, -1) @ values
        off = out[t].double() / ref - 1
        worst = max(worst, float(off.abs().max()))
        shrink += float(off.mean()) / len(some)
    # 512 products, half of 2^-23 each on average; another 2^-17 for weights of 16 bits
    assert abs(shrink) <= 512 * 2.0 ** -24, shrink
    assert worst <= 512 * 2.0 ** -23 + 2.0 ** -17, worst
