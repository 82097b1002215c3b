"""pa_compact over several pages of pairs in place, pa_decode_weights with bf16 outputs, and calls from several host
threads at once.  Bounds as in the tests they add to."""

import threading

import numpy as np
import pytest
import torch

import oracle
from test_cache_drop_gpu import batch, check_compact, f64, pools, random_keep, ready, tables_for
from test_tree_gpu import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from paged_kv_cache_382_b200 import build

    build.build()
    from paged_kv_cache_382_b200 import pa as binding

    return binding


@pytest.mark.parametrize("dtype,d,S,Hkv", [(torch.bfloat16, 128, 40, 8), (torch.float32, 64, 75, 4), (torch.bfloat16, 64, 20, 8)])
@pytest.mark.parametrize("share", [0.4, 0.98])
def test_compact_in_place_over_pages_of_pairs(pa, dtype, d, S, Hkv, share):
    """Whole rows or half rows per CTA and up to 700 pairs of a walk: pages of 256 pairs are found while others move."""
    rng = np.random.default_rng(d + S)
    lens = [int(x) for x in rng.integers(200, 720, size=S)]
    lens[0] = 719
    src, n = tables_for(lens, 16, rng, extra=3)
    keep, keep_lens = random_keep(rng, lens, Hkv, share)
    k, v = pools(n, Hkv, 16, d, dtype, 2)
    check_compact(pa, k, v, src, src, keep, keep_lens)


@pytest.mark.parametrize("P", [64, 512])
def test_decode_weights_bf16_output(pa, P):
    """Half a bf16 step, 2^-8 of the value, on top of the fp32 output's bound."""
    step = batch([1, 33, 700, 2500], 10, 2, 128, 16, torch.bfloat16, P=P)
    kc, vc, tables, lens = ready(pa, step)
    out = torch.empty(4, 10, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(4, 2, tables.shape[1] * 16, device="cuda")
    pa.decode_weights(out, w, step.q, kc, vc, tables, lens, step.scale, partition_size=P)
    ref = oracle.decode_attention(f64(step.q), f64(kc), f64(vc), step.block_tables, step.context_lens, step.scale)
    assert np.all(np.abs(f64(out) - ref) <= 2e-3 + np.abs(ref) * 2.0 ** -8)


def test_calls_from_several_host_threads(pa):
    """Each thread has a stream, workspaces and outputs of its own; what it gets is what one thread gets."""
    step = batch([500, 33, 1200], 16, 4, 128, 16, torch.bfloat16)
    kc, vc, tables, lens = ready(pa, step)
    cap = tables.shape[1] * 16
    tree, q, mask, start = inputs([300, 90], [20, 30], 16, 4, 128, 16, torch.bfloat16)
    dev = lambda x, t=np.int32: torch.from_numpy(np.ascontiguousarray(x, dtype=t)).cuda()  # noqa: E731
    t_tables, t_lens, t_start, t_mask = dev(tree.block_tables), dev(tree.context_lens), dev(start), dev(mask, np.int64)

    def work(stream, res):
        w = torch.zeros(3, 4, cap, device="cuda")
        out, keep = torch.zeros_like(step.q), torch.zeros(3, 4, 100, dtype=torch.int32, device="cuda")
        kept, t_out = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros_like(q)
        budgets = torch.tensor([100, 40, 64], dtype=torch.int32, device="cuda")
        k2, v2 = kc.clone(), vc.clone()
        for _ in range(20):
            pa.decode_weights(out, w, step.q, kc, vc, tables, lens, step.scale, weights_in=w, stream=stream)
            pa.tree_decode(t_out, q, tree.k_cache, tree.v_cache, t_tables, t_lens, t_start, t_mask, tree.scale, stream=stream)
            pa.select_tokens(keep, kept, w, lens, budgets, recent=8, stream=stream)
        pa.compact(k2, v2, tables, tables, keep, kept, weights_in=w, weights_out=w, stream=stream)
        res += [out, w, t_out, keep, kept, k2, v2]

    def on(stream, res):
        with torch.cuda.stream(stream):
            work(stream, res)

    torch.cuda.synchronize()
    results = [[] for _ in range(5)]
    on(torch.cuda.Stream(), results[0])
    torch.cuda.synchronize()
    threads = [threading.Thread(target=on, args=(torch.cuda.Stream(), r)) for r in results[1:]]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for r in results[1:]:
        assert len(r) == len(results[0])
        for got, want in zip(r, results[0]):
            assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
