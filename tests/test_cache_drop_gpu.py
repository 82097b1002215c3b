"""GPU parity of the operators that drop tokens from a paged cache
(pa_decode_weights, pa_select_tokens, pa_compact) against the fp64 oracle.

Tolerances, derived before the first run (u = 2^-24, half a step of fp32):
  * a logit is a sum of d products accumulated in fp32: its error is at most
    d * u * sum |q_i k_i| * scale, here |x| stays below 8 and the sum of
    magnitudes below 30 for standard normal rows of d <= 128 scaled by d^-1/2;
    so a logit is off by less than 128 * 2^-24 * 30 < 2.3e-4 in the worst case.
    A weight is exp of it over the sum: off by a factor within 1 +- 5e-4 (numerator and sum),
    plus the hardware exp2's 2^-22.  A total of g heads' weights is below g, its
    own sum rounds by less than g * 2^-23; bound: 6e-4 * (the exact weights' sum) + 2^-22 * |total|.
  * outputs: the bounds of the decode attention tests (1e-5 fp32, 2e-3 bf16).
  * selections and moves are exact.
"""

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_382_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    from paged_kv_cache_382_b200 import build

    build.build()
    from paged_kv_cache_382_b200 import pa as binding

    return binding


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def batch(ctx, Hq, Hkv, d, B, dtype, seed=3, poison=True, P=512):
    step = W.independent("drop", list(ctx), dtype=dtype, num_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_size=B,
                         seed=seed, device="cuda", partition_size=P, poison=poison)
    # the step's own new token is already counted in context_lens: write it
    return step


def ready(pa, step):
    """Pools with the step's new tokens written, tables and lengths on the device."""
    kc, vc = step.k_cache.clone(), step.v_cache.clone()
    pa.reshape_and_cache(step.new_key, step.new_value, kc, vc, torch.from_numpy(step.slot_mapping).cuda())
    return (kc, vc, torch.from_numpy(np.ascontiguousarray(step.block_tables, dtype=np.int32)).cuda(),
            torch.from_numpy(np.ascontiguousarray(step.context_lens, dtype=np.int32)).cuda())


# (context lengths, Hq, Hkv, d, B, partition): groups of 1, 2, 3, 4, 5, 8 and 16 heads, ragged
# lengths around tiles and partitions, an empty context, one token
CASES = [
    ([7, 16, 33, 100], 4, 4, 64, 16, 512),
    ([1, 0, 15, 17, 257], 8, 4, 128, 16, 64),
    ([31, 2, 1025], 9, 3, 64, 8, 128),
    ([300, 1, 64], 32, 8, 128, 32, 512),
    ([129, 5, 513], 10, 2, 64, 4, 96),
    ([2049, 63], 16, 2, 128, 16, 512),
    ([70, 600], 32, 2, 64, 8, 256),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", CASES)
def test_decode_weights_matches_oracle(pa, case, dtype):
    ctx, Hq, Hkv, d, B, P = case
    step = batch(ctx, Hq, Hkv, d, B, dtype, P=P)
    kc, vc, tables, lens = ready(pa, step)
    S, stride = len(ctx), tables.shape[1] * B + 3
    w_in = torch.rand(S, Hkv, stride, device="cuda")
    w_out = torch.full_like(w_in, -7.0)
    out = torch.empty(S, Hq, d, dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.decode_weights(out, w_out, step.q, kc, vc, tables, lens, step.scale, weights_in=w_in, partition_size=P,
                      dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    k64, v64 = f64(kc), f64(vc)
    ref = oracle.decode_attention(f64(step.q), k64, v64, step.block_tables, step.context_lens, step.scale)
    assert np.abs(f64(out) - ref).max() <= (1e-5 if dtype == torch.float32 else 2e-3)
    exact = oracle.attention_weights(f64(step.q), k64, step.block_tables, step.context_lens, step.scale)
    got, before = f64(w_out), f64(w_in)
    for s, c in enumerate(ctx):
        total = before[s, :, :c] + exact[s]
        assert np.all(np.abs(got[s, :, :c] - total) <= 6e-4 * exact[s] + 2.0 ** -22 * total), (s, c)
        assert np.all(got[s, :, c:] == -7.0)          # entries behind the context stay
    if dtype == torch.bfloat16:   # the output is that of pa_decode, bit for bit (no block is shared)
        plain = torch.empty_like(out)
        pa.decode(plain, step.q, kc, vc, tables, lens, step.scale, partition_size=P)
        assert torch.equal(plain, out)


def test_decode_weights_in_place_lengths_and_start_from_nothing(pa):
    """In place, in two steps, equals one step after another out of place; weights_lens cuts off what
    lies behind the old context; weights_in None starts at zero."""
    step = batch([90, 1, 300, 17], 8, 2, 128, 16, torch.bfloat16)
    kc, vc, tables, lens = ready(pa, step)
    S, Hkv, stride = 4, 2, tables.shape[1] * 16
    out = torch.empty(S, 8, 128, dtype=torch.bfloat16, device="cuda")
    first = torch.zeros(S, Hkv, stride, device="cuda")
    pa.decode_weights(out, first, step.q, kc, vc, tables, lens, step.scale)
    again = torch.zeros_like(first)
    pa.decode_weights(out, again, step.q, kc, vc, tables, lens, step.scale, weights_in=torch.zeros_like(first))
    assert torch.equal(first, again)
    two = torch.zeros_like(first)
    pa.decode_weights(out, two, step.q, kc, vc, tables, lens, step.scale, weights_in=first)
    pa.decode_weights(out, first, step.q, kc, vc, tables, lens, step.scale, weights_in=first)
    assert torch.equal(first, two)
    assert torch.allclose(first, 2 * again)          # twice the same fp32 number: exact
    stale = torch.full_like(again, float("nan"))
    cut = lens - 1
    for s, c in enumerate(cut.tolist()):
        stale[s, :, :c] = again[s, :, :c]
    pa.decode_weights(out, stale, step.q, kc, vc, tables, lens, step.scale, weights_in=stale, weights_lens=cut)
    for s, c in enumerate(lens.tolist()):
        assert torch.equal(stale[s, :, :c - 1], two[s, :, :c - 1])
        assert torch.equal(stale[s, :, c - 1], again[s, :, c - 1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode_weights_bad_block_has_no_weight(pa, dtype):
    step = batch([200, 100], 8, 4, 64, 16, dtype, P=64)
    kc, vc, tables, lens = ready(pa, step)
    tables[0, 3] = kc.shape[0]
    out = torch.empty(2, 8, 64, dtype=torch.float32, device="cuda")
    w = torch.full((2, 4, tables.shape[1] * 16), 5.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.decode_weights(out, w, step.q, kc, vc, tables, lens, step.scale, partition_size=64, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pa.DEVERR_BLOCK_ID
    assert torch.all(w[0, :, 48:64] == 0)
    assert torch.allclose(w[0, :, :200].sum(-1), torch.full((4,), 2.0, device="cuda"), atol=1e-5)
    assert torch.isfinite(out).all()


def test_decode_weights_graph_replay_and_other_stream(pa):
    """Captured on a stream of its own and replayed over new inputs: the same as eager calls."""
    step = batch([500, 33, 1200], 16, 4, 128, 16, torch.bfloat16)
    kc, vc, tables, lens = ready(pa, step)
    cap = tables.shape[1] * 16
    ws = pa.alloc_weights_workspace(3, 16, 128, cap)
    out = torch.empty(3, 16, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(3, 4, cap, device="cuda")
    q = step.q.clone()
    call = lambda: pa.decode_weights(out, w, q, kc, vc, tables, lens, step.scale, weights_in=w, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    w.zero_()
    want = torch.zeros_like(w)
    for k in range(3):
        q.copy_(step.q * (k + 1) * 0.5)
        graph.replay()
        ref = torch.empty_like(out)
        pa.decode_weights(ref, want, q, kc, vc, tables, lens, step.scale, weights_in=want)
        torch.cuda.synchronize()
        assert torch.equal(ref, out) and torch.equal(want, w)


# ---------------------------------------------------------------------------
# select
# ---------------------------------------------------------------------------

def run_select(pa, w, lens, budgets, recent, width):
    S, Hkv, _ = w.shape
    keep = torch.full((S, Hkv, width), -9, dtype=torch.int32, device="cuda")
    keep_lens = torch.full((S,), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.select_tokens(keep, keep_lens, w, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                     torch.tensor(budgets, dtype=torch.int32, device="cuda"), recent=recent, dev_err=err)
    torch.cuda.synchronize()
    return keep.cpu().numpy(), keep_lens.cpu().numpy(), int(err.item())


def check_select(pa, w, lens, budgets, recent, width):
    keep, keep_lens, err = run_select(pa, w, lens, budgets, recent, width)
    assert err == 0
    host = w.cpu().numpy()
    for s, c in enumerate(lens):
        assert keep_lens[s] == min(c, budgets[s])
        for h in range(w.shape[1]):
            ref = oracle.select_tokens(host[s, h], c, budgets[s], recent)
            assert keep[s, h, :keep_lens[s]].tolist() == ref, (s, h)
            assert np.all(keep[s, h, keep_lens[s]:] == -9)


def totals(shape, seed, kind):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.empty(shape, device="cuda").normal_(generator=g)
    if kind == "weights":      # many orders of magnitude, a tenth exactly zero
        return (2 * w - 4).exp_() * (torch.rand(shape, device="cuda", generator=g) > 0.1)
    if kind == "ties":         # a handful of values, negative ones and both zeros among them
        return (w * 1.5).round() * 0.5
    if kind == "zeros":
        return torch.zeros(shape, device="cuda")
    w[..., ::7] = float("nan")
    w[..., 1::11] = float("inf")
    w[..., 2::13] = float("-inf")
    return w


@pytest.mark.parametrize("kind", ["weights", "ties", "zeros", "odd values"])
@pytest.mark.parametrize("recent", [0, 1, 64])
def test_select_matches_oracle(pa, kind, recent):
    lens = [0, 1, 2, 33, 100, 511, 777, 1000]
    budgets = [5, 1, 1, 32, 100, 0, 200, 999]
    check_select(pa, totals((len(lens), 3, 1000), 5, kind), lens, budgets, recent, 1000)


@pytest.mark.parametrize("stride,kind", [(4097, "weights"), (9001, "ties"), (20000, "weights"), (40001, "zeros"),
                                         (70000, "weights"), (131072, "ties"), (131073, "weights")])
def test_select_long_rows_over_clusters(pa, stride, kind):
    lens = [stride, stride - 1, 1, stride // 3, 0]
    budgets = [stride // 4, 1, 7, stride // 3 - 1, 3]
    check_select(pa, totals((5, 2, stride), 6, kind), lens, budgets, 129, stride // 3)


def test_select_rows_too_long_to_hold(pa):
    """Rows of more than 8 x 16384 candidates are read again in every pass instead of held."""
    stride = 8 * 48 * 1024 + 1000
    w = totals((1, 1, stride), 7, "weights")
    k = 5000
    keep, keep_lens, err = run_select(pa, w, [stride], [k], 0, k)
    assert err == 0 and keep_lens[0] == k
    order = w[0, 0].double().sort(descending=True, stable=True).indices[:k].sort().values
    assert keep[0, 0].tolist() == order.tolist()


def test_select_clamps_and_flags(pa):
    w = totals((2, 2, 64), 8, "weights")
    keep, keep_lens, err = run_select(pa, w, [100, -3], [40, 5], 4, 32)
    assert err == pa.DEVERR_CONTEXT
    assert keep_lens.tolist() == [32, 0]
    assert keep[0, 0].tolist() == oracle.select_tokens(w[0, 0].cpu().numpy(), 64, 32, 4)
    assert np.all(keep[1] == -9)


# ---------------------------------------------------------------------------
# compact
# ---------------------------------------------------------------------------

def pools(NB, Hkv, B, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.empty(NB, Hkv, B, d, dtype=dtype, device="cuda").normal_(generator=g)
    v = torch.empty(NB, Hkv, B, d, dtype=dtype, device="cuda").normal_(generator=g)
    k[0, 0, 0, 0] = float("nan")     # copies move bits, whatever they are
    return k, v


def tables_for(lens, B, rng, extra=0, base=0):
    per = [(c + B - 1) // B for c in lens]
    ids = rng.permutation(sum(per) + extra) + base
    t = np.full((len(lens), max(max(per), 1)), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(per):
        t[s, :n] = ids[at:at + n]
        at += n
    return t, sum(per) + extra


def check_compact(pa, k, v, src, dst, keep, keep_lens, starts=None, with_totals=True):
    S, Hkv = len(keep_lens), k.shape[1]
    kb, vb = bits(k).numpy(), bits(v).numpy()
    ref_k, ref_v = oracle.compact(kb, vb, src, dst, keep, keep_lens, starts)
    dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    width = src.shape[1] * k.shape[2]
    w = torch.rand(S, Hkv, width, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ds = dev(src)
    dd = ds if dst is src else dev(dst)
    w_ref = w.clone()
    for s in range(S):
        for h in range(Hkv):
            row = keep[s][h if len(keep[s]) > 1 else 0][: keep_lens[s]]
            at = 0 if starts is None else int(starts[s])
            w_ref[s, h, at:at + len(row)] = w[s, h, torch.as_tensor(np.asarray(row, dtype=np.int64), device="cuda")]
    extra = dict(weights_in=w, weights_out=w) if with_totals else {}
    w_before = w.clone()
    pa.compact(k, v, ds, dd, dev(keep), dev(keep_lens), starts=dev(starts), dev_err=err, **extra)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert np.array_equal(bits(k).numpy(), ref_k) and np.array_equal(bits(v).numpy(), ref_v)
    assert torch.equal(w, w_ref if with_totals else w_before)


def random_keep(rng, lens, heads, share, width=None):
    n = [min(c, max(1, int(c * share))) if c else 0 for c in lens]
    width = width or max(max(n), 1)
    keep = np.full((len(lens), heads, width), -1, dtype=np.int32)
    for s, c in enumerate(lens):
        for h in range(heads):
            keep[s, h, : n[s]] = np.sort(rng.choice(c, n[s], replace=False)) if c else []
    return keep, np.array(n, dtype=np.int32)


@pytest.mark.parametrize("dtype,d,B", [(torch.bfloat16, 64, 4), (torch.bfloat16, 128, 16), (torch.float32, 64, 8),
                                       (torch.float32, 128, 32)])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("share", [0.03, 0.5, 0.97, 1.0])
def test_compact_matches_oracle(pa, dtype, d, B, in_place, share):
    rng = np.random.default_rng(B + d)
    lens = [1, 0, 700, 65, 33, 2000, 7]
    Hkv = 3
    src, n = tables_for(lens, B, rng, extra=5)
    keep, keep_lens = random_keep(rng, lens, Hkv, share)
    dst, total = src, n
    if not in_place:
        dst, more = tables_for(keep_lens.tolist(), B, rng, extra=2, base=n)
        total = n + more
    k, v = pools(total, Hkv, B, d, dtype, 1)
    check_compact(pa, k, v, src, dst, keep, keep_lens)


def test_compact_many_sequences_take_whole_rows(pa):
    """Enough (sequence, head) walks that a CTA moves whole rows instead of slices of them."""
    rng = np.random.default_rng(4)
    lens = rng.integers(1, 90, size=100).tolist()
    src, n = tables_for(lens, 16, rng, extra=3)
    keep, keep_lens = random_keep(rng, lens, 4, 0.6)
    k, v = pools(n, 4, 16, 128, torch.bfloat16, 2)
    check_compact(pa, k, v, src, src, keep, keep_lens)


def test_compact_one_long_sequence_in_place(pa):
    """Many chunks of one walk, sources and destinations interleaved all along."""
    rng = np.random.default_rng(9)
    lens = [30000]
    src, n = tables_for(lens, 16, rng)
    keep, keep_lens = random_keep(rng, lens, 1, 0.8)
    k, v = pools(n, 1, 16, 128, torch.bfloat16, 3)
    check_compact(pa, k, v, src, src, keep, keep_lens)


def test_compact_accepted_paths(pa):
    """keep_heads 1 and starts: the accepted path of a verified tree moves up behind the prefix."""
    rng = np.random.default_rng(5)
    lens, nodes = [40, 16, 130, 9], [12, 16, 64, 1]
    src, n = tables_for(lens, 16, rng, extra=2)
    starts = np.array([c - m for c, m in zip(lens, nodes)], dtype=np.int32)
    keep_lens = np.array([5, 1, 9, 1], dtype=np.int32)
    keep = np.full((4, 1, 9), -1, dtype=np.int32)
    for s in range(4):
        keep[s, 0, : keep_lens[s]] = starts[s] + np.sort(rng.choice(nodes[s], keep_lens[s], replace=False))
    k, v = pools(n, 2, 16, 64, torch.bfloat16, 6)
    check_compact(pa, k, v, src, src, keep, keep_lens, starts=starts, with_totals=False)


def test_compact_shared_block_replaced(pa):
    """One table entry replaced by a fresh block, the others in place: the shared block keeps its
    contents for its other user."""
    rng = np.random.default_rng(6)
    src, n = tables_for([100], 16, rng, extra=4)
    dst = src.copy()
    free = [b for b in range(n) if b not in src.tolist()[0]]
    dst[0, 0] = free[0]
    keep, keep_lens = random_keep(rng, [100], 2, 0.5)
    k, v = pools(n, 2, 16, 64, torch.float32, 7)
    before = k[int(src[0, 0])].clone()
    check_compact(pa, k, v, src, dst, keep, keep_lens)
    assert torch.equal(bits(k[int(src[0, 0])]), bits(before))


def test_compact_flags_and_skips(pa):
    rng = np.random.default_rng(8)
    src, n = tables_for([64, 64], 16, rng)
    k, v = pools(n, 1, 16, 64, torch.float32, 9)
    k0, v0 = k.clone(), v.clone()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    tables = dev(src.tolist())

    def call(keep, lens, starts=None, dst=None, srct=None):
        k.copy_(k0)
        v.copy_(v0)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.compact(k, v, tables if srct is None else srct, tables if dst is None else dst, dev(keep), dev(lens),
                   starts=None if starts is None else dev(starts), dev_err=err)
        torch.cuda.synchronize()
        return int(err.item())

    same = lambda: torch.equal(bits(k), bits(k0)) and torch.equal(bits(v), bits(v0))  # noqa: E731
    assert call([[[0, 0]], [[0, 1]]], [2, 2]) == pa.DEVERR_COPY and same()        # 0 would move up to 1
    assert call([[[64]], [[70]]], [1, 1]) == pa.DEVERR_COPY and same()            # past the table
    assert call([[[-5]], [[0]]], [1, 1]) == pa.DEVERR_COPY and same()
    assert call([[[0]], [[0]]], [-1, 0]) == pa.DEVERR_CONTEXT and same()
    assert call([[[0]], [[0]]], [1, 1], starts=[-1, 0]) == pa.DEVERR_CONTEXT and same()
    bad = tables.clone()
    bad[0, 1] = n
    assert call([[[20]], [[0]]], [1, 1], srct=bad) == pa.DEVERR_BLOCK_ID and same()
    assert call([[[17]], [[0]]], [1, 1], dst=torch.full_like(tables, -1)) == pa.DEVERR_BLOCK_ID and same()


def test_weights_select_compact_decode_in_a_row(pa):
    """An eviction as a serving step runs it: decode keeps totals, a selection reads them, the kept rows
    move into the table's own blocks, and the next decode attends to exactly the kept tokens."""
    ctx, Hq, Hkv, d, B = [300, 40, 513, 65], 8, 2, 128, 16
    step = batch(ctx, Hq, Hkv, d, B, torch.bfloat16)
    kc, vc, tables, lens = ready(pa, step)
    S, stride = len(ctx), tables.shape[1] * B
    w = torch.zeros(S, Hkv, stride, device="cuda")
    out = torch.empty(S, Hq, d, dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.decode_weights(out, w, step.q, kc, vc, tables, lens, step.scale, dev_err=err)
    budgets = torch.tensor([100, 64, 200, 33], dtype=torch.int32, device="cuda")
    keep = torch.zeros(S, Hkv, 200, dtype=torch.int32, device="cuda")
    new_lens = torch.zeros(S, dtype=torch.int32, device="cuda")
    pa.select_tokens(keep, new_lens, w, lens, budgets, recent=16, dev_err=err)
    k0, v0, w0 = f64(kc), f64(vc), w.clone()
    pa.compact(kc, vc, tables, tables, keep, new_lens, weights_in=w, weights_out=w, dev_err=err)
    pa.decode_weights(out, w, step.q, kc, vc, tables, new_lens, step.scale, weights_in=w, weights_lens=new_lens,
                      dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    got, g = f64(out), Hq // Hkv
    for s in range(S):
        n = int(new_lens[s])
        assert n == min(ctx[s], int(budgets[s]))
        for h in range(Hkv):
            pos = oracle.select_tokens(w0[s, h].cpu().numpy(), ctx[s], int(budgets[s]), 16)
            rows = oracle.gather_kv(k0, step.block_tables[s], ctx[s], h)[pos]
            vals = oracle.gather_kv(v0, step.block_tables[s], ctx[s], h)[pos]
            for n_h in range(h * g, (h + 1) * g):
                ref = oracle.decode_attention_one(f64(step.q[s, n_h]), rows, vals, step.scale)
                assert np.abs(got[s, n_h] - ref).max() <= 2e-3
            kept = f64(w0[s, h])[pos]
            assert np.all(f64(w[s, h])[: n] >= kept * (1 - 2.0 ** -22))
