"""GPU parity of pa_tree_decode against the fp64 oracle, on both attend kernels.

Tolerances: the bounds of the decode attention tests (1e-5 for fp32 pools, 2e-3
for bf16 pools with fp32 output); a bf16 output adds half a bf16 step of the
exact value, 2^-8 relative.
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


def random_masks(rng, nodes, words, kind):
    rows = []
    for n in nodes:
        seen = []
        for i in range(n):
            if kind == "tree":
                p = int(rng.integers(-1, i)) if i else -1
                seen.append((seen[p] if p >= 0 else 0) | (1 << i))
            elif kind == "any":       # any set, itself or not, nodes behind it too, bits past n
                seen.append(int.from_bytes(rng.bytes(8 * words), "little"))
            else:
                seen.append(0)
        rows += [[(m >> (64 * w)) & (2 ** 64 - 1) for w in range(words)] for m in seen]
    return np.array(rows, dtype=np.uint64).reshape(-1, words).view(np.int64)


def inputs(ctx, nodes, Hq, Hkv, d, B, dtype, kind="tree", seed=1, words=None, poison=True):
    step = W.independent("tree", list(ctx), dtype=dtype, num_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_size=B,
                         seed=seed, device="cuda", poison=poison)
    kc, vc = step.k_cache, step.v_cache
    # the step's one new token per sequence is in the context: write it with the history
    for t, slot in enumerate(step.slot_mapping):
        if slot >= 0:
            kc[int(slot) // B, :, int(slot) % B] = step.new_key[t]
            vc[int(slot) // B, :, int(slot) % B] = step.new_value[t]
    rng = np.random.default_rng(seed)
    words = words or max(1, -(-max(nodes) // 64))
    mask = random_masks(rng, nodes, words, kind)
    start = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    T = int(start[-1])
    q = torch.randn(T, Hq, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(dtype)
    return step, q, mask, start


def run(pa, step, q, mask, start, out_dtype=torch.float32, tables=None, ctx=None, scale=None, **kw):
    dev = lambda x, t: torch.from_numpy(np.ascontiguousarray(x, dtype=t)).cuda()  # noqa: E731
    out = torch.full(q.shape, -77.0, dtype=out_dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.tree_decode(out, q, step.k_cache, step.v_cache, dev(step.block_tables if tables is None else tables, np.int32),
                   dev(step.context_lens if ctx is None else ctx, np.int32), dev(start, np.int32),
                   torch.from_numpy(mask).cuda(), step.scale if scale is None else scale, dev_err=err, **kw)
    torch.cuda.synchronize()
    return out, int(err.item())


def reference(step, q, mask, start, scale=None):
    return oracle.tree_attention(f64(q), f64(step.k_cache), f64(step.v_cache), step.block_tables, step.context_lens,
                                 start, mask.tolist(), step.scale if scale is None else scale)


def close(out, ref, dtype):
    got = f64(out)
    assert np.all(np.isfinite(got))
    tol = 1e-5 if dtype == torch.float32 else 2e-3
    extra = np.abs(ref) * 2.0 ** -8 if out.dtype == torch.bfloat16 else 0.0
    worst = float((np.abs(got - ref) - extra).max())
    assert worst <= tol, worst


# (contexts, nodes, Hq, Hkv, d, B): one row; row tiles just below, at and above 128 and 256 rows; several row
# blocks; contexts at the edges of a 64- or 128-token tile; drafts longer than the rest of the context; a
# sequence without nodes; groups that do not divide 128; a context that is all nodes
CASES = [
    ([1], [1], 1, 1, 64, 16),
    ([5, 64, 65, 128], [1, 3, 4, 5], 4, 4, 64, 16),
    ([127, 129, 300, 256], [32, 33, 31, 1], 8, 2, 128, 16),
    ([700, 40, 90], [64, 40, 65], 8, 2, 128, 8),
    ([1000, 3, 513], [16, 0, 2], 32, 8, 128, 32),
    ([200, 333], [43, 7], 12, 4, 128, 16),
    ([150, 450], [100, 130], 5, 1, 64, 8),
    ([65, 260], [2, 37], 16, 2, 128, 16),
    ([2100], [17], 8, 8, 64, 32),
    ([90, 17], [9, 4], 8, 4, 64, 4),
    ([301, 1023, 4], [17, 40, 3], 32, 8, 128, 4),
    ([130, 2055], [45, 6], 12, 2, 64, 4),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
def test_tree_matches_oracle(pa, case, dtype):
    ctx, nodes, Hq, Hkv, d, B = case
    step, q, mask, start = inputs(ctx, nodes, Hq, Hkv, d, B, dtype)
    assert pa.tree_uses_tensor_cores(dtype, B) == (dtype == torch.bfloat16)
    out, err = run(pa, step, q, mask, start)
    assert err == 0
    close(out, reference(step, q, mask, start), dtype)


@pytest.mark.parametrize("B", [16, 4])
@pytest.mark.parametrize("kind", ["any", "none"])
def test_tree_any_mask(pa, kind, B):
    """Any set of nodes, its own bit or not; none at all; rows that see nothing (no prefix, empty mask) are zero."""
    ctx, nodes = [30, 30, 200, 64], [30, 12, 70, 64]
    step, q, mask, start = inputs(ctx, nodes, 4, 2, 64, B, torch.bfloat16, kind=kind)
    mask[3] = 0          # a node of sequence 0, which has no prefix
    out, err = run(pa, step, q, mask, start)
    assert err == 0
    close(out, reference(step, q, mask, start), torch.bfloat16)
    assert torch.all(out[3] == 0)
    if kind == "none":
        assert torch.all(out[:30] == 0) and torch.all(out[int(start[3]):] == 0)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_tree_batch_cut_over_the_gpu(pa, out_dtype):
    """Enough tiles that every CTA holds whole units, cut ones and several sequences."""
    rng = np.random.default_rng(4)
    ctx = [int(x) for x in rng.integers(1, 900, size=40)]
    nodes = [min(c, int(x)) for c, x in zip(ctx, rng.integers(0, 70, size=40))]
    step, q, mask, start = inputs(ctx, nodes, 8, 4, 64, 16, torch.bfloat16, words=2)
    out, err = run(pa, step, q, mask, start, out_dtype=out_dtype)
    assert err == 0
    close(out, reference(step, q, mask, start), torch.bfloat16)
    again, _ = run(pa, step, q, mask, start, out_dtype=out_dtype)
    assert torch.equal(out, again)


def test_tree_many_sequences(pa):
    """More sequences than a window of 32, empty ones and one-token contexts among them."""
    rng = np.random.default_rng(5)
    ctx = [int(x) for x in rng.integers(1, 40, size=333)]
    nodes = [int(x) if x < 4 else 0 for x in rng.integers(0, 7, size=333)]
    nodes = [min(a, b) for a, b in zip(nodes, ctx)]
    step, q, mask, start = inputs(ctx, nodes, 4, 2, 64, 8, torch.bfloat16)
    out, err = run(pa, step, q, mask, start)
    assert err == 0
    close(out, reference(step, q, mask, start), torch.bfloat16)


@pytest.mark.parametrize("B", [16, 4])
def test_tree_chain_equals_causal_prefill(pa, B):
    ctx, nodes = [300, 70, 129], [64, 5, 33]
    step, q, mask, start = inputs(ctx, nodes, 8, 2, 128, B, torch.bfloat16)
    chain = np.array([(1 << (i + 1)) - 1 for n in nodes for i in range(n)], dtype=np.uint64)
    mask = chain.reshape(-1, 1).view(np.int64)
    out, err = run(pa, step, q, mask, start)
    assert err == 0
    ref = oracle.prefill_attention(f64(q), f64(step.k_cache), f64(step.v_cache), step.block_tables, step.context_lens,
                                   start, step.scale)
    close(out, ref, torch.bfloat16)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tree_scales(pa, scale, dtype):
    """Zero, negative and large scales (logits of +-100: the running maximum moves)."""
    ctx, nodes = [400, 33], [20, 33]
    step, q, mask, start = inputs(ctx, nodes, 8, 2, 64, 16, dtype)
    out, err = run(pa, step, q, mask, start, scale=scale)
    assert err == 0
    ref = reference(step, q, mask, start, scale=scale)
    # a logit of size x is off by 64 products' roundings, 64 * 2^-24 * sum|q k| * scale < 1e-3 at 1.5
    tol = (2e-3 if dtype == torch.float32 else 4e-3) if abs(scale) > 1 else (1e-5 if dtype == torch.float32 else 2e-3)
    assert np.abs(f64(out) - ref).max() <= tol


def test_tree_errors_and_untouched_rows(pa):
    """A bad block is flagged and its tokens take no part; more nodes than context or than mask words, bad
    contexts and malformed ranges are flagged; rows of no sequence stay as they were."""
    ctx, nodes = [100, 60], [10, 6]
    for dtype in (torch.bfloat16, torch.float32):
        step, q, mask, start = inputs(ctx, nodes, 4, 2, 64, 16, dtype, poison=False)
        qx = torch.cat([q, q[:3]])
        mx = np.concatenate([mask, mask[:3]])
        out, err = run(pa, step, qx, mx, start)
        assert err == 0 and torch.all(out[16:] == -77.0)
        tables = step.block_tables.copy()
        tables[0, 2] = step.num_blocks
        out, err = run(pa, step, q, mask, start, tables=tables)
        assert err == pa.DEVERR_BLOCK_ID
        keep = [p for p in range(100) if not 32 <= p < 48]
        for i in range(10):
            seen = [p for p in keep if p < 90 or (int(mask[i, 0]) >> (p - 90)) & 1]
            for h in range(4):
                k = oracle.gather_kv(f64(step.k_cache), step.block_tables[0], 100, h // 2)[seen]
                v = oracle.gather_kv(f64(step.v_cache), step.block_tables[0], 100, h // 2)[seen]
                ref = oracle.decode_attention_one(f64(q[i, h]), k, v, step.scale)
                assert np.abs(f64(out[i, h]) - ref).max() <= 2e-3
        for bad in ([100, -1], [10 ** 6, 60], [8, 60]):
            out, err = run(pa, step, q, mask, start, ctx=bad, max_context_len=112)   # the first table's seven blocks
            assert err == pa.DEVERR_CONTEXT and torch.isfinite(out).all()
        for bad in ([0, 10, 17], [0, 10, 9], [-1, 10, 16]):
            out, err = run(pa, step, q, mask, np.array(bad, dtype=np.int32))
            assert err == pa.DEVERR_CONTEXT
        out, err = run(pa, step, q, mask, start, ctx=[100, 0])   # nodes without a context see nothing
        assert err == pa.DEVERR_CONTEXT and torch.all(out[10:] == 0)
    step, q, mask, start = inputs([300], [100], 4, 2, 64, 16, torch.bfloat16, words=2)
    out, err = run(pa, step, q, np.ascontiguousarray(mask[:, :1]), start)
    assert err == pa.DEVERR_CONTEXT
    cut = mask.copy()
    cut[:, 1] = 0
    close(out, reference(step, q, cut, start), torch.bfloat16)


def test_tree_capacity_bound_and_workspace_reuse(pa):
    """max_context_len clamps; one workspace serves calls of other sizes in a row."""
    step, q, mask, start = inputs([100, 50], [4, 4], 8, 2, 128, 16, torch.bfloat16)
    ws = pa.alloc_tree_workspace(64, 8, 128)
    out, err = run(pa, step, q, mask, start, workspace=ws, max_context_len=112)
    assert err == 0
    close(out, reference(step, q, mask, start), torch.bfloat16)
    step2, q2, mask2, start2 = inputs([700], [33], 8, 2, 128, 16, torch.bfloat16, seed=9)
    out, err = run(pa, step2, q2, mask2, start2, workspace=ws)
    assert err == 0
    close(out, reference(step2, q2, mask2, start2), torch.bfloat16)
    with pytest.raises(pa.PagedAttentionError):
        run(pa, step, q, mask, start, workspace=ws[:256])


def test_tree_graph_replay_on_its_own_stream(pa):
    step, q, mask, start = inputs([500, 90, 1], [20, 40, 1], 16, 4, 128, 16, torch.bfloat16)
    dev = lambda x, t: torch.from_numpy(np.ascontiguousarray(x, dtype=t)).cuda()  # noqa: E731
    tables, lens, st = dev(step.block_tables, np.int32), dev(step.context_lens, np.int32), dev(start, np.int32)
    m, ws = torch.from_numpy(mask).cuda(), pa.alloc_tree_workspace(q.shape[0], 16, 128)
    qs, out = q.clone(), torch.empty_like(q)
    call = lambda: pa.tree_decode(out, qs, step.k_cache, step.v_cache, tables, lens, st, m, step.scale, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for k in (1.0, 0.5):
        qs.copy_(q * k)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        close(out, reference(step, q * k, mask, start), torch.bfloat16)


def test_verify_and_commit_a_draft(pa):
    """A verification step as a serving loop runs it, through the block manager: drafted tokens appended and
    written, the tree attended to, an accepted path moved up (pa_bm_compact, pa_compact), and the next
    decode equal to plain attention over prefix and path."""
    Hq, Hkv, d, B = 8, 2, 128, 16
    bm = pa.NativeBlockManager(64, B, free_order=np.random.default_rng(3).permutation(64))
    kc = torch.full((64, Hkv, B, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(8)
    hist, prefix = {}, {0: 45, 1: 16}
    scale = d ** -0.5
    kv = lambda n: [torch.from_numpy(rng.standard_normal((n, Hkv, d))).to(torch.bfloat16).cuda() for _ in range(2)]  # noqa: E731
    parents = {0: [-1, 0, 0, 1, 1, 2, 3, 3, 6], 1: [-1, -1, 0, 1, 3]}
    path = {0: [0, 1, 3, 6, 8], 1: [1, 3]}

    def write(seq, n):
        slots, copies, _ = bm.append(seq, n)
        if copies:
            pa.copy_blocks(kc, vc, torch.tensor(copies, dtype=torch.int64, device="cuda"), dev_err=err)
        k, v = kv(n)
        pa.reshape_and_cache(k, v, kc, vc, torch.from_numpy(np.ascontiguousarray(slots)).cuda(), dev_err=err)
        hist.setdefault(seq, [[], []])
        hist[seq][0] += list(k)
        hist[seq][1] += list(v)

    def tables():
        rows = [bm.block_table(s) for s in (0, 1)]
        w = max(map(len, rows))
        return torch.tensor([r + [-1] * (w - len(r)) for r in rows], dtype=torch.int32, device="cuda")

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for s in (0, 1):
        bm.add(s)
        write(s, prefix[s])
    bm.fork(0, 7)                        # sequence 7 keeps sharing sequence 0's blocks
    shared = bm.block_table(7)
    before = kc[shared].clone()
    for s in (0, 1):
        write(s, len(parents[s]))
    n = [len(parents[s]) for s in (0, 1)]
    lens = [prefix[s] + n[s] for s in (0, 1)]
    q = torch.randn(sum(n), Hq, d, device="cuda").to(torch.bfloat16)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    mask = torch.cat([pa.tree_mask(parents[s]) for s in (0, 1)]).cuda()
    pa.tree_decode(out, q, kc, vc, tables(), i32(lens), i32([0, n[0], sum(n)]), mask, scale, dev_err=err)
    got, at = f64(out), 0
    for s in (0, 1):
        for i in range(n[s]):
            seen, j = [], i
            while j >= 0:
                seen.append(prefix[s] + j)
                j = parents[s][j]
            seen = list(range(prefix[s])) + seen[::-1]
            k, v = (np.stack([f64(hist[s][x][p]) for p in seen]) for x in (0, 1))
            for h in range(Hq):
                ref = oracle.decode_attention_one(f64(q[at + i, h]), k[:, h // 4], v[:, h // 4], scale)
                assert np.abs(got[at + i, h] - ref).max() <= 2e-3
        at += n[s]
    src = tables()
    new = [prefix[s] + len(path[s]) for s in (0, 1)]
    copies = bm.compact([0, 1], [prefix[0], prefix[1]], new)
    if copies:
        pa.copy_blocks(kc, vc, torch.tensor(copies, dtype=torch.int64, device="cuda"), dev_err=err)
    width = max(len(path[s]) for s in (0, 1))
    keep = i32([[[prefix[s] + p for p in path[s]] + [-1] * (width - len(path[s]))] for s in (0, 1)])
    pa.compact(kc, vc, src, tables(), keep, i32([len(path[s]) for s in (0, 1)]), starts=i32([prefix[0], prefix[1]]),
               dev_err=err)
    for s in (0, 1):
        for x in (0, 1):
            hist[s][x] = hist[s][x][: prefix[s]] + [hist[s][x][prefix[s] + p] for p in path[s]]
        write(s, 1)
    qd = torch.randn(2, Hq, d, device="cuda").to(torch.bfloat16)
    dout = torch.empty(2, Hq, d, dtype=torch.float32, device="cuda")
    pa.decode(dout, qd, kc, vc, tables(), i32([x + 1 for x in new]), scale, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for s in (0, 1):
        k, v = (np.stack([f64(t) for t in hist[s][x]]) for x in (0, 1))
        for h in range(Hq):
            ref = oracle.decode_attention_one(f64(qd[s, h]), k[:, h // 4], v[:, h // 4], scale)
            assert np.abs(f64(dout[s, h]) - ref).max() <= 2e-3
    assert torch.equal(kc[shared].view(torch.int16), before.view(torch.int16))


def test_tree_overlapping_ranges_stay_in_bounds(pa):
    """A query_start that runs back and forth names rows several times: flagged, no row of another
    sequence's range is touched, nothing faults."""
    ctx, nodes = [40] * 6, [10, 0, 0, 0, 0, 0]
    for dtype in (torch.bfloat16, torch.float32):
        step, q, mask, _ = inputs(ctx, nodes, 4, 2, 64, 16, dtype, poison=False)
        q = torch.cat([q, q])
        mask = np.concatenate([mask, mask])
        out, err = run(pa, step, q, mask, np.array([0, 10, 0, 10, 0, 10, 10], dtype=np.int32))
        assert err == pa.DEVERR_CONTEXT
        assert torch.isfinite(out[:10]).all() and torch.all(out[10:] == -77.0)


@pytest.mark.parametrize("case", [([300, 70], [40, 70], 8, 2, 128, 16), ([200], [100], 8, 2, 64, 8), ([64, 33], [9, 5], 4, 4, 64, 4)])
def test_tree_non_finite_nodes_reach_only_rows_that_see_them(pa, case):
    """NaN and infinities in K and V of some nodes: rows that do not see such a node are the same bit for bit as
    without them; rows that see one are non-finite where plain attention is."""
    ctx, nodes, Hq, Hkv, d, B = case
    step, q, mask, start = inputs(ctx, nodes, Hq, Hkv, d, B, torch.bfloat16)
    clean, err = run(pa, step, q, mask, start)
    assert err == 0
    words = mask.view(np.uint64)
    for which, bad_nodes in (("v", [1, nodes[0] - 1]), ("k", [2])):
        k0, v0 = step.k_cache.clone(), step.v_cache.clone()
        pool = step.v_cache if which == "v" else step.k_cache
        for j, value in zip(bad_nodes, (float("nan"), float("inf"))):
            p = ctx[0] - nodes[0] + j
            pool[int(step.block_tables[0, p // B]), :, p % B, 5] = value
        out, err = run(pa, step, q, mask, start)
        torch.cuda.synchronize()
        assert err == 0
        for i in range(q.shape[0]):
            own = i < nodes[0]
            sees = [j for j in bad_nodes if own and (int(words[i, j // 64]) >> (j % 64)) & 1]
            if not sees:
                assert torch.equal(out[i], clean[i]), (which, i)
            elif which == "v":
                assert not torch.isfinite(out[i, :, 5]).any()
                others = [c for c in range(d) if c != 5]
                assert torch.equal(out[i][:, others], clean[i][:, others])
                if len(sees) == 1 and sees[0] == bad_nodes[1]:
                    assert torch.all(out[i, :, 5] == float("inf"))
            else:
                assert torch.isnan(out[i]).all()
        step.k_cache.copy_(k0)
        step.v_cache.copy_(v0)


def test_tree_blocks_past_four_gigabytes(pa):
    """The pool's last blocks, element offsets above 2^32."""
    Hkv, B, d = 8, 16, 128
    NB = (1 << 32) // (Hkv * B * d) + 64
    kc = torch.empty(NB, Hkv, B, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    ids = [NB - 1, 3, NB - 7, NB - 40]
    for b in ids:
        kc[b].normal_()
        vc[b].normal_()
    ctx, n = 60, 11
    parents = [-1, 0, 0, 1, 1, 2, 2, 3, 4, 5, 6]
    mask = pa.tree_mask(parents).cuda()
    q = torch.randn(n, 16, d, device="cuda").to(torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.tree_decode(out, q, kc, vc, i32([ids]), i32([ctx]), i32([0, n]), mask, d ** -0.5, dev_err=err)
    small_k, small_v = torch.stack([kc[b] for b in ids]), torch.stack([vc[b] for b in ids])
    ref = oracle.tree_attention(f64(q), f64(small_k), f64(small_v), [[0, 1, 2, 3]], [ctx], [0, n],
                                mask.tolist(), d ** -0.5)
    assert int(err.item()) == 0
    close(out, ref, torch.bfloat16)
    # decode with totals and a move inside the same blocks
    w = torch.zeros(1, Hkv, 64, device="cuda")
    dout = torch.empty(1, 16, d, dtype=torch.float32, device="cuda")
    pa.decode_weights(dout, w, q[:1].contiguous(), kc, vc, i32([ids]), i32([ctx]), d ** -0.5, dev_err=err)
    exact = oracle.attention_weights(f64(q[:1]), f64(small_k), [[0, 1, 2, 3]], [ctx], d ** -0.5)[0]
    assert np.abs(f64(w[0, :, :ctx]) - exact).max() <= 6e-4 * exact.max()
    keep = [1, 17, 30, 40, 59]
    pa.compact(kc, vc, i32([ids]), i32([ids]), i32([[keep]]), i32([len(keep)]), dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for j, p in enumerate(keep):
        assert torch.equal(kc[ids[0], :, j], small_k[p // B, :, p % B])
        assert torch.equal(vc[ids[0], :, j], small_v[p // B, :, p % B])
