"""CPU checks of the operators that drop tokens from a paged cache: pins of their oracle, refusals of
their entry points before any launch, and the block manager's side of a compaction."""

import numpy as np
import pytest

import oracle
from paged_kv_cache_382_b200.blocks import BlockManager, BlockPool, OutOfBlocks


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_382_b200 import build

    build.build()
    from paged_kv_cache_382_b200 import pa as binding

    return binding


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------

def paged(rng, ctx, Hkv, d, B):
    nb = [-(-c // B) for c in ctx]
    ids = rng.permutation(sum(nb) + 2)
    tables = np.full((len(ctx), max(nb)), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(nb):
        tables[s, :n] = ids[at:at + n]
        at += n
    shape = (sum(nb) + 2, Hkv, B, d)
    return rng.standard_normal(shape), rng.standard_normal(shape), tables


def test_tree_attention_of_a_chain_is_causal_prefill():
    """A tree without branches masks exactly like a causal chunk."""
    rng = np.random.default_rng(1)
    ctx, new = [9, 20, 70], [3, 1, 66]
    k, v, tables = paged(rng, ctx, 2, 8, 4)
    start = np.concatenate([[0], np.cumsum(new)])
    q = rng.standard_normal((sum(new), 4, 8))
    mask = []
    for n in new:
        for i in range(n):
            m = (1 << (i + 1)) - 1
            mask.append([m & (2 ** 64 - 1), m >> 64])
    got = oracle.tree_attention(q, k, v, tables, ctx, start, mask, 0.3)
    ref = oracle.prefill_attention(q, k, v, tables, ctx, start, 0.3)
    assert np.abs(got - ref).max() < 1e-13


def test_tree_attention_siblings_do_not_see_each_other():
    """Two siblings after a prefix of 2: each equals plain attention over the prefix and itself; a row
    that sees nothing is zero."""
    rng = np.random.default_rng(2)
    k, v, tables = paged(rng, [4], 1, 8, 4)
    q = rng.standard_normal((2, 1, 8))
    got = oracle.tree_attention(q, k, v, tables, [4], [0, 2], [[1], [2]], 0.5)
    kr, vr = oracle.gather_kv(k, tables[0], 4, 0), oracle.gather_kv(v, tables[0], 4, 0)
    for i, seen in enumerate([[0, 1, 2], [0, 1, 3]]):
        ref = oracle.decode_attention_one(q[i, 0], kr[seen], vr[seen], 0.5)
        assert np.abs(got[i, 0] - ref).max() < 1e-14
    none = oracle.tree_attention(q, k, v, tables, [2], [0, 2], [[0], [3]], 0.5)
    assert np.all(none[0] == 0) and np.any(none[1] != 0)


def test_attention_weights_sum_to_the_group_and_reproduce_the_output():
    rng = np.random.default_rng(3)
    ctx = [7, 1, 0]
    k, v, tables = paged(rng, ctx, 2, 8, 4)
    q = rng.standard_normal((3, 6, 8))
    w = oracle.attention_weights(q, k, tables, ctx, 0.4)
    assert np.allclose(w[0].sum(-1), 3) and np.allclose(w[1], 3) and w[2].shape == (2, 0)
    one = oracle.attention_weights(q[:, :2], k, tables, ctx, 0.4)   # one query head per kv head
    out = oracle.decode_attention(q[:, :2], k, v, tables, ctx, 0.4)
    for h in range(2):
        assert np.allclose(one[0][h] @ oracle.gather_kv(v, tables[0], 7, h), out[0, h])


def test_select_tokens_hand_worked():
    w = np.array([0.5, 2.0, 0.5, 0.0, 9.0, 0.1, 3.0])
    assert oracle.select_tokens(w, 7, 4, 2) == [1, 4, 5, 6]
    assert oracle.select_tokens(w, 7, 5, 2) == [0, 1, 4, 5, 6]      # the tie at 0.5 goes to position 0
    assert oracle.select_tokens(w, 3, 5, 1) == [0, 1, 2]
    assert oracle.select_tokens(w, 7, 2, 5) == [5, 6]
    assert oracle.select_tokens(w, 7, 0, 3) == []
    assert oracle.select_tokens(np.array([np.nan, -1.0, -np.inf, -0.0, 0.0]), 5, 3, 0) == [1, 3, 4]


def test_compact_oracle_reads_before_it_writes():
    k = np.arange(8.0).reshape(2, 1, 4, 1)
    out, _ = oracle.compact(k, k, [[1, 0]], [[1, 0]], [[[1, 2, 5]]], [3])
    # logical order 4 5 6 7 0 1 2 3; positions 1, 2, 5 move to 0, 1, 2
    assert out[1, 0, :, 0].tolist() == [5, 6, 1, 7] and out[0, 0, :, 0].tolist() == [0, 1, 2, 3]


# ---------------------------------------------------------------------------
# refusals (before any CUDA call)
# ---------------------------------------------------------------------------

P = 1 << 20


def weights_call(pa, **over):
    a = dict(out=P, od=0, wo=P, wi=None, wl=None, stride=128, q=P, k=P, v=P, t=P, c=P, S=2, Hq=4, Hkv=2, d=64, B=16,
             NB=8, mb=8, mc=0, scale=0.1, P=512, ws=P, wsb=1 << 30, dt=0, err=None, st=None)
    a.update(over)
    return pa.lib.pa_decode_weights(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(S=0), 0), (dict(wo=None), 1), (dict(wo=P + 2), 1), (dict(wi=P + 1), 1), (dict(wl=P + 2), 1),
    (dict(stride=127), 1), (dict(stride=64, mc=65), 1), (dict(ws=None), 1), (dict(wsb=100), 3), (dict(d=96), 2),
    (dict(Hq=5), 1), (dict(Hq=514), 2), (dict(B=5), 2), (dict(od=1), 2), (dict(scale=float("inf")), 1), (dict(q=None), 1),
    (dict(S=1 << 26, mc=8, stride=128), 2),
])
def test_decode_weights_refusals(pa, over, status):
    assert weights_call(pa, **over) == status


def test_decode_weights_workspace(pa):
    f, d = pa.lib.pa_decode_weights_workspace_bytes, pa.lib.pa_decode_workspace_bytes
    r = lambda n: (n + 255) // 256 * 256  # noqa: E731
    # one partition: its (max, sum) is kept too; every case: a logit per head and token
    assert f(3, 8, 64, 300, 512) == d(3, 8, 64, 300, 512) + r(3 * 8 * 8) + r(3 * 8 * 300 * 4)
    assert f(3, 8, 64, 2000, 512) == d(3, 8, 64, 2000, 512) + r(3 * 8 * 2000 * 4)
    assert f(64, 64, 128, 131072, 512) > 2 ** 31
    assert f(-1, 8, 64, 300, 512) == 0 and f(1, 8, 64, 300, 0) == 0


@pytest.mark.parametrize("args,status", [
    ((P, P, P, P, P, 0, 2, 64, 64, 3), 0), ((None, P, P, P, P, 1, 2, 64, 64, 3), 1), ((P, P, P, P, None, 1, 2, 64, 64, 3), 1),
    ((P, P, P + 2, P, P, 1, 2, 64, 64, 3), 1), ((P, P, P, P, P, 1, 0, 64, 64, 3), 1), ((P, P, P, P, P, 1, 2, 0, 64, 3), 1),
    ((P, P, P, P, P, 1, 2, 64, 0, 3), 1), ((P, P, P, P, P, 1, 2, 64, 64, -1), 1),
    ((P, P, P, P, P, 1 << 28, 4, 64, 64, 3), 2),
])
def test_select_refusals(pa, args, status):
    assert pa.lib.pa_select_tokens(*args, None, None) == status


def compact_call(pa, **over):
    a = dict(k=P, v=P, wo=None, wi=None, stride=0, src=P, dst=P, smb=4, dmb=4, keep=P, kh=2, ks=16, starts=None, lens=P,
             S=1, Hkv=2, d=64, B=16, NB=8, dt=1, err=None, st=None)
    a.update(over)
    return pa.lib.pa_compact(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(S=0), 0), (dict(k=None), 1), (dict(k=P + 8), 1), (dict(src=None), 1), (dict(dst=P + 2), 1), (dict(keep=None), 1),
    (dict(lens=None), 1), (dict(kh=3), 1), (dict(ks=0), 1), (dict(d=32), 2), (dict(B=64), 2), (dict(dt=3), 1),
    (dict(wo=P), 1), (dict(wi=P), 1), (dict(wo=P, wi=P, stride=0), 1), (dict(starts=P + 1), 1), (dict(S=-1), 1),
    (dict(smb=0), 1), (dict(dmb=1 << 30), 1),
])
def test_compact_refusals(pa, over, status):
    assert compact_call(pa, **over) == status


def test_binding_shape_checks(pa):
    import torch

    f, i = torch.zeros(2, 3, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.select_tokens(torch.zeros(2, 2, 4, dtype=torch.int32), i, f, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        pa.select_tokens(torch.zeros(2, 3, 4, dtype=torch.int32), i, f, i, i)
    k = torch.zeros(4, 3, 16, 64)
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="come together"):
        pa.compact(k, k.clone(), t, t, torch.zeros(2, 3, 4, dtype=torch.int32), i, weights_in=f)
    with pytest.raises(ValueError):
        pa.compact(k, k.clone(), t, t, torch.zeros(2, 2, 4, dtype=torch.int32), i)


# ---------------------------------------------------------------------------
# the block manager's side
# ---------------------------------------------------------------------------

def test_bm_compact_cuts_and_frees(pa):
    bm = pa.NativeBlockManager(8, 4)
    bm.add(1)
    bm.append(1, 19)
    table = bm.block_table(1)
    assert bm.compact([1], [6], [9]) == []
    assert bm.block_table(1) == table[:3] and bm.num_tokens(1) == 9 and bm.num_free == 5
    slots, copies, _ = bm.append(1, 4)           # fills block 2, then takes a block
    assert copies == [] and [int(x) for x in slots[:3]] == [table[2] * 4 + 1 + i for i in range(3)]
    assert bm.compact([1], [0], [0]) == [] and bm.block_table(1) == [] and bm.num_free == 8
    bm.append(1, 1)
    assert bm.num_tokens(1) == 1


def test_bm_compact_replaces_shared_blocks(pa):
    bm = pa.NativeBlockManager(10, 4)
    bm.add(1)
    bm.append(1, 14)
    bm.fork(1, 2)
    old = bm.block_table(1)
    copies = bm.compact([1], [6], [11])          # blocks 1 and 2 receive tokens, block 1 keeps two
    new = bm.block_table(1)
    assert new[0] == old[0] and len(new) == 3 and not set(new[1:]) & set(old)
    assert copies == [(old[1], new[1])]
    assert bm.block_table(2) == old and [bm.ref_count(b) for b in old] == [2, 1, 1, 1]


def test_bm_compact_batch_never_hands_out_a_source(pa):
    """Both sharers compact in one call: both get fresh blocks, and the old ones are free only after."""
    bm = pa.NativeBlockManager(6, 4)
    bm.add(1)
    bm.append(1, 12)
    bm.fork(1, 2)
    old = bm.block_table(1)
    with pytest.raises(pa.PagedAttentionError):
        bm.compact([1, 2], [0, 0], [8, 8])       # four fresh blocks, three free: nothing changes
    assert bm.block_table(1) == old and bm.block_table(2) == old and bm.num_free == 3
    assert bm.compact([1, 2], [0, 0], [4, 8]) == []
    a, b = bm.block_table(1), bm.block_table(2)
    assert not set(a + b) & set(old) and len(set(a + b)) == 3 and bm.num_free == 3


def test_bm_compact_refusals(pa):
    bm = pa.NativeBlockManager(8, 4)
    bm.add(1)
    bm.append(1, 10)
    for ids, u, n in [([2], [0], [0]), ([1, 1], [0, 0], [1, 1]), ([1], [-1], [4]), ([1], [5], [4]), ([1], [0], [11])]:
        with pytest.raises(pa.PagedAttentionError):
            bm.compact(ids, u, n)
        assert bm.num_tokens(1) == 10
    with pytest.raises(ValueError):
        bm.compact([1], [0], [4], token_ids=[1, 2, 3])


def test_bm_compact_prefix_cache_with_known_ids(pa):
    """A rejected draft leaves the cache, the accepted tokens enter it as if they had been appended."""
    bm = pa.NativeBlockManager(32, 4, prefix_cache=True)
    bm.add(1)
    bm.append(1, [1, 2, 3, 4, 5])
    bm.append(1, [10, 11, 12, 13, 14, 15])       # a draft; [5, 10, 11, 12] was cached as a block
    bm.compact([1], [5], [9], token_ids=[10, 13, 20, 21])
    assert bm.num_tokens(1) == 9
    bm.add(2)
    assert bm.append(2, [1, 2, 3, 4, 5, 10, 11, 12])[2] == 4      # the rejected block is not found
    bm.add(3)
    assert bm.append(3, [1, 2, 3, 4, 5, 10, 13, 20, 21])[2] == 8  # the accepted one is
    assert bm.block_table(3)[:2] == bm.block_table(1)[:2]
    bm.append(1, [22, 23, 24])                   # [21, 22, 23, 24] chains on
    bm.add(4)
    assert bm.append(4, [1, 2, 3, 4, 5, 10, 13, 20, 21, 22, 23, 24])[2] == 12


def test_bm_compact_prefix_cache_with_unknown_ids(pa):
    """After an eviction the sequence's blocks hold no known prefix: the ones it kept are not found
    again (the dropped ones, still whole, are), and it looks none up."""
    bm = pa.NativeBlockManager(32, 4, prefix_cache=True)
    bm.add(1)
    toks = list(range(1, 17))
    bm.append(1, toks)
    old = bm.block_table(1)
    bm.compact([1], [0], [8])
    bm.add(2)
    assert bm.append(2, toks)[2] == 8
    assert bm.block_table(2)[2:] == old[2:] and not set(bm.block_table(2)[:2]) & set(old)
    bm.append(1, toks[8:])                       # would match sequence 2's blocks by id alone
    assert bm.append(1, toks)[2] == 0
    assert bm.num_tokens(1) == 32 and not set(bm.block_table(1)) & set(bm.block_table(2))


def test_bm_compact_cut_inside_a_cached_block(pa):
    """Cut inside a full, cached block: later tokens overwrite its slots, so it leaves the cache; one
    that another sequence still holds stays, and the writer copies."""
    bm = pa.NativeBlockManager(32, 4, prefix_cache=True)
    bm.add(1)
    bm.append(1, [1, 2, 3, 4])
    bm.compact([1], [2], [2])
    bm.add(2)
    assert bm.append(2, [1, 2, 3, 4])[2] == 0
    bm.add(3)
    assert bm.append(3, [1, 2, 3, 4])[2] == 4    # sequence 2's block
    bm.compact([3], [3], [3])
    _, copies, _ = bm.append(3, [9])
    assert len(copies) == 1 and copies[0][0] == bm.block_table(2)[0]
    bm.add(4)
    assert bm.append(4, [1, 2, 3, 4])[2] == 4


def test_bm_compact_lockstep_with_the_python_manager(pa):
    """Random appends, forks, compactions and frees: the native manager and its Python twin give the
    same tables, copies, counts and free blocks."""
    rng = np.random.default_rng(12)
    for _ in range(20):
        NB, B = 40, 4
        order = rng.permutation(NB)
        native, pool = pa.NativeBlockManager(NB, B, free_order=order), BlockPool(NB, order)
        twin, seqs, nxt = BlockManager(pool, B), {}, 0
        for _ in range(120):
            op = rng.integers(0, 5)
            ids = list(seqs)
            if op == 0 or not ids:
                seqs[nxt] = twin.new_sequence()
                native.add(nxt)
                nxt += 1
            elif op == 1:
                s = int(rng.choice(ids))
                n = int(rng.integers(1, 9))
                if pool.num_free * B > n + 2 * B:
                    _, copies = twin.append_tokens(seqs[s], n)
                    assert native.append(s, n)[1] == copies
            elif op == 2:
                s = int(rng.choice(ids))
                seqs[nxt] = twin.fork(seqs[s])
                native.fork(s, nxt)
                nxt += 1
            elif op == 3:
                some = [int(x) for x in rng.permutation(ids)[: rng.integers(1, 4)]]
                n = [int(rng.integers(0, seqs[x].num_tokens + 1)) for x in some]
                u = [int(rng.integers(0, x + 1)) for x in n]
                try:
                    copies = twin.compact([seqs[x] for x in some], u, n)
                    assert native.compact(some, u, n) == copies
                except OutOfBlocks:
                    with pytest.raises(pa.PagedAttentionError):
                        native.compact(some, u, n)
            else:
                s = int(rng.choice(ids))
                twin.free(seqs.pop(s))
                native.free(s)
            assert native.num_free == pool.num_free
            for x, sq in seqs.items():
                assert native.block_table(x) == sq.block_table and native.num_tokens(x) == sq.num_tokens
            assert [native.ref_count(b) for b in range(NB)] == pool.ref_cnt.tolist()


# ---------------------------------------------------------------------------
# trees
# ---------------------------------------------------------------------------

def tree_call(pa, **over):
    a = dict(out=P, od=0, q=P, k=P, v=P, t=P, c=P, qs=P, m=P, words=1, S=2, T=6, Hq=4, Hkv=2, d=64, B=16, NB=8, mb=8, mc=0,
             scale=0.1, ws=P, wsb=1 << 30, dt=1, err=None, st=None)
    a.update(over)
    return pa.lib.pa_tree_decode(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(T=0, S=0), 0), (dict(S=0), 1), (dict(T=-1), 1), (dict(q=None), 1), (dict(m=None), 1), (dict(m=P + 4), 1),
    (dict(qs=P + 2), 1), (dict(words=0), 1), (dict(words=9), 2), (dict(d=256), 2), (dict(B=12), 2), (dict(Hq=5), 1),
    (dict(od=1, dt=0), 2), (dict(ws=None), 1), (dict(ws=P + 16), 1), (dict(wsb=1000), 3), (dict(scale=float("nan")), 1),
    (dict(NB=1 << 28), 2), (dict(mb=1 << 28), 1), (dict(S=1 << 20), 2), (dict(mc=-1), 1), (dict(dt=2), 1),
])
def test_tree_decode_refusals(pa, over, status):
    assert tree_call(pa, **over) == status


def test_tree_workspace_does_not_grow_with_the_batch(pa):
    f = pa.lib.pa_tree_workspace_bytes
    assert f(1, 32, 128) < f(8, 32, 128) == f(4096, 32, 128) < 64 << 20
    assert f(-1, 32, 128) == 0 and f(1, 0, 128) == 0


def test_tree_mask_from_parents(pa):
    m = pa.tree_mask([-1, 0, 0, 1, -1])
    assert m.tolist() == [[1], [3], [5], [11], [16]]
    rng = np.random.default_rng(3)
    parents = [-1] + [int(rng.integers(-1, i)) for i in range(1, 130)]
    m = pa.tree_mask(parents, 4).numpy().astype(np.uint64)
    for i in range(130):
        seen, j = set(), i
        while j >= 0:
            seen.add(j)
            j = parents[j]
        assert seen == {b for b in range(256) if (int(m[i, b // 64]) >> (b % 64)) & 1}
    for bad in ([0], [-1, 1], [-1, 2, 0]):
        with pytest.raises(pa.PagedAttentionError):
            pa.tree_mask(bad)
    with pytest.raises(pa.PagedAttentionError):
        pa.tree_mask([-1] * 65, 1)
    assert pa.tree_mask([]).shape == (0, 1)
