"""fp64 oracle of the operators that drop tokens from a paged KV cache.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain loops over
sequences and heads, from the definitions in each function's docstring; the
gather through the block table is ``gather_kv`` of the decode oracle.
"""

from __future__ import annotations

import numpy as np

from .paged_attention import gather_kv


def tree_attention(q, k_cache, v_cache, block_tables, context_lens, query_start, tree_mask, scale):
    """Attention of drafted tokens: new token i of sequence s (of n_s) sees every position below
    context_lens[s] - n_s, and new token j when bit j of its mask row is set.

    q [T][Hq][d]; tree_mask [T][words] of 64-bit words, bit j at word j // 64, bit j % 64.  A row that
    sees nothing is zero.  Returns [T][Hq][d] in fp64."""
    T, num_heads, head_dim = q.shape
    num_kv_heads = k_cache.shape[1]
    group = num_heads // num_kv_heads
    out = np.zeros((T, num_heads, head_dim), dtype=np.float64)
    for s in range(len(context_lens)):
        ctx = int(context_lens[s])
        first, last = int(query_start[s]), int(query_start[s + 1])
        n = last - first
        for kvh in range(num_kv_heads):
            k_rows = gather_kv(k_cache, block_tables[s], ctx, kvh)
            v_rows = gather_kv(v_cache, block_tables[s], ctx, kvh)
            for i in range(n):
                words = [int(w) & (2 ** 64 - 1) for w in tree_mask[first + i]]
                seen = [p for p in range(ctx) if p < ctx - n or
                        (p - (ctx - n)) // 64 < len(words) and (words[(p - (ctx - n)) // 64] >> ((p - (ctx - n)) % 64)) & 1]
                if not seen:
                    continue
                for h in range(kvh * group, (kvh + 1) * group):
                    x = float(np.float32(scale)) * (k_rows[seen] @ np.asarray(q[first + i, h], dtype=np.float64))
                    w = np.exp(x - x.max())
                    out[first + i, h] = (w @ v_rows[seen]) / w.sum()
    return out


def attention_weights(q, k_cache, block_tables, context_lens, scale):
    """weights[s][kvh][j]: softmax weight of token j, summed over the query heads of kv head kvh.
    A list of [Hkv][ctx_s] arrays in fp64, one per sequence."""
    num_seqs, num_heads, _ = q.shape
    num_kv_heads = k_cache.shape[1]
    group = num_heads // num_kv_heads
    res = []
    for s in range(num_seqs):
        ctx = int(context_lens[s])
        w = np.zeros((num_kv_heads, ctx))
        for kvh in range(num_kv_heads):
            k_rows = gather_kv(k_cache, block_tables[s], ctx, kvh)
            for h in range(kvh * group, (kvh + 1) * group):
                if ctx:
                    x = float(np.float32(scale)) * (k_rows @ np.asarray(q[s, h], dtype=np.float64))
                    e = np.exp(x - x.max())
                    w[kvh] += e / e.sum()
        res.append(w)
    return res


def select_tokens(weights, context_len, budget, recent):
    """Kept positions of one row of totals: the last min(recent, kept) ones, then the largest totals
    (ties: lowest position; NaN as -inf), ascending."""
    kept = min(int(context_len), int(budget))
    recent = min(int(recent), kept)
    m = int(context_len) - recent
    ranked = sorted(range(m), key=lambda j: (np.inf if np.isnan(weights[j]) else -float(weights[j]), j))
    return sorted(ranked[: kept - recent] + list(range(m, int(context_len))))


def compact(k_cache, v_cache, src_tables, dst_tables, keep, keep_lens, starts=None):
    """Position keep[s][h][j] (through src_tables) goes to starts[s] + j (through dst_tables), all
    sources read before anything is written; keep has one row for all kv heads or one each.  Returns
    new pools."""
    B = k_cache.shape[2]
    k_out, v_out = k_cache.copy(), v_cache.copy()
    for s in range(len(keep_lens)):
        for h in range(k_cache.shape[1]):
            row = keep[s][h if len(keep[s]) > 1 else 0]
            for j in range(int(keep_lens[s])):
                a, b = int(row[j]), (0 if starts is None else int(starts[s])) + j
                src, dst = int(src_tables[s][a // B]), int(dst_tables[s][b // B])
                k_out[dst, h, b % B] = k_cache[src, h, a % B]
                v_out[dst, h, b % B] = v_cache[src, h, a % B]
    return k_out, v_out
