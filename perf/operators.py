"""Cases of the operators that drop tokens from a paged KV cache: drafted tokens that a verification rejects, and
cached tokens that receive little attention.

  tree     attention of a tree of drafted tokens over a paged cache: every node sees the cached prefix and the nodes
           that its mask names (its ancestors and itself)
  weights  decode attention that also adds each cached token's attention weight, summed over the query heads of its
           kv head, to a running total
  select   the tokens to keep of each sequence and kv head: the latest ones and, of the others, those with the
           largest totals (ties to the lowest position), in ascending order
  compact  moves the kept tokens' K, V and totals to consecutive positions

``run`` computes them in plain torch, or through the package's binding where ``own`` is true.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------

def _case(op, name=None, **kw):
    c = {"op": op, **kw}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # one request with a short draft: what a single interactive user waits for
        _case("tree", "tree_one", seqs=1, heads=32, kv_heads=8, dim=128, block=16, dtype="bf16", lo=1003, hi=1003,
              nodes_lo=16, nodes_hi=16),
        # a serving batch, ragged contexts and drafts
        _case("tree", "tree_batch", seqs=64, heads=32, kv_heads=8, dim=128, block=16, dtype="bf16", lo=128, hi=8191,
              nodes_lo=1, nodes_hi=33),
        # long contexts, 8 query heads to a kv head, wide drafts: several row tiles to one pass over K and V
        _case("tree", "tree_long", seqs=8, heads=64, kv_heads=8, dim=128, block=8, dtype="bf16", lo=8192, hi=32768,
              nodes_lo=24, nodes_hi=64),
        # fp32 pools, as tests and small models use them
        _case("tree", "tree_f32", seqs=4, heads=16, kv_heads=4, dim=64, block=4, dtype="f32", lo=7, hi=1025,
              nodes_lo=1, nodes_hi=24),
        # one request's decode step that keeps the totals
        _case("weights", "weights_one", seqs=1, heads=32, kv_heads=8, dim=128, block=16, dtype="bf16", lo=2000, hi=2000),
        # a layer without shared kv heads at ordinary contexts
        _case("weights", "weights_batch", seqs=64, heads=32, kv_heads=32, dim=128, block=16, dtype="bf16", lo=128, hi=2048),
        # the contexts for which eviction is made
        _case("weights", "weights_long", seqs=8, heads=64, kv_heads=8, dim=128, block=16, dtype="bf16", lo=32768, hi=131072),
        # one request that outgrew its budget
        _case("select", "select_one", seqs=1, kv_heads=8, lo=4097, hi=4097, share=0.25, recent=64),
        # a batch of long contexts cut to a quarter
        _case("select", "select_long", seqs=8, kv_heads=8, lo=32768, hi=131072, share=0.25, recent=256),
        # a batch's accepted paths after a verification, moved up in place
        _case("compact", "compact_tree", seqs=64, kv_heads=8, dim=128, block=16, dtype="bf16", lo=128, hi=8191, nodes=33,
              share=0.0),
        # one long context cut to a quarter
        _case("compact", "compact_one", seqs=1, kv_heads=8, dim=128, block=16, dtype="bf16", lo=32768, hi=32768, nodes=0,
              share=0.25),
        # a batch cut to half into fresh blocks, its prompt blocks being shared with others
        _case("compact", "compact_batch", seqs=64, kv_heads=32, dim=128, block=16, dtype="bf16", lo=128, hi=2048, nodes=0,
              share=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "weights", "select", "compact"])
    kv = rng.choice([1, 2, 4, 8, 16])
    hi = _log(rng, 9, 65536)
    lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
    # rows x length is kept below the largest listed cases
    seqs = max(1, min(_log(rng, 1, 200), 2_000_000 // (hi * kv)))
    if op == "select":
        return _case(op, seqs=seqs, kv_heads=kv, lo=lo, hi=hi, share=round(rng.uniform(0.05, 0.9), 3),
                     recent=rng.choice([0, 1, 7, 32, 129]))
    dim = rng.choice([64, 128])
    block = rng.choice([4, 8, 16, 32])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "compact":
        nodes = rng.choice([0, 9, 31, 64])
        return _case(op, seqs=seqs, kv_heads=kv, dim=dim, block=block, dtype=dtype, lo=lo, hi=hi, nodes=nodes,
                     share=0.0 if nodes else round(rng.uniform(0.05, 0.9), 3))
    group = rng.choice([1, 2, 3, 4, 5, 8])
    if op == "weights":
        return _case(op, seqs=seqs, heads=kv * group, kv_heads=kv, dim=dim, block=block, dtype=dtype, lo=lo, hi=hi)
    if dtype == "f32":
        hi, seqs = min(hi, 4096), min(seqs, 16)
    nodes = rng.choice([3, 7, 16, 25, 50, 100])
    seqs = max(1, min(seqs, 120_000_000 // (nodes * kv * group * hi)))
    return _case(op, seqs=seqs, heads=kv * group, kv_heads=kv, dim=dim, block=block, dtype=dtype, lo=min(lo, hi), hi=hi,
                 nodes_lo=max(1, nodes // 3), nodes_hi=nodes)


# ----------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------

def _ints(lo, hi, n):
    """n whole numbers, uniform in [lo, hi], the largest one among them (the first); the same for every seed, so
    that a case's outputs keep their shapes."""
    v = torch.randint(lo, hi + 1, (n,), generator=torch.Generator().manual_seed(lo * 7919 + hi))
    v[0] = hi
    return v


def _tables(gen, lens, block, spare=0):
    """Shuffled block tables of sequences of lens + spare tokens (int32 [S][max], -1 past the end), and the pool's
    blocks: a tenth more than the tables name."""
    per = [(int(c) + spare + block - 1) // block for c in lens]
    total = sum(per)
    num_blocks = total + max(1, total // 10)
    ids = torch.randperm(num_blocks, generator=gen)[:total].to(torch.int32)
    tables = torch.full((len(per), max(per)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(per):
        tables[s, :n] = ids[at:at + n]
        at += n
    return tables, num_blocks


def _normal(gen, shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)


def _totals(gen, shape):
    """Totals of attention weights: many orders of magnitude apart, and a part of them exactly zero."""
    w = torch.empty(shape, device="cuda").normal_(generator=gen).mul_(2.0).sub_(4.0).exp_()
    return w * (torch.rand(shape, device="cuda", generator=gen) > 0.1)


def _tree(gen, n):
    """Parents of a random tree of n drafted tokens, parents first (-1: the prefix itself)."""
    parents = [-1]
    for i in range(1, n):
        parents.append(int(torch.randint(max(-1, i // 3 - 3), i, (1,), generator=gen)))
    return parents


def _masks(parents, words):
    """Bit j of node i: i is j or descends from j."""
    seen = []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else 0) | (1 << i))
    rows = []
    for m in seen:
        w = [(m >> (64 * k)) & ((1 << 64) - 1) for k in range(words)]
        rows.append([x - (1 << 64) if x >> 63 else x for x in w])
    return rows


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, S, Hkv = case["op"], case["seqs"], case["kv_heads"]
    lens = _ints(case["lo"], case["hi"], S)
    st = {"op": op, "lens_host": lens.tolist(), "lens": lens.to(torch.int32).cuda()}
    if op == "select":
        st["stride"] = int(lens.max())
        st["weights"] = _totals(gen, (S, Hkv, st["stride"]))
        budgets = torch.clamp((lens.double() * case["share"]).long(), min=1)
        st["recent"] = case["recent"]
        st["budgets"] = budgets.to(torch.int32).cuda()
        st["keep"] = torch.full((S, Hkv, int(budgets.max())), -1, dtype=torch.int32, device="cuda")
        st["keep_lens"] = torch.zeros(S, dtype=torch.int32, device="cuda")
        return st

    dtype, D, B = DTYPES[case["dtype"]], case["dim"], case["block"]
    if op == "tree":
        nodes = _ints(case["nodes_lo"], case["nodes_hi"], S)
        lens = torch.maximum(lens, nodes)   # the drafted tokens are in the cache and in the context
        st["lens_host"], st["lens"] = lens.tolist(), lens.to(torch.int32).cuda()
        words = (int(nodes.max()) + 63) // 64
        rows = [r for n in nodes.tolist() for r in _masks(_tree(host, n), words)]
        st["mask"] = torch.tensor(rows, dtype=torch.int64).cuda()
        start = torch.zeros(S + 1, dtype=torch.int32)
        start[1:] = torch.cumsum(nodes, 0)
        st["start"], st["max_nodes"], T = start.cuda(), int(nodes.max()), int(nodes.sum())
        st["q"] = _normal(gen, (T, case["heads"], D), dtype)
        st["out"] = torch.empty_like(st["q"])
    if op == "weights":
        st["q"] = _normal(gen, (S, case["heads"], D), dtype)
        st["out"] = torch.empty_like(st["q"])
        st["stride"] = int(lens.max())
        st["weights"] = _totals(gen, (S, Hkv, st["stride"]))
        st["weights_out"] = torch.zeros_like(st["weights"])
    tables, num_blocks = _tables(host, lens.tolist(), B)
    st["scale"] = 1.0 / math.sqrt(D)
    if op == "compact":
        if case["nodes"]:   # the accepted path of each sequence's draft, for all kv heads alike, moved up in place
            n = torch.clamp(lens, max=case["nodes"])
            keep, keep_lens = [], []
            for s in range(S):
                n_s = int(n[s])
                a = max(1, min(n_s // 4, 8))
                late = torch.randperm(max(0, n_s - a), generator=host)[:a - 1].sort().values
                path = torch.cat([torch.zeros(1, dtype=torch.long), a + late])   # no node moved is one moved onto
                keep.append((int(lens[s]) - n_s + path).tolist())
                keep_lens.append(len(keep[-1]))
            width = max(keep_lens)
            st["keep"] = torch.tensor([[k + [-1] * (width - len(k))] for k in keep], dtype=torch.int32).cuda()
            st["starts"] = (lens - n).to(torch.int32).cuda()
            st["keep_lens"] = torch.tensor(keep_lens, dtype=torch.int32).cuda()
            dst_tables = tables
        else:               # what a selection kept, into fresh blocks
            kept = torch.clamp((lens.double() * case["share"]).long(), min=1)
            width = int(kept.max())
            order = torch.rand((S, Hkv, int(lens.max())), device="cuda", generator=gen)
            order = order.masked_fill(torch.arange(order.shape[2], device="cuda") >= st["lens"][:, None, None], 2.0)
            ranks = order.argsort(-1)[:, :, :width]
            ranks = ranks.masked_fill(torch.arange(width, device="cuda") >= kept.cuda()[:, None, None], 1 << 30)
            st["keep"] = ranks.sort(-1).values.to(torch.int32)
            st["starts"] = None
            st["keep_lens"] = kept.to(torch.int32).cuda()
            dst_tables, more = _tables(host, kept.tolist(), B)
            dst_tables = torch.where(dst_tables >= 0, dst_tables + num_blocks, dst_tables)
            num_blocks += more
            st["weights"] = _totals(gen, (S, Hkv, int(lens.max())))
            st["weights_out"] = torch.zeros_like(st["weights"])
        st["dst_tables"] = dst_tables.cuda()
    st["tables"] = tables.cuda()
    if op == "compact" and case["nodes"]:
        st["dst_tables"] = st["tables"]
    st["k"] = _normal(gen, (num_blocks, Hkv, B, D), dtype)
    st["v"] = _normal(gen, (num_blocks, Hkv, B, D), dtype)
    return st


# ----------------------------------------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------------------------------------

def _rows(pool, tables, length):
    """[S][Hkv][length][d] in 32 bits: the first `length` tokens of every sequence, gathered through its table."""
    S, B = tables.shape[0], pool.shape[2]
    blocks = tables[:, :(length + B - 1) // B].clamp(min=0).long()
    x = pool[blocks]                                             # [S][nb][Hkv][B][d]
    x = x.permute(0, 2, 1, 3, 4).reshape(S, pool.shape[1], -1, pool.shape[3])
    return x[:, :, :length].float()


def _softmax(x, seen):
    """Softmax over the last dimension of what is seen; a row that sees nothing is zero."""
    x = torch.where(seen, x, torch.full((), -math.inf, device=x.device))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def _plain_tree(st):
    q, lens, start = st["q"], st["lens"].long(), st["start"].long()
    T, H, D = q.shape
    S, Hkv, L, N = lens.shape[0], st["k"].shape[1], max(st["lens_host"]), st["max_nodes"]
    n = start[1:] - start[:-1]
    i = torch.arange(N, device=q.device)
    row = (start[:-1, None] + i).clamp(max=T - 1)                 # [S][N] row of each node, padded
    words = st["mask"][row]                                       # [S][N][W]
    pos = torch.arange(L, device=q.device)
    node = pos[None, :] - (lens - n)[:, None]                     # [S][L] node at each position, negative: the prefix
    bit = torch.gather(words, 2, (node.clamp(min=0) // 64).clamp(max=words.shape[2] - 1)[:, None, :].expand(S, N, L))
    bit = (bit >> (node.clamp(min=0) % 64)[:, None, :]) & 1
    seen = ((node < 0)[:, None, :] | (bit == 1)) & (pos[None, :] < lens[:, None])[:, None, :]     # [S][N][L]
    qs = q[row].float().reshape(S, N, Hkv, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, N * (H // Hkv), D)
    x = torch.matmul(qs, _rows(st["k"], st["tables"], L).transpose(2, 3)) * st["scale"]
    x = x.reshape(S, Hkv, N, H // Hkv, L)
    p = _softmax(x, seen[:, None, :, None, :]).reshape(S, Hkv, -1, L)
    o = torch.matmul(p, _rows(st["v"], st["tables"], L)).reshape(S, Hkv, N, H // Hkv, D)
    o = o.permute(0, 2, 1, 3, 4).reshape(S, N, H, D)
    return o[i[None, :] < n[:, None]].to(q.dtype)


def _plain_weights(st):
    q, lens = st["q"], st["lens"].long()
    S, H, D = q.shape
    Hkv, L = st["k"].shape[1], st["stride"]
    x = torch.matmul(q.float().reshape(S, Hkv, H // Hkv, D), _rows(st["k"], st["tables"], L).transpose(2, 3)) * st["scale"]
    seen = (torch.arange(L, device=q.device) < lens[:, None])[:, None, :]
    p = _softmax(x, seen[:, :, None, :])
    o = torch.matmul(p, _rows(st["v"], st["tables"], L)).reshape(S, H, D).to(q.dtype)
    return o, torch.where(seen, st["weights"] + p.sum(2), st["weights_out"])


def _plain_select(st):
    w, lens, budgets = st["weights"], st["lens"].long()[:, None, None], st["budgets"].long()[:, None, None]
    pos = torch.arange(w.shape[2], device=w.device)
    recent = torch.clamp(budgets, max=st["recent"])
    key = torch.where(torch.isnan(w), torch.full_like(w, -math.inf), w).double()
    # kept without regard to their totals, and never kept, sort before and behind all others
    key = torch.where(pos >= lens - recent, torch.full_like(key, math.inf), key)
    order = torch.where(pos < lens, key, torch.full_like(key, -math.inf)).sort(stable=True, dim=-1, descending=True).indices
    kept = torch.minimum(lens, budgets)
    width = st["keep"].shape[2]
    j = torch.arange(width, device=w.device)
    first = torch.where(j < kept, order[:, :, :width], torch.full((), 1 << 40, device=w.device)).sort(-1).values
    return torch.where(j < kept, first, st["keep"].long()).to(torch.int32), kept[:, 0, 0].to(torch.int32)


def _plain_compact(st):
    k, v, keep, B = st["k"], st["v"], st["keep"].long(), st["k"].shape[2]
    S, Hkv = keep.shape[0], k.shape[1]
    keep = keep.expand(S, Hkv, keep.shape[2])
    j = torch.arange(keep.shape[2], device=k.device)
    to = (j if st["starts"] is None else st["starts"].long()[:, None, None] + j).expand_as(keep)
    live = (j < st["keep_lens"].long()[:, None, None]).expand_as(keep)
    s, h, _ = torch.nonzero(live, as_tuple=True)
    a, b = keep[live], to[live]
    src, dst = st["tables"].long()[s, a // B], st["dst_tables"].long()[s, b // B]
    k[dst, h, b % B] = k[src, h, a % B]
    v[dst, h, b % B] = v[src, h, a % B]
    if "weights" not in st:
        return k, v
    st["weights_out"][s, h, b] = st["weights"][s, h, a]
    return k, v, st["weights_out"]


def _own(st):
    from paged_kv_cache_382_b200 import pa

    op = st["op"]
    if op in ("tree", "weights") and "ws" not in st:   # a serving program plans its workspaces once
        st["ws"] = (pa.alloc_tree_workspace(st["q"].shape[0], st["q"].shape[1], st["q"].shape[2]) if op == "tree" else
                    pa.alloc_weights_workspace(st["q"].shape[0], st["q"].shape[1], st["q"].shape[2], st["stride"]))
    if op == "tree":
        return pa.tree_decode(st["out"], st["q"], st["k"], st["v"], st["tables"], st["lens"], st["start"], st["mask"],
                              st["scale"], workspace=st["ws"])
    if op == "weights":
        pa.decode_weights(st["out"], st["weights_out"], st["q"], st["k"], st["v"], st["tables"], st["lens"], st["scale"],
                          weights_in=st["weights"], max_context_len=st["stride"], workspace=st["ws"])
        return st["out"], st["weights_out"]
    if op == "select":
        pa.select_tokens(st["keep"], st["keep_lens"], st["weights"], st["lens"], st["budgets"], recent=st["recent"])
        return st["keep"], st["keep_lens"]
    if "weights" not in st:
        pa.compact(st["k"], st["v"], st["tables"], st["dst_tables"], st["keep"], st["keep_lens"], starts=st["starts"])
        return st["k"], st["v"]
    pa.compact(st["k"], st["v"], st["tables"], st["dst_tables"], st["keep"], st["keep_lens"], starts=st["starts"],
               weights_in=st["weights"], weights_out=st["weights_out"])
    return st["k"], st["v"], st["weights_out"]


def run(state):
    if own:
        return _own(state)
    plain = {"tree": _plain_tree, "weights": _plain_weights, "select": _plain_select, "compact": _plain_compact}
    return plain[state["op"]](state)


# ----------------------------------------------------------------------------------------------------------------
# work and exact values
# ----------------------------------------------------------------------------------------------------------------

def _mean(lo, hi, n):
    """Sum of n lengths, the first `hi` and the others uniform in [lo, hi]."""
    return hi + (n - 1) * (lo + hi) / 2.0


def work(case):
    op, S, Hkv = case["op"], case["seqs"], case["kv_heads"]
    tokens = _mean(case["lo"], case["hi"], S)
    if op == "select":   # every total read, every kept position written
        return {"bytes": Hkv * tokens * 4.0 * (1.0 + case["share"]) + 12.0 * S, "flops": 0.0}
    e, D = (2 if case["dtype"] == "bf16" else 4), case["dim"]
    row = D * e
    if op == "compact":  # every kept K and V row read and written, and where it comes from
        if case["nodes"]:
            kept = S * max(1.0, min(case["nodes"] // 4, 8))
            return {"bytes": kept * (Hkv * 4.0 * row + 4.0), "flops": 0.0}
        kept = tokens * case["share"]
        return {"bytes": kept * Hkv * (4.0 * row + 12.0), "flops": 0.0}
    # K and V of every token read once, queries read, outputs written
    kv = tokens * Hkv * 2.0 * row + tokens / case["block"] * 4.0
    if op == "weights":  # and every total read and written
        return {"bytes": kv + 2.0 * S * case["heads"] * row + tokens * Hkv * 8.0, "flops": 4.0 * tokens * case["heads"] * D}
    nodes = _mean(case["nodes_lo"], case["nodes_hi"], S)
    return {"bytes": kv + 2.0 * nodes * case["heads"] * row + nodes * 8.0,
            "flops": 4.0 * tokens * (nodes / S) * case["heads"] * D}


def _gathered(pool, table, length, head):
    """[length][d] in 64 bits: one kv head of one sequence."""
    B = pool.shape[2]
    t = torch.arange(length, device=pool.device)
    return pool[table.long()[t // B], head, t % B].double()


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "select":
        return None      # whole numbers
    if op == "compact":
        pools = [st["k"].double(), st["v"].double()]
        totals = st["weights_out"].double() if "weights" in st else None
        starts = [0] * len(st["lens_host"]) if st["starts"] is None else st["starts"].tolist()
        B = case["block"]
        for s, n in enumerate(st["keep_lens"].tolist()):
            to = starts[s] + torch.arange(n, device="cuda")
            for h in range(case["kv_heads"]):
                a = st["keep"][s, h if st["keep"].shape[1] > 1 else 0, :n].long()
                for pool, given in zip(pools, (st["k"], st["v"])):
                    pool[st["dst_tables"][s].long()[to // B], h, to % B] = given[st["tables"][s].long()[a // B], h, a % B].double()
                if totals is not None:
                    totals[s, h, to] = st["weights"][s, h, a].double()
        return tuple(pools) if totals is None else (*pools, totals)
    heavy = sum(st["lens_host"]) * case["heads"] * case["dim"] * (case["nodes_hi"] if op == "tree" else 1)
    if heavy > 4e12:
        return None
    k, v, tables, q = st["k"], st["v"], st["tables"], st["q"]
    group = case["heads"] // case["kv_heads"]
    scale = torch.tensor(st["scale"], dtype=torch.float32).double().item()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    totals = st["weights_out"].double() if op == "weights" else None
    start = st["start"].tolist() if op == "tree" else list(range(len(st["lens_host"]) + 1))
    for s, length in enumerate(st["lens_host"]):
        a, b = start[s], start[s + 1]
        hidden = torch.zeros((b - a, length), dtype=torch.bool, device=q.device)
        if op == "tree":
            at = torch.arange(b - a, device=q.device)
            hidden[:, length - (b - a):] = (st["mask"][a:b][:, at // 64] >> (at % 64)) & 1 == 0
        for h in range(case["kv_heads"]):
            keys, values = _gathered(k, tables[s], length, h), _gathered(v, tables[s], length, h)
            x = torch.einsum("ngd,ld->ngl", q[a:b, h * group:(h + 1) * group].double(), keys) * scale
            e = torch.exp(x.masked_fill(hidden[:, None, :], -math.inf) - x.amax(-1, keepdim=True))
            p = e / e.sum(-1, keepdim=True)
            out[a:b, h * group:(h + 1) * group] = torch.einsum("ngl,ld->ngd", p, values)
            if op == "weights":
                totals[s, h, :length] = st["weights"][s, h, :length].double() + p.sum((0, 1))
    return (out, totals) if op == "weights" else out
